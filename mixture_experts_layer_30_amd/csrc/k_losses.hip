// The router's losses (balance, z) with the counts and probability sums under
// them, and the gradient of the logits.
//
// Per token p = softmax(l), lse = log sum exp l. Forward: counts c_e of the
// chosen experts, P_e = sum_t p_te, balance = E / (k n^2) sum c_e P_e,
// z = 1/n sum lse^2. Backward: d_te = gb E / (k n^2) p_te (c_e - sum_f c_f p_tf)
// + gz 2/n lse_t p_te, and through the combine weights w_j (g_j - sum w g) at
// each chosen expert. As the p of a token add up to 1, c may be taken from its
// mean k n / E in that difference; then nearly even counts lose no digits.
//
// Both are one pass over the logits and bound by reading (and writing) them. A
// token lies in L lanes of a wavefront, 4 I experts each (lane l: the experts
// 4 (l + L i) .. + 3), so a wavefront works on 64 / L tokens at once.
#include <type_traits>

#include "mok_device.h"
#include "router_launch.h"

namespace {

constexpr int kBT = 256, kWaves = kBT / 64;
constexpr int kGroups = 512;                     // most workgroups of the forward

template <int L>
MOK_DEV float group_max(float v) {
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <int L>
MOK_DEV float group_sum(float v) {
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// this lane's logits of one row; -infinity past E and in rows that are left out
template <int L, int I, bool VEC>
MOK_DEV void load_row(const float* row, int E, int l, bool live, float v[I][4]) {
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int e = 4 * (l + L * i);
    v[i][0] = v[i][1] = v[i][2] = v[i][3] = -INFINITY;
    if constexpr (VEC) {
      if (live && e < E) {
        const float4 q = *reinterpret_cast<const float4*>(row + e);
        v[i][0] = q.x; v[i][1] = q.y; v[i][2] = q.z; v[i][3] = q.w;
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (live && e + u < E) v[i][u] = row[e + u];
    }
  }
}

// v becomes exp(v - max); returns the sum's reciprocal and lse. A row of nothing
// but -infinity has zeros for all three; a NaN stays one.
template <int L, int I>
MOK_DEV void softmax_row(float v[I][4], float& inv, float& lse) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < I; ++i) top = fmaxf(top, fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])));
  top = group_max<L>(top);
  if (top == -INFINITY) top = 0.f;
  float den = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[i][u] = expf(v[i][u] - top);
      den += v[i][u];
    }
  den = group_sum<L>(den);
  const bool none = den == 0.f;
  inv = none ? 0.f : 1.0f / den;
  lse = none ? 0.f : top + logf(den);
}

// losses from the sums (one workgroup; prob and counts in memory it can read)
MOK_DEV void finish(const mok_losses_args& a, const float* prob, const int32_t* counts, float z, int n,
                    double (*red)[kBT]) {
  double s = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kBT) s += (double)counts[e] * (double)prob[e];
  (*red)[threadIdx.x] = s;
  __syncthreads();
  for (int d = kBT / 2; d >= 1; d >>= 1) {
    if ((int)threadIdx.x < d) (*red)[threadIdx.x] += (*red)[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double dn = n;
    a.losses[0] = n ? (float)((*red)[0] * a.E / (a.k * dn * dn)) : 0.f;
    a.losses[1] = n ? (float)((double)z / dn) : 0.f;
    a.n[0] = n;
  }
}

template <int L, int I, bool VEC>
__global__ __launch_bounds__(kBT) void losses_rows_kernel(const mok_losses_args a) {
  constexpr int SPW = 64 / L, TPB = kWaves * SPW;
  __shared__ int hist[512];
  __shared__ float ps[kWaves][512];
  __shared__ float zs[kWaves];
  __shared__ int ns[kWaves];
  __shared__ double red[kBT];
  const int lane = lane_id(), wave = (int)threadIdx.x >> 6, l = lane % L;
  for (int e = threadIdx.x; e < a.E; e += kBT) hist[e] = 0;
  __syncthreads();
  float acc[I][4];
#pragma unroll
  for (int i = 0; i < I; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  float z = 0.f;
  int n = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.T; t0 += (int64_t)gridDim.x * TPB) {
    const int64_t t = t0 + wave * SPW + lane / L;
    const bool live = t < a.T && (!a.mask || a.mask[t]);
    float v[I][4], inv, lse;
    load_row<L, I, VEC>(a.logits + t * a.E, a.E, l, live, v);
    if (live)
      for (int j = l; j < a.k; j += L) {
        const int id = a.ids[t * a.k + j];
        if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);      // integers: the order does not matter
      }
    softmax_row<L, I>(v, inv, lse);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[i][u] = fmaf(v[i][u], inv, acc[i][u]);
    if (l == 0 && live) {
      z = fmaf(lse, lse, z);
      ++n;
    }
  }
  // the tokens of a wavefront, then the wavefronts in ascending order
#pragma unroll
  for (int d = L; d < 64; d <<= 1) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[i][u] += __shfl_xor(acc[i][u], d);
    z += __shfl_xor(z, d);
    n += __shfl_xor(n, d);
  }
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (4 * (l + L * i) + u < 512) ps[wave][4 * (l + L * i) + u] = acc[i][u];
  }
  if (lane == 0) {
    zs[wave] = z;
    ns[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kWaves; ++w) {
      zs[0] += zs[w];
      ns[0] += ns[w];
    }
  const bool alone = gridDim.x == 1;
  uint32_t* part = a.part + (int64_t)blockIdx.x * (2 * a.E + 2);
  for (int e = threadIdx.x; e < a.E; e += kBT) {
    float p = ps[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) p += ps[w][e];
    if (alone) {
      a.prob[e] = ps[0][e] = p;
      a.counts[e] = hist[e];
    } else {
      part[e] = __float_as_uint(p);
      part[a.E + e] = (uint32_t)hist[e];
    }
  }
  __syncthreads();
  if (alone) {
    finish(a, ps[0], hist, zs[0], ns[0], &red);
  } else if (threadIdx.x == 0) {
    part[2 * a.E] = __float_as_uint(zs[0]);
    part[2 * a.E + 1] = (uint32_t)ns[0];
    // the next launch's count of finished workgroups
    if (blockIdx.x == 0) a.part[(int64_t)gridDim.x * (2 * a.E + 2)] = 0;
  }
}

// The workgroups' sums, in ascending order: 32 experts a workgroup, eight groups
// of partial rows each; the workgroup that ends last forms the losses.
__global__ __launch_bounds__(kBT) void losses_join_kernel(const mok_losses_args a, int groups) {
  __shared__ float pg[8][32];
  __shared__ int cg[8][32];
  __shared__ double red[kBT];
  __shared__ int last;
  const int64_t pitch = 2 * a.E + 2;
  const int c = (int)threadIdx.x & 31, r = (int)threadIdx.x >> 5, e = (int)blockIdx.x * 32 + c;
  float p = 0.f;
  int n = 0;
  if (e < a.E)
    for (int i = r; i < groups; i += 8) {
      p += __uint_as_float(a.part[i * pitch + e]);
      n += (int)a.part[i * pitch + a.E + e];
    }
  pg[r][c] = p;
  cg[r][c] = n;
  __syncthreads();
  if (r == 0 && e < a.E) {
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      p += pg[i][c];
      n += cg[i][c];
    }
    a.prob[e] = p;
    a.counts[e] = n;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.part + groups * pitch, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // z and n of the workgroups: one or two a thread, then halves in a fixed order
  double z = 0.0;
  int m = 0;
  for (int i = threadIdx.x; i < groups; i += kBT) {
    z += (double)__uint_as_float(a.part[i * pitch + 2 * a.E]);
    m += (int)a.part[i * pitch + 2 * a.E + 1];
  }
  int* im = &cg[0][0];
  red[threadIdx.x] = z;
  im[threadIdx.x] = m;
  __syncthreads();
  for (int d = kBT / 2; d >= 1; d >>= 1) {
    if ((int)threadIdx.x < d) {
      red[threadIdx.x] += red[threadIdx.x + d];
      im[threadIdx.x] += im[threadIdx.x + d];
    }
    __syncthreads();
  }
  const float zz = (float)red[0];
  m = im[0];
  __syncthreads();
  finish(a, a.prob, a.counts, zz, m, &red);
}

template <int L, int I, bool VEC>
__global__ __launch_bounds__(kBT) void losses_bwd_kernel(const mok_losses_args a) {
  constexpr int SPW = 64 / L, TPB = kWaves * SPW;
  __shared__ __attribute__((aligned(16))) float sel[kWaves][SPW][4 * L * I];   // d of the chosen logits, by expert
  const int lane = lane_id(), wave = (int)threadIdx.x >> 6, l = lane % L;
  float* mine = sel[wave][lane / L];
#pragma unroll
  for (int i = 0; i < I; ++i) *reinterpret_cast<float4*>(mine + 4 * (l + L * i)) = make_float4(0.f, 0.f, 0.f, 0.f);
  const int n = a.n[0];
  const double dn = n ? (double)n : 1.0;
  const float gb = n ? a.d_losses[0] : 0.f, gz = n ? (float)(2.0 * (double)a.d_losses[1] / dn) : 0.f;
  // E / (k n^2) (c_e - k n / E)
  float ce[I][4];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 4 * (l + L * i) + u;
      ce[i][u] = 0.f;
      if (e < a.E && n)
        ce[i][u] = (float)((double)((int64_t)a.E * a.counts[e] - (int64_t)a.k * n) / (a.k * dn * dn));
    }
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.T; t0 += (int64_t)gridDim.x * TPB) {
    const int64_t t = t0 + wave * SPW + lane / L;
    const bool in = t < a.T, live = in && (!a.mask || a.mask[t]);
    float v[I][4], inv, lse;
    load_row<L, I, VEC>(a.logits + t * a.E, a.E, l, live, v);
    if (a.w) {
      float s = 0.f;
      if (in)
        for (int j = l; j < a.k; j += L) s = fmaf(a.w[t * a.k + j], a.g[t * a.k + j], s);
      s = group_sum<L>(s);
      // one pick of every token after the other: an expert picked twice adds up in the order of the picks
      for (int j0 = 0; j0 < a.k; j0 += L) {
        int id = -1;
        float d = 0.f;
        if (in && j0 + l < a.k) {
          const int64_t at = t * a.k + j0 + l;
          id = a.ids[at];
          d = a.w[at] * (a.g[at] - s);
        }
        const int m = min(L, a.k - j0);
        for (int j = 0; j < m; ++j) {
          if (l == j && id >= 0 && id < a.E)
            (void)__hip_atomic_fetch_add(mine + id, d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
          __builtin_amdgcn_wave_barrier();       // (keeps the picks one instruction each)
        }
      }
    }
    softmax_row<L, I>(v, inv, lse);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[i][u] *= inv;
        s = fmaf(v[i][u], ce[i][u], s);
      }
    s = group_sum<L>(s);
    const float zt = gz * lse;
    // the wavefront's LDS writes above land in order before its reads here
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int e = 4 * (l + L * i);
      float o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = live ? v[i][u] * fmaf(gb, ce[i][u] - s, zt) : 0.f;
      if (a.w) {
        float4* at = reinterpret_cast<float4*>(mine + e);
        const float4 q = *at;
        *at = make_float4(0.f, 0.f, 0.f, 0.f);
        o[0] += q.x; o[1] += q.y; o[2] += q.z; o[3] += q.w;
      }
      float* d = a.d_logits + t * a.E + e;
      if constexpr (VEC) {
        if (in && e < a.E) *reinterpret_cast<float4*>(d) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (in && e + u < a.E) d[u] = o[u];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// f(L, I, whether rows are whole float4s) as constants
template <class F>
auto by_experts(int E, F&& f) {
  using std::integral_constant;
#define MOK_EXPERTS(l, i)                                                                                         \
  if (E <= 4 * (l) * (i))                                                                                         \
    return E % 4 == 0 ? f(integral_constant<int, l>{}, integral_constant<int, i>{}, std::true_type{})             \
                      : f(integral_constant<int, l>{}, integral_constant<int, i>{}, std::false_type{})
  MOK_EXPERTS(2, 1);
  MOK_EXPERTS(4, 1);
  MOK_EXPERTS(8, 1);
  MOK_EXPERTS(16, 1);
  MOK_EXPERTS(32, 1);
  MOK_EXPERTS(64, 1);
  MOK_EXPERTS(64, 2);
#undef MOK_EXPERTS
  return decltype(f(integral_constant<int, 64>{}, integral_constant<int, 2>{}, std::true_type{}))();
}

int groups_of(int64_t T, int L) {
  const int tpb = kWaves * 64 / L;
  const int64_t blocks = (T + tpb - 1) / tpb;
  return (int)(blocks < 1 ? 1 : blocks < kGroups ? blocks : kGroups);
}

}  // namespace

size_t mok_losses_part_bytes(int64_t T, int E) {
  const int groups = by_experts(E, [&](auto L, auto, auto) { return groups_of(T, decltype(L)::value); });
  return groups > 1 ? ((size_t)groups * (2 * E + 2) + 1) * 4 : 0;
}

hipError_t mok_launch_losses(const mok_losses_args& a, hipStream_t st) {
  const int groups = by_experts(a.E, [&](auto L, auto I, auto vec) {
    const int g = groups_of(a.T, decltype(L)::value);
    hipLaunchKernelGGL((losses_rows_kernel<decltype(L)::value, decltype(I)::value, decltype(vec)::value>),
                       dim3((unsigned)g), dim3(kBT), 0, st, a);
    return g;
  });
  if (groups > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(losses_join_kernel, dim3((unsigned)((a.E + 31) / 32)), dim3(kBT), 0, st, a, groups);
  }
  return hipGetLastError();
}

hipError_t mok_launch_losses_backward(const mok_losses_args& a, hipStream_t st) {
  if (a.T <= 0) return hipSuccess;
  by_experts(a.E, [&](auto L, auto I, auto vec) {
    const int tpb = kWaves * 64 / decltype(L)::value;
    const int64_t blocks = (a.T + tpb - 1) / tpb, cap = 2048;
    hipLaunchKernelGGL((losses_bwd_kernel<decltype(L)::value, decltype(I)::value, decltype(vec)::value>),
                       dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(kBT), 0, st, a);
    return 0;
  });
  return hipGetLastError();
}
