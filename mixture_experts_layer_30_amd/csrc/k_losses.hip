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
// Both are one pass over the logits and bound by reading (and writing) them, small
// ones by latency. A token lies in L lanes of a wavefront, 4 I experts each (lane l:
// the experts 4 (l + L i) .. + 3), so a wavefront works on 64 / L tokens at once.
// 65536 tokens x 512 experts: forward 36 us for 134 MB and 9 us for the joining of
// the sums, gradient 46 us for 268 MB (5.8 TB/s); 16384 x 128: 5.8, 6.5 and 8.8 us.
// Tried and dropped: several rows side by side in a lane, and loading a row ahead
// (the forward as it is, the gradient 5 to 10 us longer for its registers and LDS);
// joining in one launch whose last workgroup goes on (every wavefront's fence writes
// an L2 back: 15 us at 203 tokens).
#include <algorithm>
#include <type_traits>

#include "lane_reduce.h"
#include "router_launch.h"

namespace {

constexpr int kBT = 256, kWaves = kBT / 64;      // backward
// forward: few large workgroups, so that few partial sums have to be added
constexpr int kFT = 1024, kFWaves = kFT / 64;
constexpr int kGroups = 256;                     // most of them
// Passes that one workgroup makes by itself, without a second launch that joins: both losses' calls of 1024 to 2048
// tokens x 8 10.1 us, 11.3 where two passes are split up; 203 x 37 10.7, 10.8; 60 x 512 12.6, 13.2. Where eight passes
// stay with one, 400 x 37 takes 13.3 us, not 11.1, and 256 x 128 13.8, not 10.9.
constexpr int kAlone = 4;

// LDS accesses of a wavefront's lanes above land before those below
MOK_DEV void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

// exp(x) for x <= 0, 0 from -200 down, NaN for NaN: within 4 * 2^-24 of itself, whatever x. What the product with
// log2(e) = 0x1.715476p+0 + 0x1.4ae0cp-26 loses, r < 2^-15.5, goes in as 2^r = 1 + r log(2), which leaves r^2 / 4 <
// 2^-33. (Without it the result is off by up to 1.3 |x| 2^-24, and both calls at 65536 x 512 take 87.5 us, not 89.7.)
MOK_DEV float exp_neg(float x) {
  x = __builtin_elementwise_maximum(x, -200.f);
  const float t = x * 0x1.715476p+0f, e = __builtin_amdgcn_exp2f(t);
  const float r = fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -t));
  return fmaf(e, r * 0x1.62e43p-1f, e);
}

// v becomes exp(v - max); returns the sum's reciprocal and lse. A row of nothing
// but -infinity has zeros for all three; a NaN stays one.
template <int L, int I>
MOK_DEV void softmax_row(float v[I][4], float& inv, float& lse) {
  float top = -INFINITY, den = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i) top = fmaxf(top, fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])));
  top = lanes_max<L>(top);
  if (top == -INFINITY) top = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[i][u] = exp_neg(v[i][u] - top);
      den += v[i][u];
    }
  den = lanes_sum<L>(den);
  const bool none = den == 0.f;
  const float r = __builtin_amdgcn_rcpf(den);
  inv = none ? 0.f : fmaf(r, fmaf(-den, r, 1.0f), r);
  lse = none ? 0.f : top + __logf(den);
}

// the sum of v over a workgroup of BT threads, in its first thread: within the
// wavefronts, then theirs in ascending order
template <int BT>
MOK_DEV double block_sum(double v, double* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if (lane_id() == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < BT / 64; ++w) v += red[w];
  return v;
}

// losses from the sums, by one workgroup of BT threads: cp is this thread's share of sum counts prob
template <int BT>
MOK_DEV void finish(const mok_losses_args& a, double cp, double z, int n, double* red) {
  cp = block_sum<BT>(cp, red);
  if (threadIdx.x != 0) return;
  const double dn = n;
  a.losses[0] = n ? (float)(cp * a.E / (a.k * dn * dn)) : 0.f;
  a.losses[1] = n ? (float)(z / dn) : 0.f;
  a.n[0] = n;
}

template <int L, int I, bool VEC>
__global__ __launch_bounds__(kFT) void losses_rows_kernel(const mok_losses_args a) {
  constexpr int SPW = 64 / L, TPB = kFWaves * SPW;
  __shared__ int hist[512];
  __shared__ __attribute__((aligned(16))) float ps[kFWaves][4 * L * I];
  __shared__ double zs[kFWaves];
  __shared__ int ns[kFWaves];
  __shared__ double red[kFWaves];
  const int lane = lane_id(), wave = (int)threadIdx.x >> 6, l = lane % L;
  for (int e = threadIdx.x; e < a.E; e += kFT) hist[e] = 0;
  __syncthreads();
  float acc[I][4];
#pragma unroll
  for (int i = 0; i < I; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  double z = 0.0;                                // one term a token: in 64 bits it costs nothing
  int n = 0;
  const int64_t step = (int64_t)gridDim.x * TPB, t0 = (int64_t)blockIdx.x * TPB;
  const int at = wave * SPW + lane / L;
  int64_t left = a.T - t0;                       // tokens from this pass's first one on
  const float* row = a.logits + (t0 + at) * a.E;
  const int32_t* ids = a.ids + (t0 + at) * a.k;
  const uint8_t* mask = a.mask + (t0 + at);
  for (; left > 0; left -= step, row += step * a.E, ids += step * a.k, mask += step) {
    const bool live = at < left && (!a.mask || *mask);
    float v[I][4], inv, lse;
    load_row<L, I, VEC>(row, a.E, l, live, v);
    if (live)
      for (int j = l; j < a.k; j += L) {
        const int id = ids[j];
        if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);      // integers: the order does not matter
      }
    softmax_row<L, I>(v, inv, lse);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[i][u] = fmaf(v[i][u], inv, acc[i][u]);
    if (l == 0 && live) {
      z = fma((double)lse, (double)lse, z);
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
      *reinterpret_cast<float4*>(&ps[wave][4 * (l + L * i)]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  }
  if (lane == 0) {
    zs[wave] = z;
    ns[wave] = n;
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  uint32_t* part = a.part + (int64_t)blockIdx.x * (2 * a.E + 2);
  double cp = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kFT) {
    float p = ps[0][e];
#pragma unroll
    for (int w = 1; w < kFWaves; ++w) p += ps[w][e];
    if (alone) {
      a.prob[e] = p;
      a.counts[e] = hist[e];
      cp += (double)hist[e] * (double)p;
    } else {
      part[e] = __float_as_uint(p);
      part[a.E + e] = (uint32_t)hist[e];
    }
  }
  z = zs[0];
  n = ns[0];
#pragma unroll
  for (int w = 1; w < kFWaves; ++w) {
    z += zs[w];
    n += ns[w];
  }
  if (alone) {
    finish<kFT>(a, cp, z, n, red);
  } else if (threadIdx.x == 0) {
    part[2 * a.E] = __float_as_uint((float)z);   // (rounded once, and added in 64 bits again)
    part[2 * a.E + 1] = (uint32_t)n;
  }
}

// The workgroups' sums, in a fixed order: 32 experts a workgroup, its threads in
// kJR rows that add every kJR-th partial row each, then the rows in ascending
// order.
constexpr int kJR = 32, kJT = 32 * kJR;
__global__ __launch_bounds__(kJT) void losses_join_kernel(const mok_losses_args a, int groups) {
  __shared__ float pg[kJR][32];
  __shared__ int cg[kJR][32];
  const int pitch = 2 * a.E + 2;
  const int c = (int)threadIdx.x & 31, r = (int)threadIdx.x >> 5, e = (int)blockIdx.x * 32 + c;
  float p = 0.f;
  int n = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int i = r; i < groups; i += kJR) {
      p += __uint_as_float(a.part[(int64_t)i * pitch + e]);
      n += (int)a.part[(int64_t)i * pitch + a.E + e];
    }
  }
  pg[r][c] = p;
  cg[r][c] = n;
  __syncthreads();
  if (r != 0 || e >= a.E) return;
#pragma unroll
  for (int i = 1; i < kJR; ++i) {
    p += pg[i][c];
    n += cg[i][c];
  }
  a.prob[e] = p;
  a.counts[e] = n;
}

// The same for up to C experts by one workgroup, which goes on to the losses: rows
// of C threads. (Both losses' calls at 65536 x 8: 12.4 us, 13.7 with two launches;
// 16384 x 64: 14.2, 15.7; 16384 x 128: 21.0 either way; 256 experts: 27.0, 23.8.)
template <int C>
__global__ __launch_bounds__(1024) void losses_join_finish_kernel(const mok_losses_args a, int groups) {
  constexpr int R = 1024 / C;
  __shared__ float pg[R][C];
  __shared__ int cg[R][C];
  __shared__ double red[16], rz[16];
  __shared__ int rn[16];
  const int pitch = 2 * a.E + 2;
  const int e = (int)threadIdx.x % C, r = (int)threadIdx.x / C;
  float p = 0.f;
  double z = 0.0;
  int n = 0, m = 0;
  if ((int)threadIdx.x < groups) {
    z = (double)__uint_as_float(a.part[(int64_t)threadIdx.x * pitch + 2 * a.E]);
    m = (int)a.part[(int64_t)threadIdx.x * pitch + 2 * a.E + 1];
  }
  if (e < a.E) {
#pragma unroll 16
    for (int i = r; i < groups; i += R) {
      p += __uint_as_float(a.part[(int64_t)i * pitch + e]);
      n += (int)a.part[(int64_t)i * pitch + a.E + e];
    }
  }
  pg[r][e] = p;
  cg[r][e] = n;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m += __shfl_xor(m, d);
  if (lane_id() == 0) rn[threadIdx.x >> 6] = m;
  z = block_sum<1024>(z, rz);
  m = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) m += rn[w];
  double cp = 0.0;
  if (r == 0 && e < a.E) {
#pragma unroll
    for (int i = 1; i < R; ++i) {
      p += pg[i][e];
      n += cg[i][e];
    }
    a.prob[e] = p;
    a.counts[e] = n;
    cp = (double)n * (double)p;
  }
  finish<1024>(a, cp, z, m, red);
}

// the losses, from the joined sums and the workgroups' z and n
__global__ __launch_bounds__(512) void losses_finish_kernel(const mok_losses_args a, int groups) {
  __shared__ double red[8], rz[8];
  __shared__ int rn[8];
  const int pitch = 2 * a.E + 2;
  const int e = (int)threadIdx.x;
  const double cp = e < a.E ? (double)a.counts[e] * (double)a.prob[e] : 0.0;
  double z = 0.0;
  int n = 0;
  for (int i = threadIdx.x; i < groups; i += 512) {
    z += (double)__uint_as_float(a.part[(int64_t)i * pitch + 2 * a.E]);
    n += (int)a.part[(int64_t)i * pitch + 2 * a.E + 1];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d);
  if (lane_id() == 0) rn[threadIdx.x >> 6] = n;
  z = block_sum<512>(z, rz);
  n = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) n += rn[w];
  finish<512>(a, cp, z, n, red);
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
  const double per = n ? 1.0 / (double)n : 0.0, share = n ? (double)a.d_losses[0] * per * per / a.k : 0.0;
  const float gz = n ? (float)(2.0 * (double)a.d_losses[1] * per) : 0.f;
  // gb E / (k n^2) (c_e - k n / E)
  float ce[I][4];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 4 * (l + L * i) + u;
      ce[i][u] = 0.f;
      if (e < a.E) ce[i][u] = (float)((double)((int64_t)a.E * a.counts[e] - (int64_t)a.k * n) * share);
    }
  const int64_t step = (int64_t)gridDim.x * TPB, t0 = (int64_t)blockIdx.x * TPB;
  const int at = wave * SPW + lane / L;
  int64_t left = a.T - t0;                       // tokens from this pass's first one on
  const float* row = a.logits + (t0 + at) * a.E;
  float* out = a.d_logits + (t0 + at) * a.E;
  const uint8_t* mask = a.mask + (t0 + at);
  int64_t pick = (t0 + at) * a.k + l;
  for (; left > 0; left -= step, row += step * a.E, out += step * a.E, mask += step, pick += step * a.k) {
    const bool in = at < left, live = in && (!a.mask || *mask);
    // the first L picks, one a lane, are loaded with the row
    int id = -1;
    float v[I][4], w = 0.f, g = 0.f;
    if (a.w && in && l < a.k) {
      id = a.ids[pick];
      w = a.w[pick];
      g = a.g[pick];
    }
    load_row<L, I, VEC>(row, a.E, l, live, v);
    if (a.w) {
      float s = w * g;
      if (in)
        for (int j = L; j + l < a.k; j += L) s = fmaf(a.w[pick + j], a.g[pick + j], s);
      s = lanes_sum<L>(s);
      for (int j = 0; j < a.k; j += L) {
        if (j > 0) {
          const bool more = in && j + l < a.k;
          id = more ? a.ids[pick + j] : -1;
          w = more ? a.w[pick + j] : 0.f;
          g = more ? a.g[pick + j] : 0.f;
        }
        const float d = w * (g - s);
        const bool ok = id >= 0 && id < a.E;
        const float old = ok && a.k > L ? mine[id] : 0.f;
        wave_order();
        if (ok) (void)__hip_atomic_fetch_add(mine + id, d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
        wave_order();
        // Another pick of the same expert has been added as well: once more, one pick of each token after the other,
        // so that they add up in the order of the picks. (Where none sees the others, all are zeros.)
        if (__ballot(ok && mine[id] != old + d)) {
          wave_order();
          if (ok) mine[id] = old;
          for (int q = 0; q < L; ++q) {
            wave_order();
            if (l == q && ok) mine[id] += d;
          }
        }
        wave_order();
      }
    }
    float inv, lse, s = 0.f;
    softmax_row<L, I>(v, inv, lse);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[i][u] *= inv;
        s = fmaf(v[i][u], ce[i][u], s);
      }
    s = lanes_sum<L>(s);
    const float rest = fmaf(gz, lse, -s);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int e = 4 * (l + L * i);
      float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.w) {
        d = *reinterpret_cast<const float4*>(mine + e);
        *reinterpret_cast<float4*>(mine + e) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      // (not 0 times the coefficients in rows that are left out: a loss's gradient may have overflowed)
      if (live) {
        d.x = fmaf(v[i][0], ce[i][0] + rest, d.x);
        d.y = fmaf(v[i][1], ce[i][1] + rest, d.y);
        d.z = fmaf(v[i][2], ce[i][2] + rest, d.z);
        d.w = fmaf(v[i][3], ce[i][3] + rest, d.w);
      }
      if constexpr (VEC) {
        if (in && e < a.E) *reinterpret_cast<float4*>(out + e) = d;
      } else {
        if (in && e < a.E) out[e] = d.x;
        if (in && e + 1 < a.E) out[e + 1] = d.y;
        if (in && e + 2 < a.E) out[e + 2] = d.z;
        if (in && e + 3 < a.E) out[e + 3] = d.w;
      }
    }
    wave_order();
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
  const int tpb = kFWaves * 64 / L;
  const int64_t blocks = (T + tpb - 1) / tpb;
  return (int)(blocks <= kAlone ? 1 : blocks < kGroups ? blocks : kGroups);
}

}  // namespace

size_t mok_losses_part_bytes(int64_t T, int E) {
  const int groups = by_experts(E, [&](auto L, auto, auto) { return groups_of(T, decltype(L)::value); });
  return groups > 1 ? (size_t)groups * (2 * E + 2) * 4 : 0;
}

hipError_t mok_launch_losses(const mok_losses_args& a, hipStream_t st) {
  const int groups = by_experts(a.E, [&](auto L, auto I, auto vec) {
    const int g = groups_of(a.T, decltype(L)::value);
    hipLaunchKernelGGL((losses_rows_kernel<decltype(L)::value, decltype(I)::value, decltype(vec)::value>),
                       dim3((unsigned)g), dim3(kFT), 0, st, a);
    return g;
  });
  if (groups > 1) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.E <= 128) {
      const auto join = a.E <= 32   ? losses_join_finish_kernel<32>
                        : a.E <= 64 ? losses_join_finish_kernel<64>
                                    : losses_join_finish_kernel<128>;
      hipLaunchKernelGGL(join, dim3(1), dim3(1024), 0, st, a, groups);
      return hipGetLastError();
    }
    hipLaunchKernelGGL(losses_join_kernel, dim3((unsigned)((a.E + 31) / 32)), dim3(kJT), 0, st, a, groups);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(losses_finish_kernel, dim3(1), dim3(512), 0, st, a, groups);
  }
  return hipGetLastError();
}

hipError_t mok_launch_losses_backward(const mok_losses_args& a, hipStream_t st) {
  if (a.T <= 0) return hipSuccess;
  by_experts(a.E, [&](auto L, auto I, auto vec) {
    const int tpb = kWaves * 64 / decltype(L)::value;
    // Two passes a workgroup, once 512 have work: both losses' calls at 16384 x 128 19.6 us, with one pass 21.0, with
    // four 20.5; up to 2048 workgroups, what the card holds.
    const int64_t blocks = (a.T + tpb - 1) / tpb;
    const int64_t groups = std::min<int64_t>(blocks, std::clamp<int64_t>(blocks / 2, 512, 2048));
    hipLaunchKernelGGL((losses_bwd_kernel<decltype(L)::value, decltype(I)::value, decltype(vec)::value>),
                       dim3((unsigned)groups), dim3(kBT), 0, st, a);
    return 0;
  });
  return hipGetLastError();
}
