// Root-mean-square norm of the residual stream, forward and backward, and the
// reading back of MXFP8 rows.
//
// Forward: z = bf16(x + residual), rstd = (mean z^2 + eps)^-1/2, y = z rstd w.
// Backward, with xh = z rstd, g = dy w: dx = rstd (g - xh mean(g xh)) + d_sum,
// dw = sum over the rows of dy xh. Both are bound by memory: every operand is
// read once and every output written once.
//
// A row lies in the registers of TPR threads, CH chunks of 8 columns each
// (thread l holds the chunks l, l + TPR, ...), from its load to its store, so
// it is read from memory once although the norm needs all of it before the
// first result. TPR and CH follow from H alone: the order of a row's sum does
// too. Many threads with one chunk each are fastest for many rows (backward of
// 16384 x 7168: 166 us with 1024 threads a row, 174 with 512, 189 with 256, 266
// with 128) and for a single one (forward with MXFP8 rows: 6.1, 6.4, 7.6 us).
// Stores carry the nontemporal hint (forward of 16384 x 7168: 156 us with it,
// 164 without).
//
// Whole calls of 16384 x 7168 with a residual: forward 154 us, 6.1 TB/s; backward 164 us,
// 5.7 TB/s with the partial sums of d_weight.
#include <type_traits>

#include "dense_core.h"
#include "lane_reduce.h"
#include "norm_launch.h"
#include "rows_core.h"

using namespace mok;

namespace {

template <int TPR>
struct RowShape {
  static constexpr int BT = TPR < 256 ? 256 : TPR;   // threads of a workgroup
  static constexpr int RPB = BT / TPR;               // rows of a workgroup at a time
  static constexpr int NW = TPR / 64;                // wavefronts of a row (0: a part of one)
};

// The sum of v over the TPR threads of a row, in every one of them: pairwise
// within a wavefront, then the wavefronts' sums in ascending order. `turn`
// alternates between calls, so that one barrier a call is enough: a wavefront
// that writes a half again has passed the barrier of the call between, which
// every other one reached after its reads.
template <int TPR, class V>
MOK_DEV V row_sum(V v, V (*red)[RowShape<TPR>::BT / 64], int turn) {
  v = lanes_sum<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    constexpr int NW = RowShape<TPR>::NW;
    const int wave = (int)threadIdx.x >> 6;
    if (lane_id() == 0) red[turn][wave] = v;
    __syncthreads();
    const V* r = red[turn] + wave / NW * NW;
    v = r[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v += r[i];
  }
  return v;
}

// eight weights from column 8c on
MOK_DEV void load_weight(const void* w, int wf, int c, float v[8]) {
  if (wf == 1) {
    unpack8(reinterpret_cast<const uint4*>(w)[c], v);
  } else if (wf == 2) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * c], b = reinterpret_cast<const float4*>(w)[2 * c + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 1.0f;
  }
}

template <int TPR, int CH>
__global__ __launch_bounds__(RowShape<TPR>::BT) void norm_fwd_kernel(const mok_norm_args a) {
  using S = RowShape<TPR>;
  __shared__ double red[2][S::BT / 64];
  const int sub = (int)threadIdx.x / TPR, l = (int)threadIdx.x % TPR;
  const int n8 = a.H / 8;
  float w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int u = 0; u < 8; ++u) w[i][u] = 0.f;
    if (l + i * TPR < n8) load_weight(a.w, a.wf, l + i * TPR, w[i]);
  }
  const double inv_h = 1.0 / a.H;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * S::RPB; r0 < a.T; r0 += (int64_t)gridDim.x * S::RPB) {
    const int64_t row = r0 + sub;
    const bool live = row < a.T;
    double ss = 0.0;                             // in 64 bits, at the rate of 32
    uint4 xv[CH], rv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = l + i * TPR;
      xv[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && c < n8) {
        xv[i] = reinterpret_cast<const uint4*>(a.x + row * a.ldx)[c];
        if (a.res) rv[i] = reinterpret_cast<const uint4*>(a.res + row * a.lds)[c];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = l + i * TPR;
      if (a.res) {
        float p[8], q[8];
        unpack8(xv[i], p);
        unpack8(rv[i], q);
#pragma unroll
        for (int u = 0; u < 8; ++u) p[u] += q[u];
        xv[i] = pack8(p);                        // the stream is kept, and normed, in bf16
        if (live && c < n8) store_nt(reinterpret_cast<uint4*>(a.sum + row * a.lds) + c, xv[i]);
      }
      float z[8];
      unpack8(xv[i], z);
#pragma unroll
      for (int u = 0; u < 8; ++u) ss = fma((double)z[u], (double)z[u], ss);
      // (kept packed, and unpacked once more below: with the values held over the sum a CU holds one row of 1024
      // threads in place of two, 202 us at 16384 x 7168 for 161)
      asm volatile("" : "+v"(xv[i].x), "+v"(xv[i].y), "+v"(xv[i].z), "+v"(xv[i].w));
    }
    ss = row_sum<TPR>(ss, red, turn);
    turn ^= 1;
    // a Newton step in 64 bits from the fp32 value (0 where the sum passes fp32's range)
    const double var = fma(ss, inv_h, (double)a.eps);
    double rstd64 = 1.0f / sqrtf((float)var);
    if (rstd64 > 0.0) rstd64 += 0.5 * rstd64 * (1.0 - var * rstd64 * rstd64);
    const float rstd = (float)rstd64;
    if (live && l == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = l + i * TPR;
      const bool ok = live && c < n8;
      float z[8], y[8];
      unpack8(xv[i], z);
      if (a.y) {
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = z[u] * rstd * w[i][u];
        if (ok) store_nt(reinterpret_cast<uint4*>(a.y + row * a.ldy) + c, pack8(y));
      }
      if (a.q) {
        // (a value within its error of the middle between two codes may take either: sum, rstd and products in 64 bits
        // leave that to the one rounding of y to fp32)
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = (float)((double)z[u] * rstd64 * (double)w[i][u]);
        // four neighbouring threads hold a block (H is a multiple of 32: all four or none are in the row)
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(y[u]) & 0x7FFFFFFFu);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const bool nan = m >= 0x7F800000u;
        const int sc = nan ? 255 : mx_scale_byte(__uint_as_float(m));
        const float inv = mx_inv_scale(sc);
        const uint32_t lo = e4m3_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        const uint32_t hi = e4m3_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
        if (ok) {
          reinterpret_cast<uint2*>(a.q + row * a.H)[c] = nan ? make_uint2(0u, 0u) : make_uint2(lo, hi);
          if ((l & 3) == 0) a.scales[row * (a.H / 32) + c / 4] = (uint8_t)sc;
        }
      }
    }
  }
}

// Rows as in the forward; each thread also adds up dy xh of its columns over the
// workgroup's rows, and the workgroups' sums, one row of `part` each, are added
// in ascending order by norm_dw_kernel (one workgroup alone writes d_weight).
template <int TPR, int CH>
__global__ __launch_bounds__(RowShape<TPR>::BT) void norm_bwd_kernel(const mok_norm_args a) {
  using S = RowShape<TPR>;
  __shared__ float red[2][S::BT / 64];
  // Up to 16384 columns the weights and their gradient's sums stay in registers. Beyond, there are not enough: the sums
  // lie in LDS, one place a thread and column, and the weights are read again for each row.
  constexpr bool KEEP = CH <= 2;
  constexpr int DWS = !KEEP ? TPR * CH * 8 : S::RPB > 1 ? S::BT * CH * 8 : 1;
  __shared__ float dws[DWS];
  const int sub = (int)threadIdx.x / TPR, l = (int)threadIdx.x % TPR;
  const int n8 = a.H / 8;
  float wk[KEEP ? CH : 1][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if constexpr (KEEP) dw[i][u] = wk[i][u] = 0.f;
      else dws[(8 * i + u) * TPR + l] = 0.f;
    }
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (l + i * TPR < n8) load_weight(a.w, a.wf, l + i * TPR, wk[i]);
  }
  const auto weight = [&](int i, float v[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = KEEP ? wk[KEEP ? i : 0][u] : 0.f;
    if (!KEEP && l + i * TPR < n8) load_weight(a.w, a.wf, l + i * TPR, v);
  };
  const float inv_h = 1.0f / (float)a.H;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * S::RPB; r0 < a.T; r0 += (int64_t)gridDim.x * S::RPB) {
    const int64_t row = r0 + sub;
    const bool live = row < a.T;
    uint4 zv[CH], dv[CH], sv[CH];
    const float rstd = live ? a.rstd[row] : 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = l + i * TPR;
      zv[i] = dv[i] = sv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && c < n8) {
        zv[i] = reinterpret_cast<const uint4*>(a.x + row * a.ldx)[c];
        dv[i] = reinterpret_cast<const uint4*>(a.dy + row * a.ldy)[c];
        if (a.res) sv[i] = reinterpret_cast<const uint4*>(a.res + row * a.lds)[c];
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float z[8], d[8], w[8];
      unpack8(zv[i], z);
      unpack8(dv[i], d);
      weight(i, w);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float xh = z[u] * rstd;
        s = fmaf(d[u] * w[u], xh, s);
        if constexpr (KEEP) dw[i][u] = fmaf(d[u], xh, dw[i][u]);
        else dws[(8 * i + u) * TPR + l] = fmaf(d[u], xh, dws[(8 * i + u) * TPR + l]);
      }
    }
    s = row_sum<TPR>(s, red, turn) * inv_h;
    turn ^= 1;
    // (kept as loaded: unpacked once more below, not held in twice the registers over the sum)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      asm volatile("" : "+v"(zv[i].x), "+v"(zv[i].y), "+v"(zv[i].z), "+v"(zv[i].w));
      asm volatile("" : "+v"(dv[i].x), "+v"(dv[i].y), "+v"(dv[i].z), "+v"(dv[i].w));
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = l + i * TPR;
      float z[8], d[8], o[8], w[8];
      unpack8(zv[i], z);
      unpack8(dv[i], d);
      unpack8(sv[i], o);
      weight(i, w);
#pragma unroll
      for (int u = 0; u < 8; ++u) o[u] = fmaf(rstd, fmaf(-z[u] * rstd, s, d[u] * w[u]), o[u]);
      if (live && c < n8) store_nt(reinterpret_cast<uint4*>(a.sum + row * a.lds) + c, pack8(o));
    }
  }
  if (!a.dw) return;
  if constexpr (!KEEP) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) dw[i][u] = dws[(8 * i + u) * TPR + l];
  } else if constexpr (S::RPB > 1) {
    // the rows' threads of one column, in ascending order
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) dws[(8 * i + u) * S::BT + threadIdx.x] = dw[i][u];
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u)
        for (int r = 1; r < S::RPB; ++r) dw[i][u] += dws[(8 * i + u) * S::BT + r * TPR + l];
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = l + i * TPR;
    if (c >= n8) continue;
    if (gridDim.x == 1 && a.wf == 1) {
      reinterpret_cast<uint4*>(a.dw)[c] = pack8(dw[i]);
    } else {
      float4* d = reinterpret_cast<float4*>(gridDim.x == 1 ? (float*)a.dw : a.part + (int64_t)blockIdx.x * a.H) + 2 * c;
      d[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      d[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// d_weight[h] = the sum of the n partial rows: 32 columns a workgroup, 32 rows of
// threads that add every 32nd partial row each, then theirs in ascending order
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ part, int n, int H, int wf,
                                                      void* __restrict__ dw) {
  __shared__ float g[32][32];
  const int c = (int)threadIdx.x & 31, r = (int)threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int i = r; i < n; i += 32) s += part[(int64_t)i * H + col];
  }
  g[r][c] = s;
  __syncthreads();
  if (r != 0 || col >= H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += g[i][c];
  if (wf == 1) static_cast<bf16_t*>(dw)[col] = f32_to_bf16(s);
  else static_cast<float*>(dw)[col] = s;
}

// Sixteen codes a thread: E4M3 to fp32 is exact, and so is the product with
// 2^(s-127) by ldexp (the smallest, 2^-9 * 2^-127, is an fp32 subnormal), so the
// one rounding is that to bf16. Bound by memory.
__global__ __launch_bounds__(256) void mxfp8_dequantize_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ scales, int64_t n16,
                                                               bf16_t* __restrict__ dst) {
  const int64_t idx = flat_block() * 256 + threadIdx.x;
  if (idx >= n16) return;
  const uint4 v = reinterpret_cast<const uint4*>(q)[idx];
  const int s = scales[idx >> 1];
  const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)wd[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)wd[i], true);
    f[4 * i] = lo[0]; f[4 * i + 1] = lo[1]; f[4 * i + 2] = hi[0]; f[4 * i + 3] = hi[1];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = s == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(f[i], s - 127);
  uint4* d = reinterpret_cast<uint4*>(dst) + 2 * idx;
  d[0] = pack8(f);
  d[1] = pack8(f + 8);
}

// f(RowShape's TPR, CH) as constants, for rows of H columns
template <class F>
auto by_width(int H, F&& f) {
  using std::integral_constant;
#define MOK_ROW(tpr, ch) \
  if (H <= 8 * (tpr) * (ch)) return f(integral_constant<int, tpr>{}, integral_constant<int, ch>{})
  MOK_ROW(8, 1);
  MOK_ROW(16, 1);
  MOK_ROW(32, 1);
  MOK_ROW(64, 1);
  MOK_ROW(128, 1);
  MOK_ROW(256, 1);
  MOK_ROW(512, 1);
  MOK_ROW(1024, 1);
  MOK_ROW(1024, 2);
#undef MOK_ROW
  return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

}  // namespace

hipError_t mok_launch_norm_forward(const mok_norm_args& a, hipStream_t st) {
  if (a.T <= 0) return hipSuccess;
  by_width(a.H, [&](auto tpr, auto ch) {
    using S = RowShape<decltype(tpr)::value>;
    // A workgroup for each RPB rows: 157 us at 16384 x 7168, against 170 with workgroups that go round and keep the
    // weights. (A launch holds 2^32 threads; more rows go round.)
    const int64_t blocks = (a.T + S::RPB - 1) / S::RPB, cap = (int64_t)1 << 21;
    hipLaunchKernelGGL((norm_fwd_kernel<decltype(tpr)::value, decltype(ch)::value>),
                       dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(S::BT), 0, st, a);
  });
  return hipGetLastError();
}

// 1024 threads a CU, as one workgroup or several: 16384 x 7168 166 us, with half as many 255, with twice as many 173;
// 1000 x 32768 95, 113, 112; 4096 x 4096 31.3, 32.4, 35.3; 24871 x 128 11.0, 10.7, 11.9. (More workgroups make more
// partial rows, fewer leave loads unissued.)
int mok_norm_groups(int64_t T, int H) {
  return by_width(H, [&](auto tpr, auto) {
    using S = RowShape<decltype(tpr)::value>;
    const int64_t blocks = (T + S::RPB - 1) / S::RPB, cap = 256 * 1024 / S::BT;
    return (int)(blocks < cap ? (blocks < 1 ? 1 : blocks) : cap);
  });
}

hipError_t mok_launch_norm_backward(const mok_norm_args& a, hipStream_t st) {
  const int groups = mok_norm_groups(a.T, a.H);
  by_width(a.H, [&](auto tpr, auto ch) {
    using S = RowShape<decltype(tpr)::value>;
    hipLaunchKernelGGL((norm_bwd_kernel<decltype(tpr)::value, decltype(ch)::value>), dim3((unsigned)groups),
                       dim3(S::BT), 0, st, a);
  });
  if (groups > 1 && a.dw) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(1024), 0, st, a.part, groups, a.H, a.wf,
                       a.dw);
  }
  return hipGetLastError();
}

hipError_t mok_launch_mxfp8_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K, bf16_t* dst,
                                       hipStream_t st) {
  const int64_t n16 = rows * (K / 16);
  if (n16 <= 0) return hipSuccess;
  hipLaunchKernelGGL(mxfp8_dequantize_kernel, flat_grid((n16 + 255) / 256), dim3(256), 0, st, q, scales, n16, dst);
  return hipGetLastError();
}
