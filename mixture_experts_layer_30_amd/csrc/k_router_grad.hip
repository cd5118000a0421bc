// Router backward from the gradient of every logit: dx = dl . Wr (+ residual)
// and dWr = dl^T . x, on the matrix cores (v_mfma_f32_32x32x16_bf16). dl and Wr
// are fp32, the operands bf16: for dWr, which is fp32, dl is split exactly into
// three bf16 parts (x is bf16, so every product is exact); for dx, which is
// rounded to bf16, dl and Wr go in as two parts each, the nearest bf16 and the
// nearest to what that leaves (at most 2^-16 of a value is lost), and the
// product of the two small parts, at most 2^-16 of the whole, is left out.
//
// A lane l of the instruction supplies row l % 32 of an operand, 8 values of K
// from 8 (l / 32) on, and holds of the result column l % 32 the rows
// 8 (i / 4) + 4 (l / 32) + i % 4, i = 0 .. 15.
#include <type_traits>

#include "mok_device.h"
#include "router_launch.h"

namespace {

typedef __attribute__((ext_vector_type(4))) short i16x4_t;
typedef __attribute__((ext_vector_type(8))) short i16x8_t;
typedef __attribute__((address_space(3))) i16x4_t* lds_i16x4_ptr;

MOK_DEV float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
MOK_DEV float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// the nearest bf16 of a pair, and the nearest to what it leaves
MOK_DEV void split2(float a, float b, uint32_t& hi, uint32_t& mid) {
  hi = pack_bf16x2(a, b);
  mid = pack_bf16x2(a - bf_lo(hi), b - bf_hi(hi));
}
// and a third part: hi + mid + lo is exact (8 + 8 + 8 bits)
MOK_DEV void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  const float ra = a - bf_lo(hi), rb = b - bf_hi(hi);
  mid = pack_bf16x2(ra, rb);
  lo = pack_bf16x2(ra - bf_lo(mid), rb - bf_hi(mid));
}

MOK_DEV f32x16_t mfma(const uint4& a, const uint4& b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

// four values of row t of dl from expert e on; zeros past the ends
MOK_DEV float4 load_dl(const mok_logits_bwd_args& a, int64_t t, int64_t t1, int e, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* p = a.dl + t * a.E + e;
  if (t >= t1) return v;
  if (vec) {
    if (e < a.E) v = *reinterpret_cast<const float4*>(p);
  } else {
    if (e < a.E) v.x = p[0];
    if (e + 1 < a.E) v.y = p[1];
    if (e + 2 < a.E) v.z = p[2];
    if (e + 3 < a.E) v.w = p[3];
  }
  return v;
}

// ---------------------------------------------------------------- dx
// The columns of dx are rows of the first operand, tokens columns of the second,
// so a lane ends up with 16 neighbouring columns of one token. A wavefront keeps
// its 32 columns of Wr, both parts, in registers (8 KS of them, KS = E / 16) and
// the tokens stream past: 32 at a time are split into LDS by the whole workgroup,
// the next 32 on their way in registers meanwhile.
template <int KS, int NW>
__global__ __launch_bounds__(64 * NW) void router_dx_kernel(const mok_logits_bwd_args a, int panels, int slices) {
  constexpr int EP = 16 * KS, PITCH = EP + 8, BT = 64 * NW, NL = (32 * EP / 4 + BT - 1) / BT;
  __shared__ __attribute__((aligned(16))) bf16_t tile[2][32 * PITCH];
  const int panel = (int)blockIdx.x % panels, slice = (int)blockIdx.x / panels;
  const int wave = (int)threadIdx.x >> 6, lane = lane_id(), r = lane & 31, half = lane >> 5;
  const int64_t blocks = (a.T + 31) / 32;
  const int64_t t0 = blocks * slice / slices * 32, te = blocks * (slice + 1) / slices * 32, t1 = te < a.T ? te : a.T;
  const int h0 = panel * 32 * NW + 32 * wave;
  const bool cols = h0 < a.H;                    // (H is a multiple of 32)
  const bool vec = a.E % 4 == 0;
  const int nks = (a.E + 15) / 16;
  // row r of the operand is column 16 ((r / 4) % 2) + 4 (r / 8) + r % 4, so that lane half b holds columns 16 b .. + 15
  const int col = h0 + 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);
  uint4 whi[KS], wmid[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = 16 * s + 8 * half + u;
      v[u] = cols && e < a.E ? a.wr[(int64_t)e * a.H + col] : 0.f;
    }
    split2(v[0], v[1], whi[s].x, wmid[s].x);
    split2(v[2], v[3], whi[s].y, wmid[s].y);
    split2(v[4], v[5], whi[s].z, wmid[s].z);
    split2(v[6], v[7], whi[s].w, wmid[s].w);
  }
  float4 next[NL];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = (int)threadIdx.x + BT * i;
      next[i] = q < 32 * EP / 4 ? load_dl(a, t + q / (EP / 4), t1, 4 * (q % (EP / 4)), vec)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(t0);
  for (int64_t t = t0; t < t1; t += 32) {
    __syncthreads();                             // the last tile's reads are done
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = (int)threadIdx.x + BT * i;
      if (q >= 32 * EP / 4) break;
      uint2 hi, mid;
      split2(next[i].x, next[i].y, hi.x, mid.x);
      split2(next[i].z, next[i].w, hi.y, mid.y);
      const int at = q / (EP / 4) * PITCH + 4 * (q % (EP / 4));
      *reinterpret_cast<uint2*>(tile[0] + at) = hi;
      *reinterpret_cast<uint2*>(tile[1] + at) = mid;
    }
    __syncthreads();
    load(t + 32);
    if (!cols) continue;
    const int64_t tok = t + r;
    bf16_t* out = a.dx + tok * a.H + h0 + 16 * half;
    uint4 rv[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (a.res && tok < t1) {
      const uint4* p = reinterpret_cast<const uint4*>(a.res + tok * a.H + h0 + 16 * half);
      rv[0] = p[0];
      rv[1] = p[1];
    }
    f32x16_t acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (s < nks) {
        const uint4 dhi = *reinterpret_cast<const uint4*>(tile[0] + r * PITCH + 16 * s + 8 * half);
        const uint4 dmid = *reinterpret_cast<const uint4*>(tile[1] + r * PITCH + 16 * s + 8 * half);
        acc = mfma(wmid[s], dhi, acc);
        acc = mfma(whi[s], dmid, acc);
        acc = mfma(whi[s], dhi, acc);
      }
    }
    if (tok < t1) {
      const uint32_t rw[8] = {rv[0].x, rv[0].y, rv[0].z, rv[0].w, rv[1].x, rv[1].y, rv[1].z, rv[1].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(acc[2 * i] + bf_lo(rw[i]), acc[2 * i + 1] + bf_hi(rw[i]));
      reinterpret_cast<uint4*>(out)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(out)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// ---------------------------------------------------------------- dWr
// A workgroup sums 32 MT experts x 128 columns over its slice of the tokens, 32
// at a time through LDS: x as it is, dl in its three parts, both read transposed
// (ds_read_b64_tr_b16: lane 4 q + p of 16 names row q and columns 4 p .. + 3, and
// gets column l of the four rows). The slices' sums, one [E][H] each, are added
// in ascending order by router_dwr_join_kernel.
constexpr int kNC = 128;
template <int MT>
__global__ __launch_bounds__(256) void router_dwr_slices_kernel(const mok_logits_bwd_args a, int panels, int eblocks,
                                                                int slices) {
  constexpr int EB = 32 * MT;
  constexpr int XP = 2 * kNC + 64, DP = 2 * EB + (EB > 32 ? 64 : 0);   // row pitches in bytes
  constexpr int WM = MT == 4 ? 2 : 1;            // wavefronts along the experts
  constexpr int TM = MT / WM, TN = MT == 4 ? 2 : 1;
  constexpr int NL = EB / 32;                    // float4s of dl a thread loads
  __shared__ __attribute__((aligned(16))) uint8_t xs[32 * XP];
  __shared__ __attribute__((aligned(16))) uint8_t ds[3][32 * DP];
  const int panel = (int)blockIdx.x % panels, eb = (int)blockIdx.x / panels % eblocks;
  const int slice = (int)blockIdx.x / (panels * eblocks);
  const int wave = (int)threadIdx.x >> 6, lane = lane_id();
  const int wm = wave % WM, wn = wave / WM;
  const int64_t blocks = (a.T + 31) / 32;
  const int64_t t0 = blocks * slice / slices * 32, te = blocks * (slice + 1) / slices * 32, t1 = te < a.T ? te : a.T;
  const int c0 = panel * kNC, e0 = eb * EB;
  const bool vec = a.E % 4 == 0;
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
  uint4 xn[2];
  float4 dn[NL];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = (int)threadIdx.x + 256 * i;
      const int64_t tok = t + q / 16;
      xn[i] = make_uint4(0u, 0u, 0u, 0u);
      if (tok < t1) xn[i] = *reinterpret_cast<const uint4*>(a.x + tok * a.H + c0 + 8 * (q % 16));
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = (int)threadIdx.x + 256 * i;
      dn[i] = load_dl(a, t + q / (EB / 4), t1, e0 + 4 * (q % (EB / 4)), vec);
    }
  };
  // this lane's place in a transposed read: row 8 (l / 32) + (l % 16) / 4, columns 16 ((l / 16) % 2) + 4 (l % 4)
  const int tr = 8 * (lane >> 5) + ((lane & 15) >> 2), tc = 2 * (16 * ((lane >> 4) & 1) + 4 * (lane & 3));
  auto frag = [&](const uint8_t* base, int pitch, int k, int c) {
    const uint8_t* p = base + (16 * k + tr) * pitch + 2 * c + tc;
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_ptr)(p));
    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_ptr)(p + 4 * pitch));
    return __builtin_bit_cast(uint4, i16x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
  };
  load(t0);
  for (int64_t t = t0; t < t1; t += 32) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = (int)threadIdx.x + 256 * i;
      *reinterpret_cast<uint4*>(xs + q / 16 * XP + 16 * (q % 16)) = xn[i];
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int q = (int)threadIdx.x + 256 * i;
      uint2 p[3];
      split3(dn[i].x, dn[i].y, p[0].x, p[1].x, p[2].x);
      split3(dn[i].z, dn[i].w, p[0].y, p[1].y, p[2].y);
#pragma unroll
      for (int s = 0; s < 3; ++s)
        *reinterpret_cast<uint2*>(ds[s] + q / (EB / 4) * DP + 8 * (q % (EB / 4))) = p[s];
    }
    __syncthreads();
    load(t + 32);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4 xf[TN];
#pragma unroll
      for (int n = 0; n < TN; ++n) xf[n] = frag(xs, XP, k, 32 * (wn * TN + n));
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int s = 2; s >= 0; --s) {
          const uint4 df = frag(ds[s], DP, k, 32 * (wm * TM + m));
#pragma unroll
          for (int n = 0; n < TN; ++n) acc[m][n] = mfma(df, xf[n], acc[m][n]);
        }
    }
  }
  float* out = slices > 1 ? a.part + (int64_t)slice * a.E * a.H : a.dwr;
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = e0 + 32 * (wm * TM + m) + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
        if (e < a.E) out[(int64_t)e * a.H + c0 + 32 * (wn * TN + n) + (lane & 31)] = acc[m][n][i];
      }
}

__global__ __launch_bounds__(256) void router_dwr_join_kernel(const float* __restrict__ part, int slices, int64_t n4,
                                                             float* __restrict__ dwr) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 s = reinterpret_cast<const float4*>(part)[i];
#pragma unroll 4
  for (int k = 1; k < slices; ++k) {
    const float4 v = reinterpret_cast<const float4*>(part)[k * n4 + i];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  reinterpret_cast<float4*>(dwr)[i] = s;
}

struct DwrPlan {
  int mt, panels, eblocks, slices;
};
DwrPlan dwr_plan(int64_t T, int H, int E) {
  DwrPlan p;
  p.mt = E <= 32 ? 1 : E <= 64 ? 2 : 4;
  p.panels = H / kNC;
  p.eblocks = (E + 32 * p.mt - 1) / (32 * p.mt);
  const int64_t blocks = (T + 31) / 32;
  int64_t s = 512 / ((int64_t)p.panels * p.eblocks);
  if (s > blocks / 2) s = blocks / 2;
  p.slices = (int)(s < 1 ? 1 : s);
  return p;
}

}  // namespace

size_t mok_logits_bwd_part_bytes(int64_t T, int H, int E) {
  const DwrPlan p = dwr_plan(T, H, E);
  return p.slices > 1 ? (size_t)p.slices * E * H * 4 : 0;
}

hipError_t mok_launch_logits_bwd_dx(const mok_logits_bwd_args& a, hipStream_t st) {
  if (a.T <= 0) return hipSuccess;
  const int64_t blocks = (a.T + 31) / 32;
  const auto launch = [&](auto ks, auto nw) {
    constexpr int KS = decltype(ks)::value, NW = decltype(nw)::value;
    const int panels = (a.H + 32 * NW - 1) / (32 * NW);
    int64_t s = (512 + panels - 1) / panels;
    if (s > blocks) s = blocks;
    hipLaunchKernelGGL((router_dx_kernel<KS, NW>), dim3((unsigned)(panels * s)), dim3(64 * NW), 0, st, a, panels, (int)s);
  };
  using std::integral_constant;
  if (a.E <= 16) launch(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  else if (a.E <= 32) launch(integral_constant<int, 2>{}, integral_constant<int, 8>{});
  else if (a.E <= 64) launch(integral_constant<int, 4>{}, integral_constant<int, 8>{});
  else if (a.E <= 128) launch(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  else if (a.E <= 256) launch(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else launch(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t mok_launch_logits_bwd_dwr(const mok_logits_bwd_args& a, hipStream_t st) {
  const DwrPlan p = dwr_plan(a.T, a.H, a.E);
  const dim3 grid((unsigned)(p.panels * p.eblocks * p.slices));
  if (p.mt == 1)
    hipLaunchKernelGGL(router_dwr_slices_kernel<1>, grid, dim3(256), 0, st, a, p.panels, p.eblocks, p.slices);
  else if (p.mt == 2)
    hipLaunchKernelGGL(router_dwr_slices_kernel<2>, grid, dim3(256), 0, st, a, p.panels, p.eblocks, p.slices);
  else
    hipLaunchKernelGGL(router_dwr_slices_kernel<4>, grid, dim3(256), 0, st, a, p.panels, p.eblocks, p.slices);
  if (p.slices > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n4 = (int64_t)a.E * a.H / 4;
    hipLaunchKernelGGL(router_dwr_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st, a.part, p.slices,
                       n4, a.dwr);
  }
  return hipGetLastError();
}
