// Tile machinery of the dense products (k_ffn.hip, k_mx.hip): operand copies
// for matrices that no schedule gathers, with tails in K, a 128 x 128 tile and
// row epilogues. The 256 x 256 bf16 tile runs the main loop of gemm_core.h on
// the copies defined here.
//
// LDS slots hold 64 bf16 (128 MX elements) of K per row. The layouts are those
// of gemm_core.h: 128-byte rows [rows][128 B] for K-contiguous operands,
// [64 k][2R B] for K-outer ones, and for 4-bit operands, whose rows have 64
// bytes per slot, two rows to a 128-byte line (below).
#pragma once
#include "gemm_core.h"

namespace mok {

// ------------------------------------------------------------------ layouts
// 64-byte rows: row r lies in line swap02(r / 2), half r % 2, its 16-byte chunk
// c at c ^ ((r / 2) & 3). Eight lanes reading chunk c of rows 8m .. 8m+7 then hit
// eight different 16-byte slots of a line, and address bit 7 (the line's bit 0)
// equals lane bit 3: the conflict-free pattern of gemm_core.h.
MOK_DEV int swap02(int v) { return (v & ~0x5) | ((v >> 2) & 1) | ((v & 1) << 2); }
MOK_DEV int lds_at64(int row, int chunk) {
  return swap02(row >> 1) * 128 + ((row & 1) << 6) + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// ------------------------------------------------------------------ copies
// K-contiguous operand of R rows, RB bytes of K per row and slot. Rows past the
// end repeat the last row (their products land in rows that are not stored);
// bytes past kbytes read as zero, on both operands, so that nothing stored
// behind a row (or behind the matrix) enters a product.
template <int R, int RB>
struct CopyK {
  static_assert(RB == 64 || RB == 128, "bytes of K per row and slot");
  static constexpr int kDma = R * RB / 4096;     // 1 KiB windows per wavefront
  static constexpr int kReads = 1;
  const uint8_t* rowp[kDma];                     // this lane's 16 bytes of slot 0, per copy
  int lcb, kbytes;
  mutable uint32_t mb;
  mutable bool tail;
  template <class Rows>
  MOK_DEV CopyK(const Rows& src, int64_t kbytes_) : kbytes((int)kbytes_) {
    const int w = (int)(threadIdx.x >> 6), l = lane_id();
    // the window's rows differ between copies q by multiples of 32 (64-byte
    // rows: 64) only, which leaves the chunk of a lane the same in all of them
    int row0, lc;
    if constexpr (RB == 128) {
      row0 = swap03(8 * w + (l >> 3));
      lc = (l & 7) ^ (row0 & 7);
    } else {
      row0 = 2 * swap02(8 * w + (l >> 3)) + ((l >> 2) & 1);
      lc = (l & 3) ^ ((row0 >> 1) & 3);
    }
    lcb = lc * 16;
#pragma unroll
    for (int q = 0; q < kDma; ++q) rowp[q] = src.row(row0 + q * (RB == 128 ? 32 : 64)) + lcb;
  }
  MOK_DEV void dma1(int j, uint32_t slot, int q) const {
    if (q == 0) {
      mb = slot + wave_id() * 1024;
      tail = (j + 1) * RB > kbytes;
    }
    const uint8_t* gp = rowp[q] + (int64_t)j * RB;
    if (tail) {                                  // wave-uniform branch
      asm volatile("");
      if (j * RB + lcb >= kbytes) gp = kZeroRow;
    }
    copy16_to_lds(gp, mb + q * 4096);
  }
  MOK_DEV void dma(int j, uint32_t slot) const {
#pragma unroll
    for (int q = 0; q < kDma; ++q) dma1(j, slot, q);
  }
  // bf16 fragment of 32 rows from r0: 16-wide K step kk of stage half h
  MOK_DEV static bf16x8_t frag(const uint8_t* t, int r0, int h, int kk) {
    const int l = lane_id();
    return *reinterpret_cast<const bf16x8_t*>(t + lds_at(r0 + (l & 31), 4 * h + 2 * kk + (l >> 5)));
  }
};

// K-outer bf16 operand of R columns: element (k, n) at src0 + k*ld + 2n for the
// first segment of kseg k-rows (a multiple of 64) and at src1 + (k - kseg)*ld +
// 2n for the second; k-rows past kvalid in either segment read as zero, columns
// past ncols repeat the last ones.
template <int R>
struct CopyT {
  static constexpr int kDma = R / 32;
  static constexpr int kReads = 2;
  static constexpr int kCh = R / 8;              // 16-byte chunks per k-row
  static constexpr int kRows = 64 / kCh;         // k-rows per 1 KiB window
  const uint8_t* src0;
  const uint8_t* src1;
  int kseg, kvalid;
  int64_t ld;
  int64_t off[kDma];
  int zoff;                                      // this lane's chunk of the zero row
  mutable const uint8_t* pb;
  mutable uint32_t mb;
  mutable int kr;
  MOK_DEV CopyT(const uint8_t* s0, const uint8_t* s1, int kseg_, int kvalid_, int64_t ld_, int ncols)
      : src0(s0), src1(s1), kseg(kseg_), kvalid(kvalid_), ld(ld_) {
    const int w = (int)(threadIdx.x >> 6), l = lane_id();
#pragma unroll
    for (int q = 0; q < kDma; ++q) {
      const int kl = kRows * (w + 4 * q) + l / kCh;
      const int c = min((l % kCh) ^ ((kl & 3) << 2), (ncols >> 3) - 1);
      off[q] = (int64_t)kl * ld + c * 16;
    }
    zoff = (l & 31) * 16;
  }
  MOK_DEV void dma1(int j, uint32_t slot, int q) const {
    if (q == 0) {
      const bool second = j * 64 >= kseg;
      const int k0 = second ? j * 64 - kseg : j * 64;
      pb = (second ? src1 : src0) + (int64_t)k0 * ld;
      mb = slot + wave_id() * 1024;
      kr = kvalid - k0;
    }
    const uint8_t* gp = pb + off[q];
    if (kr < 64) {
      asm volatile("");
      const int kl = kRows * ((int)(threadIdx.x >> 6) + 4 * q) + lane_id() / kCh;
      if (kl >= kr) gp = kZeroRow + zoff;
    }
    copy16_to_lds(gp, mb + q * 4096);
  }
  MOK_DEV void dma(int j, uint32_t slot) const {
#pragma unroll
    for (int q = 0; q < kDma; ++q) dma1(j, slot, q);
  }
  MOK_DEV static bf16x8_t frag(const uint8_t* t, int r0, int h, int kk) {
    const int l = lane_id(), g = l >> 4, L = l & 15;
    const int n = r0 + 16 * (g & 1) + 4 * (L & 3);
    const int k = 32 * h + 16 * kk + 8 * (g >> 1) + (L >> 2);
    typedef __attribute__((address_space(3))) v4i16_t* lds_v4_ptr;
    const auto at = [&](int kk_) {
      return (lds_v4_ptr)(t + kk_ * (2 * R) + (((n >> 3) ^ ((kk_ & 3) << 2)) << 4) + ((2 * n) & 15));
    };
    const v4i16_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k));
    const v4i16_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k + 4));
    typedef __attribute__((ext_vector_type(8))) short v8i16_t;
    const v8i16_t v = v8i16_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  }
};

// ------------------------------------------------------------------ 128 x 128 tile
// Four wavefronts of 64 x 64 (2 x 2 fragments of 32 x 32). Two slots of 32 KiB
// leave room for two workgroups on a CU, each multiplying while the other waits.
using G128 = Geo<128, 128, 2, 2>;
constexpr int kPitch128 = 128 * 4 + 16;          // fp32 staging of the tile
constexpr int kLds128 = 128 * kPitch128;         // 67584 B, above the two slots' 65536 B

// bf16 product over slots [j0, j1)
template <class LA, class LB>
MOK_DEV void loop128(uint8_t* lds, const LA& la, const LB& lb, int j0, int j1, Acc<2, 2>& acc) {
  constexpr int kSlot = 32768, kB = 16384, kD = LA::kDma + LB::kDma;
  const uint32_t base = lds_addr(lds);
  acc.zero();
  const auto issue = [&](int j, int s) {
    la.dma(j, base + s * kSlot);
    lb.dma(j, base + s * kSlot + kB);
  };
  if (j0 < j1) issue(j0, 0);
  if (j0 + 1 < j1) issue(j0 + 1, 1);
  for (int j = j0; j < j1; ++j) {
    const int s = (j - j0) & 1;
    if (j + 1 < j1) wait_vm_lds<kD>();
    else wait_vm_lds<0>();
    barrier_lds();
    const uint8_t* ta = lds + s * kSlot;
    const uint8_t* tb = ta + kB;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = LA::frag(ta, G128::wm() * 64 + 32 * i, ks >> 1, ks & 1);
        b[i] = LB::frag(tb, G128::wn() * 64 + 32 * i, ks >> 1, ks & 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          acc.c[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[n], acc.c[i][n], 0, 0, 0);
    }
    barrier_lds_only();
    if (j + 2 < j1) issue(j + 2, s);
  }
}

// stage the fp32 tile in LDS (the slots are free: every loop ends in a barrier)
MOK_DEV void stage128(uint8_t* lds, const Acc<2, 2>& acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        *reinterpret_cast<float*>(lds + G128::row(i, q) * kPitch128 + G128::col(n) * 4) = acc.c[i][n][q];
  barrier_lds_only();
}

// W consecutive fp32 values (W a multiple of 4) at p
template <int W>
MOK_DEV void load_f32(const void* p, float v[W]) {
#pragma unroll
  for (int u = 0; u < W / 4; ++u) {
    const float4 x = reinterpret_cast<const float4*>(p)[u];
    v[4 * u] = x.x; v[4 * u + 1] = x.y; v[4 * u + 2] = x.z; v[4 * u + 3] = x.w;
  }
}

// ------------------------------------------------------------------ few rows
// Products with at most kFewRows rows of x read the weights once and are bound by
// that. A workgroup of eight wavefronts takes 16 weight rows (one 16 x 16
// fragment; for gate|up 8 gate and 8 up rows, so that the gate's product stays in
// the workgroup) and every wavefront a contiguous eighth of K, straight from
// global memory into registers in the layout of the matrix instructions, two
// batches of K in flight and no barrier until the eight partial sums meet in
// LDS, in wavefront order. Sixteen rows per workgroup make enough workgroups to
// draw on every CU's share of the bandwidth (an expert of 2048 x 7168: 256).
constexpr int kFewRows = 64;
constexpr int kFewThreads = 512, kFewWaves = 8;
typedef __attribute__((ext_vector_type(4))) float f4_t;

// acc[nt][q] of lane l: weight row 4 * (l / 16) + q, token 16 nt + l % 16
template <int NT>
MOK_DEV void few_put(float* red, const f4_t acc[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<f4_t*>(red + ((wave_id() * NT + n) * 64 + lane_id()) * 4) = acc[n];
  __syncthreads();
}
// the sum over the wavefronts of weight row `row`, token `t`
template <int NT>
MOK_DEV float few_get(const float* red, int row, int t) {
  const float* p = red + ((t >> 4) * 64 + (row >> 2) * 16 + (t & 15)) * 4 + (row & 3);
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) s += p[w * NT * 256];
  return s;
}
// batches [b, e) of this wavefront in units of K: run load(buffer, k), compute(buffer, k)
// with the next batch's loads issued before the current one is used
template <int U, class Load, class Compute>
MOK_DEV void few_pipeline(int b, int e, Load&& load, Compute&& compute) {
  if (b >= e) return;
  load(0, b);
  for (int j = b; j < e; j += 2 * U) {
    if (j + U < e) load(1, j + U);
    compute(0, j);
    if (j + 2 * U < e) load(0, j + 2 * U);
    if (j + U < e) compute(1, j + U);
  }
}

// ------------------------------------------------------------------ tile order
// The nr x nc tiles of a product are numbered in groups of `grp` row tiles,
// column by column within a group, and XCD k (workgroups wg with wg mod 8 = k)
// takes the k-th eighth of them: the tiles in flight on one XCD form a block
// that shares its operand panels in that XCD's L2, and every XCD has work
// however few row tiles there are. Grid: 8 * ceil(n / 8) workgroups for n tiles; -1 past the end.
MOK_DEV int dense_index(int64_t n) {
  const int per = (int)((n + kXcds - 1) / kXcds), k = (int)blockIdx.x / kXcds;
  const int i = ((int)blockIdx.x % kXcds) * per + k;
  return k < per && i < n ? i : -1;
}
MOK_DEV void dense_tile(int i, int nr, int nc, int grp, int& row, int& col) {
  const int gi = i / (grp * nc), hg = min(grp, nr - grp * gi), j = i - gi * grp * nc;
  col = j / hg;
  row = grp * gi + j % hg;
}
inline unsigned dense_grid(int64_t n) { return (unsigned)((n + kXcds - 1) / kXcds * kXcds); }

// ------------------------------------------------------------------ gates
// act(a) and its derivative; KIND 0: SiLU a*s(a), 1: GELU in its tanh form,
// a/2 (1 + tanh u) = a*s(2u), u = sqrt(2/pi)(a + 0.044715 a^3), with the logistic s.
template <int KIND>
MOK_DEV float gate_act(float a) {
  if constexpr (KIND == 0) return a * sigmoidf_(a);
  return a * sigmoidf_(1.5957691216057308f * (a + 0.044715f * a * a * a));
}
template <int KIND>
MOK_DEV void gate_act_grad(float a, float& act, float& dact) {
  if constexpr (KIND == 0) {
    const float s = sigmoidf_(a);
    act = a * s;
    dact = s * (1.0f + a * (1.0f - s));
  } else {
    const float s = sigmoidf_(1.5957691216057308f * (a + 0.044715f * a * a * a));
    act = a * s;
    dact = s + act * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * a * a);
  }
}

}  // namespace mok
