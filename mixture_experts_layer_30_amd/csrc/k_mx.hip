// MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements, one E8M0 scale per 32
// along a row): quantization, reading back, and the product of an MXFP4 or
// MXFP8 matrix with an MXFP4 matrix on the scaled matrix instructions,
//
//   D[m][n] = sum over blocks of 32 k of 2^(sa + sb - 254) * sum_k A[m][k] B[n][k],
//
// blocks added in fp32. Within a block the instruction adds the 32 products before that: it
// aligns them to the largest and keeps 13 bits below that one's leading bit (measured: of
// 2^8 - 2^8 + x, x = 2^-5 stays and 2^-6 is lost). Products of two E2M1 values never reach
// below that and their sums are exact; with E4M3 each product loses less than 2^-13 of the
// block's largest, and D differs by 2 to 3 parts in 10^4 (in norm) from the rounded exact
// sums, which the rounding to bf16 leaves 17 in 10^4 off. That is the choice here: bf16
// operands, whose products fp32 holds, run at less than half the rate. With the gate it
// computes the first half of a feed-forward block with 4-bit weights: h = act(A Wg^T) *
// (A Wu^T), quantized along its row to MXFP8 from the fp32 values (no bf16 rounding between).
#include "dense_core.h"
#include "dense_launch.h"

using namespace mok;

namespace {

// ------------------------------------------------------------------ quantize
// E8M0 scale as a float: 2^(s - 127), NaN for 255
MOK_DEV float e8m0(int s) {
  return __uint_as_float(s == 255 ? 0x7FC00000u : s == 0 ? 0x00400000u : (uint32_t)s << 23);
}

// bits of the largest magnitude of a block held by four adjacent lanes, eight
// elements each (as integers, so that a NaN is the largest of all)
MOK_DEV uint32_t block_max_bits(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(v[u]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  return max(m, (uint32_t)__shfl_xor((int)m, 2));
}

// Four adjacent lanes per block, eight elements each: 16-byte loads along the row, the
// block's largest magnitude over the four lanes, 4 bytes of codes per lane. The scale
// byte is clamp(floor(log2 amax) - 2 + 127, 0, 254) (2: the exponent of the largest E2M1
// value, 6 = 1.5 * 2^2), which from the exponent field f of a bf16 amax is max(f - 2, 0),
// 0 for zeros and subnormals too. The codes are the hardware's (v_cvt_scalef32_pk_fp4_bf16:
// value / 2^(s-127) to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code,
// saturating, sign kept): equal to the definition on gfx950 for every bf16 value at every
// scale. A block that holds a NaN or an infinity, which the format cannot, gets the NaN
// scale 255: it reads back, and multiplies, as NaN.
// Bound by memory: 16384 x 7168 in 58 us (5.1 TB/s); seven comparisons per element in
// place of the conversion took 80 us.
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const bf16_t* __restrict__ src, int64_t n8,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  const int64_t idx = flat_block() * 256 + threadIdx.x;
  if (idx >= n8) return;                         // n8 is a multiple of 4: whole blocks leave
  const uint4 raw = reinterpret_cast<const uint4*>(src)[idx];
  const auto mag = [](uint32_t v) { return __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu); };
  const u16x2 m2 = __builtin_elementwise_max(__builtin_elementwise_max(mag(raw.x), mag(raw.y)),
                                             __builtin_elementwise_max(mag(raw.z), mag(raw.w)));
  int m = max((int)m2[0], (int)m2[1]);
  m = max(m, __shfl_xor(m, 1));
  m = max(m, __shfl_xor(m, 2));
  const bool nan = m >= 0x7F80;
  const int sc = nan ? 255 : max((m >> 7) - 2, 0);
  const float x = e8m0(nan ? 127 : sc);
  const auto pair = [](uint32_t v) { return __builtin_bit_cast(bf16x2_t, v); };
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, pair(raw.x), x, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(raw.y), x, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(raw.z), x, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(raw.w), x, 3);
  reinterpret_cast<uint32_t*>(q)[idx] = nan ? 0u : w;
  if ((idx & 3) == 0) scales[idx >> 2] = (uint8_t)sc;
}

// code * 2^(s-127), exact in bf16 (v_cvt_scalef32_pk_bf16_fp4); 16384 x 7168 right after
// quantizing in 48 to 55 us (part of the codes still in the last-level cache)
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ scales, int64_t n8,
                                                              bf16_t* __restrict__ dst) {
  const int64_t idx = flat_block() * 256 + threadIdx.x;
  if (idx >= n8) return;
  const uint32_t w = reinterpret_cast<const uint32_t*>(q)[idx];
  const float x = e8m0(scales[idx >> 2]);
  const auto bits = [](bf16x2_t v) { return __builtin_bit_cast(uint32_t, v); };
  reinterpret_cast<uint4*>(dst)[idx] = make_uint4(bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, x, 0)),
                                                  bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, x, 1)),
                                                  bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, x, 2)),
                                                  bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, x, 3)));
}

// MXFP8 rows (E4M3, the scale rule of the layer's quantizer) of a bf16 or fp32
// matrix of row pitch ld, for the activations of a block with 4-bit weights;
// blocks that are not finite get the scale 255, so that their tokens come out NaN.
template <class T>
__global__ __launch_bounds__(256) void mxfp8_rows_kernel(const T* __restrict__ src, int64_t ld, int64_t n8,
                                                        int k8, uint8_t* __restrict__ q,
                                                        uint8_t* __restrict__ scales) {
  const int64_t idx = flat_block() * 256 + threadIdx.x;
  if (idx >= n8) return;
  const int64_t r = idx / k8, c = idx - r * k8;
  float v[8];
  if constexpr (sizeof(T) == 2) unpack_bf16x8(reinterpret_cast<const uint4*>(src + r * ld)[c], v);
  else load_f32<8>(src + r * ld + 8 * c, v);
  const uint32_t m = block_max_bits(v);
  const bool nan = m >= 0x7F800000u;
  const int sc = nan ? 255 : mx_scale_byte(__uint_as_float(m));
  const float inv = mx_inv_scale(sc);
  const uint32_t lo = e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  const uint32_t hi = e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  reinterpret_cast<uint2*>(q)[idx] = nan ? make_uint2(0, 0) : make_uint2(lo, hi);
  if ((idx & 3) == 0) scales[idx >> 2] = (uint8_t)sc;
}

// ------------------------------------------------------------------ product, 128 x 128 tile
// A slot holds SK elements of K per row: 128 where A is E4M3 (128-byte rows of A,
// 64-byte rows of B), 256 where both are E2M1 (128-byte rows of both). A lane of
// v_mfma_scale_f32_32x32x64_f8f6f4 supplies row l % 32: of E2M1 the 32 elements
// from 32 * (l / 32) on (16 bytes), of E4M3 the 16 bytes from 16 * (l / 32) on and
// those 32 further; the scale of block l / 32 of its row (checked on gfx950).
template <bool A8>
struct MxTile {
  static constexpr int SK = A8 ? 128 : 256;
  static constexpr int RBA = 128, RBB = SK / 2;
  static constexpr int kA = 128 * RBA, kB = 128 * RBB, kS = SK / 128 * 1024;
  static constexpr int kSlot = kA + kB + kS;
};

// Scale words (four blocks of 32, one word per 128 of K) of 64 rows: lane l copies those
// of row l; words past K read as zero.
template <int WORDS>
struct CopyScales {
  static constexpr int kDma = WORDS;
  srd_t srd;
  int off, nb;                                   // nb: scale bytes per row
  MOK_DEV CopyScales(const uint8_t* p, int n, int K) : nb(K / 32) {
    srd = make_srd(p, (int64_t)min(n, 64) * nb);
    off = lane_id() * nb;
  }
  // word q of every row at lds + q * pitch
  MOK_DEV void dma(int j, uint32_t lds, int pitch) const {
#pragma unroll
    for (int q = 0; q < WORDS; ++q) {
      const int o = (j * WORDS + q) * 4;
      buf4_to_lds(srd, o < nb ? off + o : kNowhere, 0, lds + q * pitch);
    }
  }
};
// of a tile's scale words: the place of second-operand row r. With the gate the rows go in
// blocks of 128, each 64 gate rows and then the 64 up rows of the same columns.
template <bool GLU>
MOK_DEV int scale_at(int r) {
  return GLU ? (r & ~127) | ((r >> 5) & 1) << 6 | ((r >> 6) & 1) << 5 | (r & 31) : r;
}

template <bool A8, bool GLU, int S, class LA, class LB, class LS>
MOK_DEV void mx_loop128(uint8_t* lds, const LA& la, const LB& lb, const LS& ls, int j0, int j1, Acc<2, 2>& acc) {
  using X = MxTile<A8>;
  const uint32_t base = lds_addr(lds);
  const int l = lane_id(), lr = l & 31, hl = l >> 5;
  acc.zero();
  const auto issue = [&](int j, int s) {
    la.dma(j, base + s * X::kSlot);
    lb.dma(j, base + s * X::kSlot + X::kA);
    ls.dma(j, base + s * X::kSlot + X::kA + X::kB + copy_wave() * 256, 1024);
  };
  ring128<S, LA::kDma + LB::kDma + LS::kDma>(j0, j1, issue, [&](int s) {
    const uint8_t* ta = lds + s * X::kSlot;
    const uint8_t* tb = ta + X::kA;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(tb + X::kB);
#pragma unroll
    for (int ks = 0; ks < X::SK / 64; ++ks) {
      i32x8_t a[2], b[2];
      int as[2], bs[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ra = G128::wm() * 64 + 32 * i + lr, rb = G128::wn() * 64 + 32 * i + lr;
        const auto at = [](const uint8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); };
        const i32x4_t z = {0, 0, 0, 0};
        i32x4_t a0, a1 = z, b0;
        if constexpr (A8) {
          a0 = at(ta + lds_at(ra, 4 * ks + hl));
          a1 = at(ta + lds_at(ra, 4 * ks + 2 + hl));
          b0 = at(tb + lds_at64(rb, 2 * ks + hl));
        } else {
          a0 = at(ta + lds_at(ra, 2 * ks + hl));
          b0 = at(tb + lds_at(rb, 2 * ks + hl));
        }
        a[i] = i32x8_t{a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
        b[i] = i32x8_t{b0[0], b0[1], b0[2], b0[3], 0, 0, 0, 0};
        const int sh = 8 * (2 * (ks & 1) + hl), wd = (ks >> 1) * 256;
        as[i] = (int)((sc[wd + ra] >> sh) & 0xFFu);
        bs[i] = (int)((sc[wd + 128 + scale_at<GLU>(rb)] >> sh) & 0xFFu);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          acc.c[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[n], acc.c[i][n], A8 ? 0 : 4, 4, 0,
                                                                        as[i], 0, bs[n]);
    }
  });
}

// ------------------------------------------------------------------ epilogues
// Eight columns from c on of row r as bf16, with the residual added before the
// one rounding; rows that start off a 16-byte boundary, or end inside the eight
// columns, go by element.
MOK_DEV void mx_store8(const mok_mx_args& a, bool vec, int r, int c, float v[8]) {
  if (c >= a.N) return;
  const int64_t o = (int64_t)r * a.ldd + c;
  if (vec && c + 8 <= a.N) {
    if (a.res) {
      float s[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a.res + o), s);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] += s[u];
    }
    store_nt(a.d + o, pack_bf16x8(v));
  } else {
    for (int u = 0; u < 8 && c + u < a.N; ++u)
      a.d[o + u] = f32_to_bf16(a.res ? v[u] + bf16_to_f32(a.res[o + u]) : v[u]);
  }
}

// Eight columns from c on of row r of h = act(g) * u as E4M3 codes; four adjacent lanes
// hold a block, and the first writes its scale.
template <int ACT>
MOK_DEV void mx_gate8(const mok_mx_args& a, int r, int c, const float g[8], const float u[8]) {
  float h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = gate_act<ACT>(g[i]) * u[i];
  const uint32_t m = block_max_bits(h);
  const bool nan = m >= 0x7F800000u;
  const int sc = nan ? 255 : mx_scale_byte(__uint_as_float(m));
  const float inv = mx_inv_scale(sc);
  const uint32_t lo = e4m3_pack4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
  const uint32_t hi = e4m3_pack4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
  *reinterpret_cast<uint2*>(a.hq + (int64_t)r * a.N + c) = nan ? make_uint2(0, 0) : make_uint2(lo, hi);
  if ((c & 31) == 0) a.hs[(int64_t)r * (a.N / 32) + c / 32] = (uint8_t)sc;
}

template <bool GLU>
constexpr int mx_cols() { return GLU ? 64 : 128; }   // output columns of a tile

// The copies of 128 rows of A from m0, of 128 rows of B from n0 (with the gate 64 gate and 64
// up rows), and of the scale words of these by four wavefronts: the first two A's, the others B's.
// (halves past the matrix: as in k_ffn.hip)
template <bool A8>
MOK_DEV auto mx_copy_a(const mok_mx_args& a, int m0) {
  const int64_t ka = A8 ? a.K : a.K / 2;
  m0 = min(m0, a.M - 1);
  return CopyK<MxTile<A8>::RBA, false>(Rows1{a.a + m0 * ka, ka, a.M - m0}, ka);
}
template <bool A8, bool GLU>
MOK_DEV auto mx_copy_b(const mok_mx_args& a, int n0) {
  const int64_t kb = a.K / 2;
  n0 = min(n0, a.N - 1);
  if constexpr (GLU) return CopyK<MxTile<A8>::RBB, true>(Rows2{a.b + n0 * kb, a.b2 + n0 * kb, kb, a.N - n0}, kb);
  else return CopyK<MxTile<A8>::RBB, false>(Rows1{a.b + n0 * kb, kb, a.N - n0}, kb);
}
template <bool A8, bool GLU>
MOK_DEV auto mx_copy_s(const mok_mx_args& a, int m0, int n0) {
  const int64_t ks = a.K / 32;
  const int w = copy_wave(), second = w & 1;
  if (w < 2) {
    m0 = min(m0 + 64 * second, a.M - 1);
    return CopyScales<MxTile<A8>::SK / 128>(a.sa + m0 * ks, a.M - m0, a.K);
  }
  n0 = min(n0 + (GLU ? 0 : 64 * second), a.N - 1);
  return CopyScales<MxTile<A8>::SK / 128>((GLU && second ? a.sb2 : a.sb) + n0 * ks, a.N - n0, a.K);
}

// scale bytes of 64 rows, 16 a row and copy, bytes past a row's end undefined
struct CopyScales16 {
  srd_t srd;
  int off;
  MOK_DEV CopyScales16(const uint8_t* p, int n, int K) {
    srd = make_srd(p, (int64_t)min(n, 64) * (K / 32));
    off = lane_id() * (K / 32);
  }
  MOK_DEV void dma(int m, uint32_t lds) const { buf16_to_lds(srd, off + 16 * m, 0, lds); }
};

// of a 256 x 256 tile: wavefront c of group 0 the scale bytes of 64 of B's rows, of group 1 of
// A's (places of scale_at: with the gate 64 gate, 64 up, 64 gate, 64 up rows)
template <bool GLU>
MOK_DEV auto mx_copy_s16(const mok_mx_args& a, int m0, int n0) {
  const int64_t ks = a.K / 32;
  const int c = pp_col();
  if (pp_group()) {
    m0 = min(m0 + 64 * c, a.M - 1);
    return CopyScales16(a.sa + m0 * ks, a.M - m0, a.K);
  }
  n0 = min(n0 + 64 * (GLU ? c >> 1 : c), a.N - 1);
  return CopyScales16((GLU && (c & 1) ? a.sb2 : a.sb) + n0 * ks, a.N - n0, a.K);
}

template <bool A8, bool GLU, int ACT, bool SPLIT, int S>
__global__ __launch_bounds__(kThreads128<S>, S == 2 ? 2 : 1) void mx128_kernel(mok_mx_args a, bool vec, int nr,
                                                                               int nc, int splits) {
  using X = MxTile<A8>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[lds128<S, X::kSlot>()];
  const int tiles = nr * nc, i = dense_index((int64_t)tiles * splits);
  if (i < 0) return;
  const int split = SPLIT ? i / tiles : 0, t = SPLIT ? i % tiles : i;
  int row, col;
  dense_tile(t, nr, nc, 8, row, col);
  const int m0 = row * 128, n0 = col * mx_cols<GLU>(), nrows = min(128, a.M - m0);
  const int ns = (a.K + X::SK - 1) / X::SK;
  const int j0 = SPLIT ? (int)((int64_t)ns * split / splits) : 0;
  const int j1 = SPLIT ? (int)((int64_t)ns * (split + 1) / splits) : ns;
  Acc<2, 2> acc;
  mx_loop128<A8, GLU, S>(lds, mx_copy_a<A8>(a, m0), mx_copy_b<A8, GLU>(a, n0), mx_copy_s<A8, GLU>(a, m0, n0), j0, j1,
                         acc);
  stage128<S>(lds, acc);
  if constexpr (SPLIT) {
    float* p = a.part + ((int64_t)split * tiles + t) * 16384;
    for (int idx = threadIdx.x; idx < nrows * 32; idx += kThreads128<S>)
      reinterpret_cast<float4*>(p)[idx] =
          *reinterpret_cast<const float4*>(lds + (idx >> 5) * kPitch128 + (idx & 31) * 16);
  } else if constexpr (GLU) {
    for (int idx = threadIdx.x; idx < nrows * 8; idx += kThreads128<S>) {
      const int r = idx >> 3, c = (idx & 7) * 8;
      if (n0 + c >= a.N) continue;               // (N a multiple of 128: whole blocks)
      float g[8], u[8];
      const uint8_t* p = lds + r * kPitch128 + ((c >> 5) * 64 + (c & 31)) * 4;
      load_f32<8>(p, g);
      load_f32<8>(p + 128, u);
      mx_gate8<ACT>(a, m0 + r, n0 + c, g, u);
    }
  } else {
    for (int idx = threadIdx.x; idx < nrows * 16; idx += kThreads128<S>) {
      const int r = idx >> 4, c = (idx & 15) * 8;
      float v[8];
      load_f32<8>(lds + r * kPitch128 + c * 4, v);
      mx_store8(a, vec, m0 + r, n0 + c, v);
    }
  }
}

template <bool GLU, int ACT, int TS>
__global__ __launch_bounds__(kThreads) void mx_join_kernel(mok_mx_args a, bool vec, int nr, int nc, int splits) {
  constexpr int NC = GLU ? TS / 2 : TS, CH = NC / 8;
  const int tiles = nr * nc, t = (int)blockIdx.y;
  int row, col;
  dense_tile(t, nr, nc, TS == 256 ? 4 : 8, row, col);
  const int idx = (int)blockIdx.x * kThreads + (int)threadIdx.x;
  const int r = idx / CH, c = (idx % CH) * 8, gc = col * NC + c;
  if (r >= min(TS, a.M - row * TS) || gc >= a.N) return;
  const float* p = a.part + (int64_t)t * TS * TS + r * TS + (GLU ? (c >> 5) * 64 + (c & 31) : c);
  float v[8], u[8];
  sum_splits(p, (int64_t)tiles * TS * TS, splits, v);
  if constexpr (GLU) {
    sum_splits(p + 32, (int64_t)tiles * TS * TS, splits, u);
    mx_gate8<ACT>(a, row * TS + r, gc, v, u);
  } else {
    mx_store8(a, vec, row * TS + r, gc, v);
  }
}

// ------------------------------------------------------------------ product, 256 x 256 tile
// The two alternating groups of dense_core.h. A slot holds SK elements of K; the
// products of half a slot take as long as those of half a bf16 slot. With both operands
// in E2M1 there is room for a third buffer of only one half of A: group 1 copies its
// half of s+1 in interval 4s+3 and waits for it in 4s+4, before it reads in 4s+5.
// Scale bytes come 16 per row (512 of K) and copy, every 512 / SK slots: a copy of one
// word per row takes as long, and they would be a third of all cache lines asked for.
template <bool A8>
struct MxPp {
  static constexpr int SK = A8 ? 128 : 256;
  static constexpr int RBB = SK / 2;             // bytes of a row of B per slot; of A: 128
  static constexpr int kD1 = A8 ? 3 : 2;         // buffers of group 1's half of A
  static constexpr int kHA = 128 * 128, kHB = 128 * RBB;
  static constexpr int kOffB = (3 + kD1) * kHA, kOffS = kOffB + 4 * kHB, kS = 512 * 16;
  static constexpr int kLds = kOffS + 2 * kS;    // 144 and 160 KiB
  static constexpr int kPer = 512 / SK;          // slots per copy of scales
};

// first operand B (E2M1), second A: the transposed product. OPS: the byte of the scale words
template <bool A8, int OPS>
MOK_DEV f32x16_t mx_mma(const i32x8_t& b, const i32x8_t& a, const f32x16_t& c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 4, A8 ? 0 : 4, OPS, sb, OPS, sa);
}

template <bool A8, bool GLU, class LA, class LB>
MOK_DEV void mx_pp_loop(uint8_t* lds, const LA& la, const LB& lb, const CopyScales16& ls, int K, int j0, int ns,
                        Acc<4, 2>& acc) {
  using X = MxPp<A8>;
  const int grp = pp_group(), c = pp_col(), l = lane_id(), lr = l & 31, hl = l >> 5;
  const bool third = !grp || X::kD1 == 3;        // a third buffer of this group's half of A
  const uint32_t base = lds_addr(lds), oa = grp * 3 * X::kHA, last = (third ? 2 : 1) * X::kHA;
  const uint32_t sdst = base + X::kOffS + (grp ? 0 : 4096) + c * 1024;   // A's rows, then B's
  acc.zero();
  ls.dma(j0 / X::kPer, sdst + ((j0 / X::kPer) & 1) * X::kS);
  lb.dma(j0, base + X::kOffB + grp * X::kHB);
  la.dma(j0, base + oa);
  if (third && ns > j0 + 1) {
    la.dma(j0 + 1, base + oa + X::kHA);
    wait_vm_lds<4>();
  } else {
    wait_vm_lds<0>();
  }
  barrier_lds();
  if (grp) barrier_lds();
  // fragments of half a slot: one K step of 64 (A8) or two
  constexpr int KK = A8 ? 1 : 2;
  i32x4_t a[KK][4][A8 ? 2 : 1], b[KK][2];
  int as[4], bs[2];
  const auto read = [&](const uint8_t* ta, const uint8_t* tb, const uint8_t* ts, int s, int h) {
    const auto at = [](const uint8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); };
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int ks = KK * h + kk;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = 64 * (c & 1) + 32 * n + lr;
        b[kk][n] = at(tb + (A8 ? lds_at64(r, 2 * ks + hl) : lds_at(r, 2 * ks + hl)));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lr;
        if constexpr (A8) {
          a[kk][i][0] = at(ta + lds_at(r, 4 * ks + hl));
          a[kk][i][A8 ? 1 : 0] = at(ta + lds_at(r, 4 * ks + 2 + hl));
        } else {
          a[kk][i][0] = at(ta + lds_at(r, 2 * ks + hl));
        }
      }
    }
    if (A8 && h) return;                         // the word of both halves
    // scale words of these 128 of K: byte 2 kk + hl (A8: 2 h + hl) is this lane's block
    const int w = 4 * (A8 ? s % X::kPer : 2 * (s % X::kPer) + h);
    // (past K the bytes are another row's)
    const uint32_t in = A8 || X::SK * s + 128 * h < K ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(ts + (128 * grp + 32 * i + lr) * 16 + w);
      as[i] = (int)((v & in) >> (8 * hl));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint32_t v =
          *reinterpret_cast<const uint32_t*>(ts + 4096 + scale_at<GLU>(64 * c + 32 * n + lr) * 16 + w);
      bs[n] = (int)((v & in) >> (8 * hl));
    }
  };
  const auto multiply = [&](auto hc) {
    constexpr int h = decltype(hc)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    pin(b[0][0]);
    const auto step = [&](auto kc) {
      constexpr int kk = decltype(kc)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const i32x4_t lo = a[kk][i][0];
        i32x8_t av = {lo[0], lo[1], lo[2], lo[3], 0, 0, 0, 0};
        if constexpr (A8) {
          const i32x4_t hi = a[kk][i][A8 ? 1 : 0];
          av = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const i32x4_t q = b[kk][n];
          const i32x8_t bv = {q[0], q[1], q[2], q[3], 0, 0, 0, 0};
          acc.c[i][n] = mx_mma<A8, 2 * (A8 ? h : kk)>(bv, av, acc.c[i][n], bs[n], as[i]);
        }
      }
    };
    step(std::integral_constant<int, 0>{});
    if constexpr (KK == 2) step(std::integral_constant<int, 1>{});
    pin_acc(acc);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  const int ahead = third ? 2 : 1;               // A of s + ahead is copied during s
  uint32_t s0 = 0, sn = last;                    // A's buffers of s and s + ahead
  for (int s = j0; s < ns; ++s) {
    const int par = (s - j0) & 1;
    const uint8_t* ta = lds + oa + s0;
    const uint8_t* tb = lds + X::kOffB + (par * 2 + (c >> 1)) * X::kHB;
    const uint8_t* ts = lds + X::kOffS + ((s / X::kPer) & 1) * X::kS;
    const bool more = s + ahead < ns;
    read(ta, tb, ts, s, 0);
    // (the other buffer of scales was last read for slot s - 1, or not yet)
    if ((s % X::kPer == 0 || s == j0) && (s / X::kPer + 1) * X::kPer < ns)
      ls.dma(s / X::kPer + 1, sdst + ((s / X::kPer + 1) & 1) * X::kS);
    if (s + 1 < ns) lb.dma(s + 1, base + X::kOffB + ((par ^ 1) * 2 + grp) * X::kHB);
    barrier_lds_only();
    multiply(std::integral_constant<int, 0>{});
    barrier_lds();
    read(ta, tb, ts, s, 1);
    if (more) la.dma(s + ahead, base + oa + sn);
    if (grp) pp_wait<4>(more);
    barrier_lds_only();
    multiply(std::integral_constant<int, 1>{});
    if (!grp) pp_wait<4>(more);
    else if (X::kD1 == 2) wait_vm_lds<0>();
    barrier_lds();
    s0 = s0 == last ? 0 : s0 + X::kHA;
    sn = sn == last ? 0 : sn + X::kHA;
  }
  if (!grp) barrier_lds();
}

// VAR: the gate's kind, or 1 = with a residual
template <bool A8, bool GLU, int VAR, bool SPLIT>
__global__ __launch_bounds__(kPpThreads, 1) void mx256_kernel(mok_mx_args a, bool vec, int nr, int nc, int splits) {
  using X = MxPp<A8>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[X::kLds];
  const int tiles = nr * nc, ix = dense_index((int64_t)tiles * splits);
  if (ix < 0) return;
  const int split = SPLIT ? ix / tiles : 0, t = SPLIT ? ix % tiles : ix;
  int row, col;
  dense_tile(t, nr, nc, 4, row, col);
  const int ns = (a.K + X::SK - 1) / X::SK;
  const int j0 = SPLIT ? (int)((int64_t)ns * split / splits) : 0;
  const int j1 = SPLIT ? (int)((int64_t)ns * (split + 1) / splits) : ns;
  const int m0 = row * 256, n0 = col * (GLU ? 128 : 256), nrows = min(256, a.M - m0);
  Acc<4, 2> acc;
  const int g = pp_group();
  mx_pp_loop<A8, GLU>(lds, mx_copy_a<A8>(a, m0 + 128 * g), mx_copy_b<A8, GLU>(a, n0 + mx_cols<GLU>() * g),
                      mx_copy_s16<GLU>(a, m0, n0), a.K, j0, j1, acc);
  if constexpr (SPLIT) {
    pp_store32(lds, acc, nrows, a.part + ((int64_t)split * tiles + t) * 65536);
  } else if constexpr (GLU) {
    // a lane holds 16 of the 32 columns of a block of h, lane l ^ 32 the others. Codes go
    // through LDS (128 bytes a row, 16-byte chunk c of row r at c ^ (r & 7))
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float h[16];
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        h[q] = gate_act<VAR>(acc.c[i][0][q]) * acc.c[i][1][q];
        m = max(m, __float_as_uint(h[q]) & 0x7FFFFFFFu);
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      const bool nan = m >= 0x7F800000u;
      const int sc = nan ? 255 : mx_scale_byte(__uint_as_float(m)), r = pp_row(i), c = pp_col(), hl = lane_id() >> 5;
      const float inv = mx_inv_scale(sc);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = e4m3_pack4(h[4 * q] * inv, h[4 * q + 1] * inv, h[4 * q + 2] * inv, h[4 * q + 3] * inv);
        *reinterpret_cast<uint32_t*>(lds + r * 128 + (((2 * c + (q >> 1)) ^ (r & 7)) << 4) + (q & 1) * 8 + hl * 4) =
            nan ? 0u : w;
      }
      if (hl == 0 && r < nrows && n0 + 32 * c < a.N)
        a.hs[(int64_t)(m0 + r) * (a.N / 32) + n0 / 32 + c] = (uint8_t)sc;
    }
    barrier_lds_only();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int idx = (int)threadIdx.x + u * kPpThreads, r = idx >> 3, ch = idx & 7;
      if (r < nrows && n0 + 16 * ch < a.N)
        *reinterpret_cast<uint4*>(a.hq + (int64_t)(m0 + r) * a.N + n0 + 16 * ch) =
            *reinterpret_cast<const uint4*>(lds + r * 128 + ((ch ^ (r & 7)) << 4));
    }
  } else {
    if constexpr (VAR == 1) {                    // (a block's y: aligned rows, N a multiple of 128)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          pp_add_residual(acc.c[i][n], a.res, a.ldd, m0 + min(pp_row(i), nrows - 1), n0 + pp_col0(n, 0), a.N);
      __syncthreads();                           // (the residual may be y itself)
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          pp_put4(lds + pp_at16<256>(pp_row(i), pp_col0(n, q)), acc.c[i][n][4 * q], acc.c[i][n][4 * q + 1],
                  acc.c[i][n][4 * q + 2], acc.c[i][n][4 * q + 3]);
    barrier_lds_only();
    pp_rows16<256>(lds, nrows, [&](int r, int c, uint4 v) {
      if (n0 + c >= a.N) return;
      bf16_t* d = a.d + (int64_t)(m0 + r) * a.ldd + n0 + c;
      if (vec && n0 + c + 8 <= a.N) {
        store_nt(d, v);
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int u = 0; u < 8 && n0 + c + u < a.N; ++u) d[u] = (bf16_t)(w[u >> 1] >> (16 * (u & 1)));
      }
    });
  }
}

// ------------------------------------------------------------------ few rows
// The scheme of dense_core.h with v_mfma_scale_f32_16x16x128_f8f6f4: the 16 weight
// rows (E2M1) are the first operand, 16 rows of A the second; lane l supplies row
// l % 16 with the 32 weights from 32 g on (g = l / 16, 16 bytes), of E4M3 the 16 bytes
// from 16 g on and those 64 further, and the scale of block g (checked on gfx950).
// The rows of A are quantized by a launch of their own, which takes 2.5 us: every
// workgroup quantizing them as it reads them (256 or more repeat the work, on two or four
// times the bytes) took 9 us more for x at 16 rows of 7168, and for h at rows of 2048 2 us
// more at one row and 5 us at 16. So h, of which a workgroup makes 8 columns and a block has 32,
// goes out as fp32.
// Up to 32 rows this is the faster way at every size timed. us against 128 x 128 tiles, A in
// MXFP8: 4096 x 7168 at 1, 16, 32 rows 6.3, 9.3, 12.9 against 13.9, 15.4, 15.8; 7168 x 2048 4.6,
// 6.3, 9.6 against 9.9, 10.1, 10.3; 512 x 1024 2.7, 3.4, 4.1 against 6.4, 6.5, 6.5; in MXFP4 at
// 32 rows 10.4 against 14.0, 7.7 against 8.4, 3.7 against 5.7. (More rows have no variant here.)
constexpr int kMxFewRows = 32;

template <bool A8, bool GLU, int ACT, int NT>
__global__ __launch_bounds__(kFewThreads) void mx_few_kernel(mok_mx_args a) {
  constexpr int kX = A8 ? 2 : 1;                 // 16-byte pieces of a row of A per step
  constexpr int U = 4;                           // steps per batch: one scale word per lane group
  __shared__ __attribute__((aligned(16))) float red[kFewWaves * NT * 256];
  const int l = lane_id(), lr = l & 15, g = l >> 4;
  const int c0 = (int)flat_block() * (GLU ? 8 : 16);
  if (c0 >= a.N) return;                         // (the last row of a flat grid)
  const int64_t kb = a.K / 2, ks = a.K / 32;
  const uint8_t* wp;
  const uint8_t* wsp;
  if constexpr (GLU) {
    wp = (lr < 8 ? a.b : a.b2) + (c0 + (lr & 7)) * kb;
    wsp = (lr < 8 ? a.sb : a.sb2) + (c0 + (lr & 7)) * ks;
  } else {
    wp = a.b + min(c0 + lr, a.N - 1) * kb;
    wsp = a.sb + min(c0 + lr, a.N - 1) * ks;
  }
  const uint8_t* xp[NT];
  const uint8_t* xsp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = min(16 * n + lr, a.M - 1);
    xp[n] = a.a + t * (A8 ? (int64_t)a.K : kb);
    xsp[n] = a.sa + t * ks;
  }
  const int ns = a.K / 128;
  const int b = ns * wave_id() / kFewWaves, e = ns * (wave_id() + 1) / kFewWaves;
  i32x4_t wv[2][U], xv[2][U][NT][kX];
  int wsv[2], xsv[2][NT];                        // scale words of step j0 + g
  f4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f4_t{0.f, 0.f, 0.f, 0.f};
  const auto load = [&](int s, int j0) {
    const int jg = min(j0 + g, ns - 1);
    wsv[s] = *reinterpret_cast<const int*>(wsp + 4 * jg);
#pragma unroll
    for (int n = 0; n < NT; ++n) xsv[s][n] = *reinterpret_cast<const int*>(xsp[n] + 4 * jg);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      if (j >= e) continue;                      // wave-uniform
      wv[s][u] = *reinterpret_cast<const i32x4_t*>(wp + 64 * j + 16 * g);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < kX; ++q)
          xv[s][u][n][q] = *reinterpret_cast<const i32x4_t*>(xp[n] + (A8 ? 128 * j + 64 * q : 64 * j) + 16 * g);
    }
  };
  const auto compute = [&](int s, int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u >= e) continue;                 // wave-uniform
      const i32x4_t w = wv[s][u];
      const i32x8_t wa = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
      const int from = 16 * u + lr;              // the lane that holds this step's scale words
      const int sw = (__shfl(wsv[s], from) >> (8 * g)) & 0xFF;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        i32x8_t x = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < kX; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[4 * q + i] = xv[s][u][n][q][i];
        const int sx = (__shfl(xsv[s][n], from) >> (8 * g)) & 0xFF;
        acc[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, x, acc[n], 4, A8 ? 0 : 4, 0, sw, 0, sx);
      }
    }
  };
  few_pipeline<U>(b, e, load, compute);
  few_put<NT>(red, acc);
  if constexpr (GLU) {
    for (int i = threadIdx.x; i < 8 * a.M; i += kFewThreads) {
      const int c = i & 7, t = i >> 3;
      a.hf[(int64_t)t * a.N + c0 + c] = gate_act<ACT>(few_get<NT>(red, c, t)) * few_get<NT>(red, c + 8, t);
    }
  } else {
    for (int i = threadIdx.x; i < 16 * a.M; i += kFewThreads) {
      const int c = i & 15, t = i >> 4;
      if (c0 + c >= a.N) continue;
      float v = few_get<NT>(red, c, t);
      const int64_t o = t * a.ldd + c0 + c;
      if (a.res) v += bf16_to_f32(a.res[o]);
      a.d[o] = f32_to_bf16(v);
    }
  }
}

template <bool A8, bool GLU, int ACT>
hipError_t launch_few(const mok_mx_args& a, hipStream_t st) {
  const dim3 grid = flat_grid(GLU ? a.N / 8 : (a.N + 15) / 16), block(kFewThreads);
  if (a.M <= 16) hipLaunchKernelGGL((mx_few_kernel<A8, GLU, ACT, 1>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((mx_few_kernel<A8, GLU, ACT, 2>), grid, block, 0, st, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ host
struct Plan {
  int tile, nr, nc, splits;                      // tile 0: few rows
};
// (slots of 128, of 256)
constexpr dense_cost kCost8 = {10.1f, 1.80f, 10.5f, 1.36f, 0.28f, 3.5f, 6.7e6f};
constexpr dense_cost kCost4 = {17.3f, 1.85f, 8.7f, 1.25f, 0.31f, 2.2f, 2.8e6f};

Plan plan_of(const mok_mx_args& a, bool glu) {
  if (mok_mx_few(a.M)) return Plan{0, 0, 0, 1};
  Plan p;
  const int64_t cols = (glu ? 2 : 1) * (int64_t)a.N;
  const int slot = a.a8 ? 128 : 256;             // of K; the last may be half full
  dense_plan(a.M, cols, 1, (a.K + slot - 1) / slot, a.a8 ? kCost8 : kCost4, &p.tile, &p.splits);
  p.nr = (a.M + p.tile - 1) / p.tile;
  p.nc = (int)((cols + p.tile - 1) / p.tile);
  return p;
}

template <bool A8, bool GLU, int ACT>
hipError_t launch(const mok_mx_args& a, const Plan& p, hipStream_t st) {
  const int64_t tiles = (int64_t)p.nr * p.nc;
  if (tiles == 0) return hipSuccess;
  const bool vec = a.ldd % 8 == 0 && ((uintptr_t)a.d | (uintptr_t)a.res) % 16 == 0;
  const dim3 grid(dense_grid(tiles * p.splits)), block(p.tile == 256 || tiles * p.splits <= 256 ? 512 : 256);
  const int nr = p.nr, nc = p.nc;
  if (p.splits > 1) {
    if (p.tile == 256)
      hipLaunchKernelGGL((mx256_kernel<A8, GLU, 0, true>), grid, block, 0, st, a, vec, nr, nc, p.splits);
    else if (tiles * p.splits <= 256)
      hipLaunchKernelGGL((mx128_kernel<A8, GLU, 0, true, 4>), grid, block, 0, st, a, vec, nr, nc, p.splits);
    else
      hipLaunchKernelGGL((mx128_kernel<A8, GLU, 0, true, 2>), grid, block, 0, st, a, vec, nr, nc, p.splits);
    const int ch = p.tile * (GLU ? p.tile / 2 : p.tile) / 8;
    const dim3 jgrid((ch + kThreads - 1) / kThreads, (unsigned)tiles);
    if (p.tile == 256)
      hipLaunchKernelGGL((mx_join_kernel<GLU, ACT, 256>), jgrid, dim3(kThreads), 0, st, a, vec, nr, nc, p.splits);
    else
      hipLaunchKernelGGL((mx_join_kernel<GLU, ACT, 128>), jgrid, dim3(kThreads), 0, st, a, vec, nr, nc, p.splits);
  } else if (p.tile == 256) {
    if (!GLU && a.res)
      hipLaunchKernelGGL((mx256_kernel<A8, GLU, GLU ? ACT : 1, false>), grid, block, 0, st, a, vec, nr, nc, 1);
    else
      hipLaunchKernelGGL((mx256_kernel<A8, GLU, ACT, false>), grid, block, 0, st, a, vec, nr, nc, 1);
  } else if (tiles <= 256) {
    hipLaunchKernelGGL((mx128_kernel<A8, GLU, ACT, false, 4>), grid, block, 0, st, a, vec, nr, nc, 1);
  } else {
    hipLaunchKernelGGL((mx128_kernel<A8, GLU, ACT, false, 2>), grid, block, 0, st, a, vec, nr, nc, 1);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t mok_launch_mxfp4_quantize(const bf16_t* src, int64_t rows, int64_t K, uint8_t* q, uint8_t* scales,
                                     hipStream_t st) {
  const int64_t n8 = rows * (K / 8);
  if (n8 <= 0) return hipSuccess;
  const dim3 grid = flat_grid((n8 + 255) / 256);
  hipLaunchKernelGGL(mxfp4_quantize_kernel, grid, dim3(256), 0, st, src, n8, q, scales);
  return hipGetLastError();
}

hipError_t mok_launch_mxfp4_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K,
                                       bf16_t* dst, hipStream_t st) {
  const int64_t n8 = rows * (K / 8);
  if (n8 <= 0) return hipSuccess;
  const dim3 grid = flat_grid((n8 + 255) / 256);
  hipLaunchKernelGGL(mxfp4_dequantize_kernel, grid, dim3(256), 0, st, q, scales, n8, dst);
  return hipGetLastError();
}

hipError_t mok_launch_mxfp8_rows(const void* src, bool f32, int64_t ld, int64_t rows, int64_t K, uint8_t* q,
                                 uint8_t* scales, hipStream_t st) {
  const int64_t n8 = rows * (K / 8);
  if (n8 <= 0) return hipSuccess;
  const dim3 grid = flat_grid((n8 + 255) / 256);
  if (f32)
    hipLaunchKernelGGL(mxfp8_rows_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(src), ld, n8,
                       (int)(K / 8), q, scales);
  else
    hipLaunchKernelGGL(mxfp8_rows_kernel<bf16_t>, grid, dim3(256), 0, st, static_cast<const bf16_t*>(src), ld, n8,
                       (int)(K / 8), q, scales);
  return hipGetLastError();
}

size_t mok_mx_part_bytes(const mok_mx_args& a, bool glu) {
  const Plan p = plan_of(a, glu);
  return p.splits > 1 ? (size_t)p.splits * p.nr * p.nc * p.tile * p.tile * 4 : 0;
}

bool mok_mx_few(int M) { return M <= kMxFewRows; }

hipError_t mok_launch_mx(const mok_mx_args& a, bool glu, int act, hipStream_t st) {
  if (mok_mx_few(a.M)) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    if (glu) return act == 0 ? launch_few<true, true, 0>(a, st) : launch_few<true, true, 1>(a, st);
    return a.a8 ? launch_few<true, false, 0>(a, st) : launch_few<false, false, 0>(a, st);
  }
  const Plan p = plan_of(a, glu);
  if (!glu) return a.a8 ? launch<true, false, 0>(a, p, st) : launch<false, false, 0>(a, p, st);
  if (!a.a8) return hipErrorInvalidValue;
  return act == 0 ? launch<true, true, 0>(a, p, st) : launch<true, true, 1>(a, p, st);
}
