// Router backward from the gradient of every logit: dx = dl . Wr (+ residual)
// and dWr = dl^T . x, on the matrix cores. dl and Wr are fp32, the operands bf16: dl
// and Wr are split exactly into three bf16 parts each. For dWr, x is bf16, so every
// product is exact. For dx, of the nine products of parts the six down to 2^-16 of the
// whole go in, all exact; the other three are less than 2^-21 of it, in the mean square
// less than half of what fp32 sums lose. Two parts each do not do, although dx is
// rounded to bf16 in the end: a row of dl adds up to nearly zero over the experts, and
// they moved 0.3% of the roundings at 1037 x 2048 with 60 experts, an fp32 product 0.01%.
//
// Bound by memory with few experts (16384 x 7168, 32 experts, residual: 141 us for
// 708 MB, 5.0 TB/s; a copy reaches 4.9), by the matrix instructions and the staging
// beside them with many (16384 x 4096 with 128: 155 GFLOP in 155 us, the matrix cores
// busy 48% of dx's 91 us and 43% of dWr's 58).
#include <algorithm>
#include <type_traits>

#include "bf16_split.h"
#include "gemm_core.h"
#include "router_launch.h"

using namespace mok;

namespace {

typedef __attribute__((ext_vector_type(4))) short i16x4_t;
typedef __attribute__((ext_vector_type(8))) short i16x8_t;
typedef __attribute__((address_space(3))) i16x4_t* lds_i16x4_ptr;

MOK_DEV float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
MOK_DEV float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

MOK_DEV f32x16_t mfma32(const uint4& a, const uint4& b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}
MOK_DEV f32x4_t mfma16(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

// Loads and stores go through buffer descriptors: what lies past a descriptor's
// bytes reads as zero and is not written, so that no access stands in a branch.
// (With branches round them the compiler cannot tell how many are in flight at the
// wait for one, and waits for all: dWr of 16384 x 4096 with 128 experts 77 us against
// 57.) A 16-byte load that the end of the bytes cuts reads its part before the end and
// zeros (checked on gfx950). Offsets are 32 bits: a step's rows, at most 2^26 bytes of
// x, dx and the residual, and 2^27 of Wr.
typedef __amdgpu_buffer_rsrc_t buf_t;
constexpr uint32_t kOut = 0x7ffffff0u;           // past every descriptor's bytes
MOK_DEV buf_t make_buf(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(p && bytes > 0 ? bytes : 0), 0x00020000);
}
MOK_DEV uint4 load16(buf_t b, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}
MOK_DEV void store16(buf_t b, uint32_t off, const uint4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), b, (int)off, 0, 2);
}

// Workgroup b of n in an order that gives each of the eight dies (workgroups go
// round them) a contiguous share, so that the panels of one slice of tokens, which
// read the same rows of dl, share an L2.
MOK_DEV int die_order(int b, int n) { return n % 8 ? b : b % 8 * (n / 8) + b / 8; }

// tokens of slice s of n, in whole blocks of 32
struct Slice {
  int64_t t0, t1;
  MOK_DEV Slice(int64_t T, int s, int n) {
    const int64_t blocks = (T + 31) / 32;
    t0 = blocks * s / n * 32;
    t1 = min(blocks * (s + 1) / n * 32, T);
  }
};

// f(step's buffer, first token) for every ST tokens. With the loads of two steps in
// flight (AHEAD) the buffer is a constant, as the registers that hold a step are; with
// one it is not, and the accumulators have one place (in two copies of the step, which
// the loop leaves after either, they take twice their registers).
template <int AHEAD, int ST, class F>
MOK_DEV void steps(const Slice& s, F&& f) {
  if constexpr (AHEAD == 1) {
    int p = 0;
#pragma unroll 1
    for (int64_t t = s.t0; t < s.t1; t += ST, p ^= 1) f(p, t);
  } else {
    for (int64_t t = s.t0; t < s.t1; t += 2 * ST) {
      f(0, t);
      if (t + ST >= s.t1) break;
      f(1, t + ST);
    }
  }
}

// ---------------------------------------------------------------- kernel
// A workgroup of eight wavefronts takes 128 MT columns and a slice of the tokens, ST
// tokens at a time through two sets of LDS buffers: while one is multiplied, the other
// is filled from registers that were loaded two steps ahead (one where registers are
// few). Its barriers wait for LDS alone (__syncthreads would wait for every load and
// store in flight). With much data a workgroup forms both results (DX and DWR) up to 64
// experts, so that dl is read and split once (16384 x 4096 with 64 experts: 104 us, as a
// pair 113), and beyond, where Wr leaves no registers for that, there is a launch for
// each. With little data, up to 128 experts, workgroups of either kind share the CUs,
// two on each, one's instructions beside the other's copies. DWR takes 128 experts a
// workgroup at most.
//
// dl of a step lies in LDS as bf16 parts [ST tokens][EP experts]; 16-byte chunk c
// of token row t at c ^ swz(t): eight rows at one chunk (dx), and four rows at two
// neighbouring chunks (dWr, transposed), fall on the eight places of 128 bytes.
//
// dx: the columns of dx are rows of the first operand, tokens columns of the
// second. A wavefront keeps its 16 MT columns of Wr, all parts, in registers (12 MT KS
// of them, KS = EP / 32) and the tokens stream past. v_mfma_f32_16x16x32_bf16: lane
// l supplies row l % 16 of an operand, 8 values of K from 8 (l / 16) on, and holds
// of result column l % 16 the rows 4 (l / 16) + i. Row r of the wavefront's tile m
// is column 4 MT (r / 4) + 4 m + r % 4, so a lane ends up with 4 MT neighbouring
// columns of a token. dx goes through LDS once more, in fp32, so that rows of it and
// of the residual are written and read in 256 MT bytes (with 32 experts and two parts
// 16384 x 7168 took 155 us in the operand's 64-byte pieces, so 138). One tile a wavefront
// halves Wr's registers and doubles the reading of dl from LDS: beyond 256 experts
// (16384 x 4096 with 512: 580 us in eight wavefronts of one tile, 755 in four of two).
//
// dWr: x as it is and dl in its three parts are both read transposed
// (ds_read_b64_tr_b16: lane 4 q + p of 16 names row q and columns 4 p .. + 3, and
// gets column l of the four rows) for v_mfma_f32_32x32x16_bf16 (lane l supplies row
// l % 32 of an operand, 8 values of K from 8 (l / 32) on, and holds of result column
// l % 32 the rows 8 (i / 4) + 4 (l / 32) + i % 4). The slices' sums, one [E][H] each,
// are added in ascending order by router_dwr_join_kernel.
MOK_DEV int swz(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

struct Plan {
  int panels, eblocks, slices;
  __host__ __device__ int groups() const { return panels * eblocks * slices; }
};

// LOW: registers for two workgroups on a CU
constexpr int NW = 8;
template <int KS, bool DX, bool DWR, int AHEAD, bool LOW, int MT = 2, int ST = 32>
struct Body {
  static_assert((!DWR || (MT == 2 && ST == 32)) && ST % 16 == 0, "dWr's tiles");
  static constexpr int BT = 64 * NW, NC = 16 * MT * NW, EP = 32 * KS, NT = ST / 16;
  static constexpr int DP = 2 * EP < 128 ? 128 : 2 * EP, XP = 2 * NC;  // row pitches of dl and x in bytes
  static constexpr int PARTS = 3;
  static constexpr int kD = ST * DP, kX = DWR ? ST * XP : 0;
  static constexpr int kW = DX ? 32 * (NC + 4) * 4 : 0;                // 32 rows of Wr, before the first step
  static constexpr int OP = 4 * NC + 16, kO = DX ? ST * OP : 0, NO = (ST * NC / 8 + BT - 1) / BT;
  static constexpr int kBuf = 2 * (PARTS * kD + kX) + kO, kLds = kBuf > kW ? kBuf : kW;
  static constexpr int WM = KS == 4 ? 2 : 1, TM = KS / WM, TN = WM;    // dWr: 32 x 32 tiles of a wavefront
  static constexpr int ND = (ST * EP / 4 + BT - 1) / BT, NX = ST * NC / 8 / BT;   // 16-byte loads of a thread and step

  MOK_DEV static void run(const mok_logits_bwd_args& a, const Plan& plan, int block, uint8_t* lds);
};

template <int KS, bool DX, bool DWR, int AHEAD, bool LOW, int MT, int ST>
MOK_DEV void Body<KS, DX, DWR, AHEAD, LOW, MT, ST>::run(const mok_logits_bwd_args& a, const Plan& plan, int block,
                                                        uint8_t* lds) {
  const int panels = plan.panels, eblocks = plan.eblocks, slices = plan.slices;
  const auto dl_buf = [&](int buf, int part) { return lds + (buf * PARTS + part) * kD; };
  const auto x_buf = [&](int buf) { return lds + 2 * PARTS * kD + buf * kX; };
  const int b = die_order(block, plan.groups());
  const int panel = b % panels, eb = b / panels % eblocks, slice = b / (panels * eblocks);
  const Slice sl(a.T, slice, slices);
  const int wave = wave_id(), lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int c0 = panel * NC, e0 = eb * EP;
  const int nks = (a.E - e0 + 31) / 32;          // steps of 32 experts that hold any

  // ---- Wr: 32 rows at a time through LDS into the operand's registers
  uint4 w[3][MT][DX ? KS : 1];
  if constexpr (DX) {
    constexpr int NWL = 32 * NC / 4 / BT;
    float* wl = reinterpret_cast<float*>(lds);
    uint4 wn[NWL];
    const auto load_w = [&](int s) {
      const buf_t src = make_buf(a.wr + (int64_t)32 * s * a.H + c0, ((int64_t)min(a.E - 32 * s, 32) * a.H - c0) * 4);
#pragma unroll
      for (int i = 0; i < NWL; ++i) {
        const int q = (int)threadIdx.x + BT * i;
        wn[i] = load16(src, 4u * (q / (NC / 4) * a.H + 4 * (q % (NC / 4))));
      }
    };
    load_w(0);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int i = 0; i < NWL; ++i) {
        const int q = (int)threadIdx.x + BT * i;
        *reinterpret_cast<uint4*>(wl + q / (NC / 4) * (NC + 4) + 4 * (q % (NC / 4))) = wn[i];
      }
      if (s + 1 < KS) load_w(s + 1);
      barrier_lds_only();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = wl[(8 * g + u) * (NC + 4) + 16 * MT * wave + 4 * MT * (r >> 2) + 4 * m + (r & 3)];
        split3(v[0], v[1], w[0][m][s].x, w[1][m][s].x, w[2][m][s].x);
        split3(v[2], v[3], w[0][m][s].y, w[1][m][s].y, w[2][m][s].y);
        split3(v[4], v[5], w[0][m][s].z, w[1][m][s].z, w[2][m][s].z);
        split3(v[6], v[7], w[0][m][s].w, w[1][m][s].w, w[2][m][s].w);
      }
      barrier_lds_only();
    }
  }

  f32x16_t acc[DWR ? TM : 1][DWR ? TN : 1];
  if constexpr (DWR) {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
  }

  // a thread's places in a step's rows, in bytes from the first of them
  uint8_t* o_buf = lds + 2 * (PARTS * kD + kX);
  uint32_t doff[ND], xoff[DWR ? NX : 1], roff[NO];
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int q = (int)threadIdx.x + BT * i, row = q / (EP / 4), e = 4 * (q % (EP / 4));
    doff[i] = row < ST && e0 + e < a.E ? 4u * (row * a.E + e) : kOut;
  }
  if constexpr (DWR) {
    // (columns past H read the next row, for sums that are not stored)
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int q = (int)threadIdx.x + BT * i;
      xoff[i] = 2u * (q / (NC / 8) * a.H + 8 * (q % (NC / 8)));
    }
  }
#pragma unroll
  for (int i = 0; i < NO; ++i) {
    const int q = (int)threadIdx.x + BT * i, c = c0 + 8 * (q % (NC / 8));
    roff[i] = c < a.H && q / (NC / 8) < ST ? 2u * (q / (NC / 8) * a.H + c) : kOut;
  }
  // of four experts from 4 j on, how many there are (E is not always a multiple of 4: the others' place holds the next
  // token's, and must not enter a product)
  const auto loaded = [&](int i) { return a.E - e0 - 4 * (((int)threadIdx.x + BT * i) % (EP / 4)); };

  uint4 dn[AHEAD][ND], xn[AHEAD][DWR ? NX : 1], rn[AHEAD][DX ? NO : 1];
  const auto load = [&](int buf, int64_t t) {
    const int P = buf % AHEAD;
    const int64_t left = min(sl.t1 - t, (int64_t)ST);                  // tokens of the step
    const buf_t dl = make_buf(a.dl + t * a.E + e0, (left * a.E - e0) * 4);
#pragma unroll
    for (int i = 0; i < ND; ++i) dn[P][i] = load16(dl, doff[i]);
    if constexpr (DWR) {
      const buf_t x = make_buf(a.x + t * a.H + c0, (left * a.H - c0) * 2);
#pragma unroll
      for (int i = 0; i < NX; ++i) xn[P][i] = load16(x, xoff[i]);
    }
  };
  // the residual of a step, loaded where that of an earlier step has been used
  const auto load_res = [&](int buf, int64_t t) {
    const int P = buf % AHEAD;
    if constexpr (DX) {
      const buf_t res = make_buf(a.res ? a.res + t * a.H : nullptr, min(sl.t1 - t, (int64_t)ST) * a.H * 2);
#pragma unroll
      for (int i = 0; i < NO; ++i) rn[P][i] = load16(res, roff[i]);
    }
  };
  load(0, sl.t0);
  load_res(0, sl.t0);
  if constexpr (AHEAD == 2) {
    load(1, sl.t0 + ST);
    load_res(1, sl.t0 + ST);
  }

  // places in dl's buffers: this thread's when it fills them, and this lane's of the two kinds of operand. A step of 32
  // experts is four chunks on, which the exchange of chunks turns into bit 6 of the place and whole 128 bytes.
  constexpr int RI = BT / (EP / 4);              // rows between a thread's loads (a multiple of 8, or one load, or few)
  const auto put_at = [&](int row, int j) { return row * DP + (((j >> 1) ^ swz(row)) << 4) + 8 * (j & 1); };
  const int put0 = put_at((int)threadIdx.x / (EP / 4), (int)threadIdx.x % (EP / 4));
  const int get0 = r * DP + ((g ^ swz(r)) << 4);
  const auto at_step = [](int place, int s) { return (place ^ ((s & 1) << 6)) + (s >> 1) * 128; };
  // a transposed read: row 8 (l / 32) + (l % 16) / 4, columns 16 ((l / 16) % 2) + 4 (l % 4)
  const int tr = 8 * (lane >> 5) + (r >> 2), tc = 16 * (g & 1) + 4 * (lane & 3);
  const int trl = tr * DP + (((tc >> 3) ^ swz(tr)) << 4) + 2 * (tc & 7);
  const int trh = (tr + 4) * DP + (((tc >> 3) ^ swz(tr + 4)) << 4) + 2 * (tc & 7);
  const int wm = wave % WM, wn = wave / WM;
  const int xc = 4 * wn * TN + (tc >> 3);
  const auto x_at = [&](int row) { return row * XP + (((xc & 7) ^ swz(row)) << 4) + (xc >> 3) * 128 + 2 * (tc & 7); };
  const int trx = x_at(tr), trxh = x_at(tr + 4);

  // a step's values from its registers into its buffers, and the loads of a later one into the registers
  const auto stage = [&](int buf, int64_t t) {
    const int P = buf, R = P % AHEAD;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int q = (int)threadIdx.x + BT * i;
      if (ST * EP / 4 < BT && wave >= ST * EP / 4 / 64) break;         // (fewer places than threads)
      const int at = RI % 8 == 0 ? put0 + i * RI * DP : put_at(q / (EP / 4), q % (EP / 4));
      uint2 p[3];
      const int n = loaded(i);
      const auto within = [n](int u, uint32_t word) { return n > u ? __uint_as_float(word) : 0.f; };
      const float4 v = make_float4(__uint_as_float(dn[R][i].x), within(1, dn[R][i].y), within(2, dn[R][i].z),
                                   within(3, dn[R][i].w));
      split3(v.x, v.y, p[0].x, p[1].x, p[2].x);
      split3(v.z, v.w, p[0].y, p[1].y, p[2].y);
#pragma unroll
      for (int s = 0; s < PARTS; ++s) *reinterpret_cast<uint2*>(dl_buf(P, s) + at) = p[s];
    }
    if constexpr (DWR) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        const int q = (int)threadIdx.x + BT * i;
        const int row = q / (NC / 8);
        *reinterpret_cast<uint4*>(x_buf(P) + row * XP + ((q % (NC / 8) ^ swz(row)) << 4)) = xn[R][i];
      }
    }
    load(buf, t + ST * AHEAD);
  };
  stage(0, sl.t0);
  steps<AHEAD, ST>(sl, [&](int buf, int64_t t) {
    const int P = buf, R = P % AHEAD;
    // everyone has written this step's buffers, and is done with the other ones
    barrier_lds_only();
    if constexpr (DWR) {
      const auto pair = [&](const uint8_t* lo, const uint8_t* hi) {
        const i16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_ptr)lo);
        const i16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_ptr)hi);
        return __builtin_bit_cast(uint4, i16x8_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
      };
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint4 xf[TN];
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          const uint8_t* p = x_buf(P) + 16 * k * XP;
          xf[n] = pair(p + (trx ^ (n << 6)), p + (trxh ^ (n << 6)));
        }
        if (k == 0) stage(P ^ 1, t + ST);
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int s = 2; s >= 0; --s) {
            // (WM = 2 wavefronts along the experts take the tiles 0, 1 and 2, 3: the second pair is 128 bytes on)
            const uint8_t* p = dl_buf(P, s) + 16 * k * DP + wm * 128;
            const uint4 df = pair(p + at_step(trl, m), p + at_step(trh, m));
#pragma unroll
            for (int n = 0; n < TN; ++n) acc[m][n] = mfma32(df, xf[n], acc[m][n]);
            if constexpr (LOW) __builtin_amdgcn_sched_barrier(0);      // (fragments for one part at a time)
          }
      }
    }
    if constexpr (DX) {
      f32x4_t o[MT][NT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) o[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (s < nks) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint4 d[3];
#pragma unroll
            for (int p = 0; p < 3; ++p)
              d[p] = *reinterpret_cast<const uint4*>(dl_buf(P, p) + 16 * n * DP + at_step(get0, s));
            if (!DWR && s == 0 && n == NT - 1) stage(P ^ 1, t + ST);
            // part i of one with part j of the other, the small products first
#pragma unroll
            for (int sum = 2; sum >= 0; --sum)
#pragma unroll
              for (int i = sum; i >= 0; --i)
#pragma unroll
                for (int m = 0; m < MT; ++m) o[m][n] = mfma16(w[i][m][s], d[sum - i], o[m][n]);
          }
        }
      }
      // through LDS, so that rows are read and written 256 MT bytes at a time
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<f32x4_t*>(o_buf + (16 * n + r) * OP + 4 * (16 * MT * wave + 4 * MT * g + 4 * m)) = o[m][n];
      barrier_lds_only();
      const buf_t dx = make_buf(a.dx + t * a.H, min(sl.t1 - t, (int64_t)ST) * a.H * 2);
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        const int q = (int)threadIdx.x + BT * i;
        const float4* p = reinterpret_cast<const float4*>(o_buf + min(q / (NC / 8), ST - 1) * OP + 32 * (q % (NC / 8)));
        const float4 x = p[0], y = p[1];
        const uint4 v = rn[R][i];
        const uint4 sum = make_uint4(pack_bf16x2(x.x + bf_lo(v.x), x.y + bf_hi(v.x)),
                                     pack_bf16x2(x.z + bf_lo(v.y), x.w + bf_hi(v.y)),
                                     pack_bf16x2(y.x + bf_lo(v.z), y.y + bf_hi(v.z)),
                                     pack_bf16x2(y.z + bf_lo(v.w), y.w + bf_hi(v.w)));
        store16(dx, roff[i], sum);
      }
      load_res(buf, t + ST * AHEAD);
    }
  });

  if constexpr (DWR) {
    float* out = slices > 1 ? a.part + (int64_t)slice * a.E * a.H : a.dwr;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = e0 + 32 * (wm * TM + m) + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
          const int c = c0 + 32 * (wn * TN + n) + (lane & 31);
          if (e < a.E && c < a.H) out[(int64_t)e * a.H + c] = acc[m][n][i];
        }
  }
}

template <int KS, bool DX, bool DWR, int AHEAD, int MT, int ST>
__global__ __launch_bounds__(64 * NW, 2) void router_grad_kernel(const mok_logits_bwd_args a, const Plan p) {
  using B = Body<KS, DX, DWR, AHEAD, false, MT, ST>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[B::kLds];
  B::run(a, p, (int)blockIdx.x, lds);
}

// dx and dWr in one launch, two workgroups a CU: pw.groups() that form dWr, and R for each of them that form dx (or
// fewer, where H leaves the last one no columns). They take turns by eights, so that each die has both, and what
// eights leave comes last.
template <int KS>
constexpr int kPairMT = KS < 4 ? 2 : 1;
template <int KS>
__global__ __launch_bounds__(64 * NW, 4) void router_grad_pair_kernel(const mok_logits_bwd_args a, const Plan px,
                                                                  const Plan pw) {
  using X = Body<KS, true, false, 1, true, kPairMT<KS>>;
  using W = Body<KS, false, true, 1, true>;
  constexpr int R = W::NC / X::NC;
  __shared__ __attribute__((aligned(16))) uint8_t lds[X::kLds > W::kLds ? X::kLds : W::kLds];
  const int b = (int)blockIdx.x, nx = px.groups(), nw = pw.groups();
  const int rounds = min(nx / (8 * R), nw / 8), rest = b - rounds * 8 * (R + 1), left = nw - 8 * rounds;
  const int turn = b / 8 % (R + 1);
  const bool w = rest < 0 ? turn == 1 : rest < left;
  if (w) W::run(a, pw, rest < 0 ? b / (8 * (R + 1)) * 8 + (b & 7) : 8 * rounds + rest, lds);
  else X::run(a, px, rest < 0 ? (b / (8 * (R + 1)) * R + turn / 2) * 8 + (b & 7) : 8 * R * rounds + rest - left, lds);
}

__global__ __launch_bounds__(256) void router_dwr_join_kernel(const float* __restrict__ part, int slices, int64_t n4,
                                                             float* __restrict__ dwr) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 s = reinterpret_cast<const float4*>(part)[i];
#pragma unroll 8
  for (int k = 1; k < slices; ++k) {
    const float4 v = reinterpret_cast<const float4*>(part)[k * n4 + i];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  reinterpret_cast<float4*>(dwr)[i] = s;
}

// Partial sums against workgroups: `workgroups` of them at most, and about two steps of 32 tokens each at least (200
// experts, 1000 x 4096: 40.5 us, 44.1 with three; 300 x 1024: 29.9, 34.4). The steps are spread evenly over the slices:
// where they do not divide, slices differ by one step, and of so few some have one.
constexpr int kWorkgroups = 256;
int64_t steps_of(int64_t T, int64_t tiles, int workgroups) {
  const int64_t steps = (T + 31) / 32, slices = std::max<int64_t>(1, workgroups / tiles);
  return (steps + slices - 1) / slices;
}
Plan plan_of(int64_t T, int H, int columns, int eblocks, int workgroups) {
  Plan p;
  p.panels = (H + columns - 1) / columns;
  p.eblocks = eblocks;
  const int64_t per = std::max<int64_t>(2, steps_of(T, (int64_t)p.panels * eblocks, workgroups));
  p.slices = (int)std::max<int64_t>(1, ((T + 31) / 32 + per - 1) / per);
  return p;
}
// With much data, and x read for both at once, the one kernel is nearer the memory (64 experts, 8192 x 4096 with a
// residual 60.5 us, as a pair 64.9; 32 experts 49.3, 51.5); with less the pair's shorter ways count (4096 x 4096:
// 34.9, 34.0; 26.6, 25.5; 1037 x 2048: 17.0, 14.3; 13.5, 11.3). From 65 to 128 experts, with two launches in place of
// the one: 8192 x 4096 97 us, as a pair 107; 4096 x 4096 59, 59; 2048 x 4096 40.1, 35.4; 1000 x 4096 29.8, 25.1.
bool paired(int64_t T, int H, int E) { return E <= 128 && T * H <= (int64_t)1 << 24; }
// Of the launch that forms dWr. Of a pair's two kinds of workgroups each has half of the CUs, up to 64 experts while
// that makes slices of six steps at most (64 experts, 1000 x 4096: all 19.8 us, half 18.2; 32 experts, 1037 x 2048:
// 12.4, 11.4; eight steps, 16 experts, 2048 x 4096: 17.2, 18.0; 128 experts, where dx comes in twice as many
// workgroups: 1000 x 4096 29.1, 25.3; 3000 x 2048 33.2, 29.9; 2048 x 4096 40.0, 35.4; 4096 x 4096 62, 59).
Plan dwr_plan(int64_t T, int H, int E) {
  const bool half = paired(T, H, E) && (E > 64 || steps_of(T, (H + 255) / 256, kWorkgroups / 2) <= 6);
  return plan_of(T, H, 256, (E + 127) / 128, half ? kWorkgroups / 2 : kWorkgroups);
}

template <int KS, bool DX, bool DWR, int AHEAD, int MT = 2, int ST = 32>
hipError_t launch(const mok_logits_bwd_args& a, const Plan& p, hipStream_t st) {
  hipLaunchKernelGGL((router_grad_kernel<KS, DX, DWR, AHEAD, MT, ST>), dim3((unsigned)p.groups()), dim3(64 * NW), 0, st,
                     a, p);
  return hipGetLastError();
}

template <int KS>
hipError_t launch_pair(const mok_logits_bwd_args& a, const Plan& pw, hipStream_t st) {
  constexpr int NC = 128 * kPairMT<KS>;
  Plan px = pw;
  px.panels = (a.H + NC - 1) / NC;
  hipLaunchKernelGGL(router_grad_pair_kernel<KS>, dim3((unsigned)(px.groups() + pw.groups())), dim3(64 * NW), 0, st, a,
                     px, pw);
  return hipGetLastError();
}

}  // namespace

size_t mok_logits_bwd_part_bytes(int64_t T, int H, int E) {
  const Plan p = dwr_plan(T, H, E);
  return p.slices > 1 ? (size_t)p.slices * E * H * 4 : 0;
}

hipError_t mok_launch_logits_bwd(const mok_logits_bwd_args& a, hipStream_t st) {
  const Plan p = dwr_plan(a.T, a.H, a.E);
  hipError_t e = hipSuccess;
  // no tokens: empty sums, and nothing that reads Wr, which may be NULL then
  if (a.T == 0) return launch<4, false, true, 2>(a, p, st);
  if (paired(a.T, a.H, a.E)) {
    e = a.E <= 32 ? launch_pair<1>(a, p, st) : a.E <= 64 ? launch_pair<2>(a, p, st) : launch_pair<4>(a, p, st);
  } else if (a.E <= 64) {
    e = a.E <= 32 ? launch<1, true, true, 2>(a, p, st) : launch<2, true, true, 2>(a, p, st);
  } else {
    const Plan px = plan_of(a.T, a.H, a.E <= 256 ? 256 : 128, 1, kWorkgroups);
    e = a.E <= 128   ? launch<4, true, false, 2>(a, px, st)
        : a.E <= 256 ? launch<8, true, false, 1, 2, 16>(a, px, st)
                     : launch<16, true, false, 1, 1, 16>(a, px, st);
    if (e != hipSuccess) return e;
    e = launch<4, false, true, 2>(a, p, st);
  }
  if (e != hipSuccess || p.slices <= 1) return e;
  const int64_t n4 = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(router_dwr_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st, a.part, p.slices, n4,
                     a.dwr);
  return hipGetLastError();
}
