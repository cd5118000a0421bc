// Dense gated feed-forward block in bf16 (a shared expert, which every token
// passes): h = act(x Wg^T) * (x Wu^T), y = h Wd^T (+ residual), and its backward
//
//   dh = dy Wd          da = dh * b * act'(a)     db = dh * act(a)    h = act(a) * b
//   dWd = dy^T h        dWg = da^T x              dWu = db^T x        dx = da Wg + db Wu
//
// Both projections, the gate and the product are one launch; so are dh with the
// gate's backward, and the weight gradients with dx (its two terms one sum over 2I).
// Sums are fp32 in ascending K (split products: fp32 partial sums, added in
// ascending order), so results are bitwise reproducible. Rounded to bf16: y, the
// saved a and b, and the operands of the next product, h, da and db (the matrix
// cores take bf16): each adds at most 2^-8 relative to its element.
#include <utility>

#include "dense_core.h"
#include "dense_launch.h"

using namespace mok;

namespace {

constexpr int kNoSeg = 0x7fffffc0;               // one segment of K (CopyT)

// row tiles that an XCD's tiles in flight span (dense_core.h): about a square block of them
template <int TS>
constexpr int kGroup = TS == 256 ? 4 : 8;

// rows, columns and contracted length of a product, in tiles' terms
struct Shape {
  int M, N, K, batch;                            // batch 2: dWg and dWu, rows of one product each
};
inline Shape shape_of(const mok_ffn_args& a, mok_ffn_op op) {
  switch (op) {
    case FFN_GATEUP: return {a.T, 2 * ((a.I + 31) / 32 * 32), a.H, 1};
    case FFN_DOWN: return {a.T, a.H, a.I, 1};
    case FFN_DH: return {a.T, a.Ip, a.H, 1};
    case FFN_DWD: return {a.H, a.I, a.T, 1};
    case FFN_DWGU: return {a.I, a.H, a.T, 2};
    default: return {a.T, a.H, 2 * a.Ip, 1};
  }
}

// ------------------------------------------------------------------ epilogues
// da, db and h of eight columns (c < I) from dh and the saved a, b
template <int ACT>
MOK_DEV void gate_backward8(const mok_ffn_args& a, int r, int c, const float dh[8], uint4 araw, uint4 braw) {
  float av[8], bv[8], da[8], db[8], h[8];
  unpack_bf16x8(araw, av);
  unpack_bf16x8(braw, bv);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float act, dact;
    gate_act_grad<ACT>(av[u], act, dact);
    h[u] = act * bv[u];
    da[u] = dh[u] * bv[u] * dact;
    db[u] = dh[u] * act;
  }
  bf16_t* d = a.dab + (int64_t)r * 2 * a.Ip + c;
  store_nt(d, pack_bf16x8(da));
  store_nt(d + a.Ip, pack_bf16x8(db));
  store_nt(a.h + (int64_t)r * a.I + c, pack_bf16x8(h));
}

// Eight columns c .. c+7 of output row r from fp32 sums (gate/up: v = a, w = b).
template <int OP, int ACT>
MOK_DEV void finish8(const mok_ffn_args& a, int r, int c, int half, float v[8], const float w[8]) {
  if constexpr (OP == FFN_GATEUP) {
    if (c >= a.I) return;
    float h[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) h[u] = gate_act<ACT>(v[u]) * w[u];
    store_nt(a.h + (int64_t)r * a.I + c, pack_bf16x8(h));
    if (a.ab) {
      bf16_t* p = a.ab + (int64_t)r * 2 * a.I + c;
      store_nt(p, pack_bf16x8(v));
      store_nt(p + a.I, pack_bf16x8(w));
    }
  } else if constexpr (OP == FFN_DH) {
    if (c >= a.Ip) return;
    bf16_t* d = a.dab + (int64_t)r * 2 * a.Ip + c;
    if (c >= a.I) {                              // the pad columns of da and db
      store_nt(d, make_uint4(0, 0, 0, 0));
      store_nt(d + a.Ip, make_uint4(0, 0, 0, 0));
      return;
    }
    const bf16_t* p = a.ab + (int64_t)r * 2 * a.I + c;
    gate_backward8<ACT>(a, r, c, v, *reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + a.I));
  } else if constexpr (OP == FFN_DWD) {
    if (c >= a.I) return;
    store_nt(a.dwd + (int64_t)r * a.I + c, pack_bf16x8(v));
  } else if constexpr (OP == FFN_DWGU) {
    if (c >= a.H) return;
    store_nt((half ? a.dwu : a.dwg) + (int64_t)r * a.H + c, pack_bf16x8(v));
  } else {
    if (c >= a.H) return;
    if constexpr (OP == FFN_DOWN)
      if (a.res) {
        float s[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(a.res + (int64_t)r * a.ldy + c), s);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] += s[u];
      }
    bf16_t* d = OP == FFN_DOWN ? a.y + (int64_t)r * a.ldy : a.dx + (int64_t)r * a.ldx;
    store_nt(d + c, pack_bf16x8(v));
  }
}

// output columns of a tile of N accumulator columns, and the accumulator column
// of output column c (gate/up tiles alternate 32 gate and 32 up columns)
template <int OP, int N>
constexpr int out_cols() { return OP == FFN_GATEUP ? N / 2 : N; }
template <int OP>
MOK_DEV int acc_col(int c) { return OP == FFN_GATEUP ? (c >> 5) * 64 + (c & 31) : c; }

// rows [0, nrows) of fp32 staging at pitch P -> finish8; row0/col0 of the tile
template <int OP, int ACT, int THREADS>
MOK_DEV void finish_rows(const mok_ffn_args& a, const uint8_t* st, int pitch, int nrows, int row0, int col0,
                         int half) {
  constexpr int CH = out_cols<OP, 128>() / 8;
  for (int idx = threadIdx.x; idx < nrows * CH; idx += THREADS) {
    const int r = idx / CH, c = (idx % CH) * 8;
    const uint8_t* p = st + r * pitch + acc_col<OP>(c) * 4;
    float v[8], w[8];
    load_f32<8>(p, v);
    if constexpr (OP == FFN_GATEUP) load_f32<8>(p + 128, w);
    finish8<OP, ACT>(a, row0 + r, col0 + c, half, v, w);
  }
}

// ------------------------------------------------------------------ products
// The copies of 128 rows from m0 of the first operand and 128 columns from n0 (gate/up: 64 of
// gate and 64 of up) of the second. A half of a 256 x 256 tile that lies past the matrix copies
// its last rows or columns instead; those products are not stored.
template <int OP>
MOK_DEV auto copy_a(const mok_ffn_args& a, int m0, int half) {
  if constexpr (OP == FFN_DWD) {
    m0 = min(m0, a.H - 8);
    return CopyT(a.dy + m0, a.dy + m0, kNoSeg, a.T, 2 * a.ldy, a.H - m0);
  } else if constexpr (OP == FFN_DWGU) {
    m0 = min(m0, a.I - 8);
    const bf16_t* da = a.dab + (half ? a.Ip : 0) + m0;
    return CopyT(da, da, kNoSeg, a.T, 4 * (int64_t)a.Ip, a.I - m0);
  } else {
    const int64_t ld = OP == FFN_GATEUP ? a.ldx : OP == FFN_DOWN ? a.I : OP == FFN_DH ? a.ldy : 2 * a.Ip;
    const int K = OP == FFN_DOWN ? a.I : OP == FFN_DX ? 2 * a.Ip : a.H;
    const bf16_t* p = OP == FFN_GATEUP ? a.x : OP == FFN_DOWN ? a.h : OP == FFN_DH ? a.dy : a.dab;
    m0 = min(m0, a.T - 1);
    return CopyK<128, false>(Rows1{p + m0 * ld, 2 * ld, a.T - m0}, 2 * K);
  }
}
template <int OP>
MOK_DEV auto copy_b(const mok_ffn_args& a, int n0) {
  n0 = min(n0, (OP == FFN_DOWN || OP == FFN_DWGU || OP == FFN_DX ? a.H : a.I) - 8);
  if constexpr (OP == FFN_GATEUP) {
    const int64_t o = (int64_t)n0 * a.H;
    return CopyK<128, true>(Rows2{a.wg + o, a.wu + o, 2 * (int64_t)a.H, a.I - n0}, 2 * a.H);
  } else if constexpr (OP == FFN_DOWN) {
    return CopyK<128, false>(Rows1{a.wd + (int64_t)n0 * a.I, 2 * (int64_t)a.I, a.H - n0}, 2 * a.I);
  } else if constexpr (OP == FFN_DH) {
    return CopyT(a.wd + n0, a.wd + n0, kNoSeg, a.H, 2 * (int64_t)a.I, a.I - n0);
  } else if constexpr (OP == FFN_DWD) {
    return CopyT(a.h + n0, a.h + n0, kNoSeg, a.T, 2 * (int64_t)a.I, a.I - n0);
  } else if constexpr (OP == FFN_DWGU) {
    return CopyT(a.x + n0, a.x + n0, kNoSeg, a.T, 2 * a.ldx, a.H - n0);
  } else {
    return CopyT(a.wg + n0, a.wu + n0, a.Ip, a.I, 2 * (int64_t)a.H, a.H - n0);
  }
}

// tile i of the product, counted over its splits along K; split in two or more, to partial
// tiles (split, tile) of fp32 rows at `part`
template <int OP, int ACT, int S>
MOK_DEV void tile128(const mok_ffn_args& a, uint8_t* lds, float* part, int i, int M, int K, int nr, int nc, int batch,
                     int splits) {
  const int tiles = nr * nc * batch, split = splits > 1 ? i / tiles : 0, t = splits > 1 ? i % tiles : i;
  const int half = t / (nr * nc);
  int row, col;
  dense_tile(t - half * nr * nc, nr, nc, kGroup<128>, row, col);
  const int m0 = row * 128, n0 = col * out_cols<OP, 128>();
  const int ns = (K + 63) / 64;
  const int j0 = splits > 1 ? (int)((int64_t)ns * split / splits) : 0;
  const int j1 = splits > 1 ? (int)((int64_t)ns * (split + 1) / splits) : ns;
  Acc<2, 2> acc;
  loop128<S>(lds, copy_a<OP>(a, m0, half), copy_b<OP>(a, n0), j0, j1, acc);
  stage128<S>(lds, acc);
  const int nrows = min(128, M - m0);
  if (splits > 1) {
    float* p = part + ((int64_t)split * tiles + t) * 16384;
    for (int idx = threadIdx.x; idx < nrows * 32; idx += kThreads128<S>)
      reinterpret_cast<float4*>(p)[idx] =
          *reinterpret_cast<const float4*>(lds + (idx >> 5) * kPitch128 + (idx & 31) * 16);
  } else {
    finish_rows<OP, ACT, kThreads128<S>>(a, lds, kPitch128, nrows, m0, n0, half);
  }
}
template <int OP, int ACT, bool SPLIT, int S>
__global__ __launch_bounds__(kThreads128<S>, S == 2 ? 2 : 1) void ffn128_kernel(mok_ffn_args a, int M, int K, int nr,
                                                                                int nc, int batch, int splits) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[lds128<S, 32768>()];
  if constexpr (SPLIT) __builtin_assume(splits > 1);
  const int i = dense_index((int64_t)nr * nc * batch * splits);
  if (i >= 0) tile128<OP, ACT, S>(a, lds, a.part, i, M, K, nr, nc, batch, SPLIT ? splits : 1);
}

// Sums of the partial tiles of TS x TS, and the epilogue: chunk idx of eight output columns of
// tile t. One workgroup takes 256 chunks.
template <int OP, int ACT, int TS>
MOK_DEV void join_tile(const mok_ffn_args& a, const float* part, int t, int idx, int M, int nr, int nc, int batch,
                       int splits) {
  constexpr int CH = out_cols<OP, TS>() / 8;
  const int tiles = nr * nc * batch, half = t / (nr * nc);
  int row, col;
  dense_tile(t - half * nr * nc, nr, nc, kGroup<TS>, row, col);
  const int r = idx / CH, c = (idx % CH) * 8;
  if (r >= min(TS, M - row * TS)) return;
  const float* p = part + (int64_t)t * TS * TS + r * TS + acc_col<OP>(c);
  float v[8], w[8];
  sum_splits(p, (int64_t)tiles * TS * TS, splits, v);
  if constexpr (OP == FFN_GATEUP) sum_splits(p + 32, (int64_t)tiles * TS * TS, splits, w);
  finish8<OP, ACT>(a, row * TS + r, col * out_cols<OP, TS>() + c, half, v, w);
}
template <int OP, int ACT, int TS>
__global__ __launch_bounds__(kThreads) void ffn_join_kernel(mok_ffn_args a, int M, int nr, int nc, int batch,
                                                            int splits) {
  join_tile<OP, ACT, TS>(a, a.part, (int)blockIdx.y, (int)blockIdx.x * kThreads + (int)threadIdx.x, M, nr, nc, batch,
                         splits);
}

// Epilogue of a 256 x 256 tile (the main loop ends in a barrier: LDS is free). VAR: the
// gate's kind, or of the down product 1 = with a residual.
template <int OP, int VAR>
MOK_DEV void finish256(const mok_ffn_args& a, uint8_t* lds, Acc<4, 2>& acc, int nrows, int m0, int n0, int half) {
  if constexpr (OP == FFN_GATEUP) {
    // fragment columns n = 0, 1 are gate and up of the same 32 columns: h in registers, then
    // [h | a] and b through LDS, 128 columns each
    const auto put = [&](int plane, auto&& f) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = f(acc.c[i][0][4 * q + e], acc.c[i][1][4 * q + e]);
          const int c = 32 * pp_col() + 8 * q + 4 * (lane_id() >> 5);
          pp_put4(lds + plane * 65536 + pp_at16<128>(pp_row(i), c), v[0], v[1], v[2], v[3]);
        }
    };
    put(0, [](float g, float u) { return gate_act<VAR>(g) * u; });
    if (a.ab) put(1, [](float g, float) { return g; });
    barrier_lds_only();
    pp_rows16<128>(lds, nrows, [&](int r, int c, uint4 v) {
      if (n0 + c < a.I) store_nt(a.h + (int64_t)(m0 + r) * a.I + n0 + c, v);
    });
    if (!a.ab) return;
    pp_rows16<128>(lds + 65536, nrows, [&](int r, int c, uint4 v) {
      if (n0 + c < a.I) store_nt(a.ab + (int64_t)(m0 + r) * 2 * a.I + n0 + c, v);
    });
    barrier_lds_only();
    put(0, [](float, float u) { return u; });
    barrier_lds_only();
    pp_rows16<128>(lds, nrows, [&](int r, int c, uint4 v) {
      if (n0 + c < a.I) store_nt(a.ab + (int64_t)(m0 + r) * 2 * a.I + a.I + n0 + c, v);
    });
  } else if constexpr (OP == FFN_DH) {
    // dh stays fp32 until the gate's backward has used it: two passes of 128 columns, each
    // with its loads of a, b issued before the staging and its stores after
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint4 av[8], bv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int idx = (int)threadIdx.x + u * kPpThreads, r = idx >> 4, x = (idx & 15) * 8;
        const int c = n0 + 64 * (x >> 5) + 32 * n + (x & 31);
        if (r < nrows && c < a.I) {
          const bf16_t* p = a.ab + (int64_t)(m0 + r) * 2 * a.I + c;
          av[u] = *reinterpret_cast<const uint4*>(p);
          bv[u] = *reinterpret_cast<const uint4*>(p + a.I);
        }
      }
      if (n) barrier_lds_only();
      pp_stage32(lds, acc, n);
      barrier_lds_only();
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int idx = (int)threadIdx.x + u * kPpThreads, r = idx >> 4, x = (idx & 15) * 8;
        const int c = n0 + 64 * (x >> 5) + 32 * n + (x & 31);
        if (r >= nrows || c >= a.Ip) continue;
        float v[8];
        load_f32<8>(lds + r * kPpPitch + x * 4, v);
        if (c < a.I) {
          gate_backward8<VAR>(a, m0 + r, c, v, av[u], bv[u]);
        } else {
          bf16_t* d = a.dab + (int64_t)(m0 + r) * 2 * a.Ip + c;
          store_nt(d, make_uint4(0, 0, 0, 0));
          store_nt(d + a.Ip, make_uint4(0, 0, 0, 0));
        }
      }
    }
  } else {
    if constexpr (OP == FFN_DOWN && VAR == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          pp_add_residual(acc.c[i][n], a.res, a.ldy, m0 + min(pp_row(i), nrows - 1), n0 + pp_col0(n, 0), a.H);
      // a residual that is y itself: every row is read before its stores, which other
      // wavefronts make
      __syncthreads();
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
    bf16_t* d;
    int64_t ld;
    int cols;
    if constexpr (OP == FFN_DOWN) { d = a.y; ld = a.ldy; cols = a.H; }
    else if constexpr (OP == FFN_DX) { d = a.dx; ld = a.ldx; cols = a.H; }
    else if constexpr (OP == FFN_DWD) { d = a.dwd; ld = a.I; cols = a.I; }
    else { d = half ? a.dwu : a.dwg; ld = a.H; cols = a.H; }
    pp_rows16<256>(lds, nrows, [&](int r, int c, uint4 v) {
      if (n0 + c < cols) store_nt(d + (m0 + r) * ld + n0 + c, v);
    });
  }
}

template <int OP, int VAR>
MOK_DEV void tile256(const mok_ffn_args& a, uint8_t* lds, float* part, int i, int M, int K, int nr, int nc, int batch,
                     int splits) {
  const int tiles = nr * nc * batch, split = splits > 1 ? i / tiles : 0, t = splits > 1 ? i % tiles : i;
  const int half = t / (nr * nc);
  int row, col;
  dense_tile(t - half * nr * nc, nr, nc, kGroup<256>, row, col);
  const int ns = (K + 63) / 64;
  const int j0 = splits > 1 ? (int)((int64_t)ns * split / splits) : 0;
  const int j1 = splits > 1 ? (int)((int64_t)ns * (split + 1) / splits) : ns;
  const int m0 = row * 256, n0 = col * out_cols<OP, 256>();
  const int nrows = min(256, M - m0), g = pp_group();
  Acc<4, 2> acc;
  pp_loop(lds, copy_a<OP>(a, m0 + 128 * g, half), copy_b<OP>(a, n0 + out_cols<OP, 128>() * g), j0, j1, acc);
  if (splits > 1) pp_store32(lds, acc, nrows, part + ((int64_t)split * tiles + t) * 65536);
  else finish256<OP, VAR>(a, lds, acc, nrows, m0, n0, half);
}
template <int OP, int VAR, bool SPLIT>
__global__ __launch_bounds__(kPpThreads, 1) void ffn256_kernel(mok_ffn_args a, int M, int K, int nr, int nc,
                                                               int batch, int splits) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kPpLds];
  if constexpr (SPLIT) __builtin_assume(splits > 1);
  const int i = dense_index((int64_t)nr * nc * batch * splits);
  if (i >= 0) tile256<OP, VAR>(a, lds, a.part, i, M, K, nr, nc, batch, SPLIT ? splits : 1);
}

// ------------------------------------------------------------------ dWd, dWg and dWu, dx in one launch
// The three products that follow dh need nothing of each other. Launched one after the
// other, each ends with CUs that wait for its last tiles; here the workgroups of the next
// fill them. The products go in descending time of a workgroup, so that the last ones are the short
// ones (the other way round up to 16% slower), and of two equal ones dWd first, whose operands
// dh's launch has just read and written (dWg and dWu first: 2 to 4% slower). Against one launch
// each, the whole backward from a graph, both in one run: 51 -> 31 us at T = 777 of 1000 x 712,
// 41 -> 23 at 4096 of 256 x 256, 116 -> 99 at 4093 of 2048 x 768, 1163 -> 1093 at 16384 of
// 4096 x 1536, 59 -> 57 at 64 and 2433 -> 2409 at 16384 of 7168 x 2048.
struct GradsPart {
  int op, M, K, nr, nc, batch, splits;
  int n, per;                                    // workgroups, and per XCD
  int joins;                                     // tiles with partial sums
  int64_t part;                                  // theirs, in floats
};
struct GradsPlan {
  int tile, blocks, joins;
  int64_t part;
  GradsPart p[3];
};
template <int TS, int S>
constexpr int grads_lds() { return TS == 256 ? kPpLds : lds128<S, 32768>(); }
template <int TS, int S>
__global__ __launch_bounds__(TS == 256 ? kPpThreads : kThreads128<S>, TS == 128 && S == 2 ? 2 : 1) void
ffn_grads_kernel(mok_ffn_args a, GradsPlan g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[grads_lds<TS, S>()];
  int k = (int)blockIdx.x / kXcds, r = 0;
  if (k >= g.p[0].per) { k -= g.p[0].per; r = 1; }
  if (r == 1 && k >= g.p[1].per) { k -= g.p[1].per; r = 2; }
  const GradsPart q = r == 0 ? g.p[0] : r == 1 ? g.p[1] : g.p[2];
  const int i = ((int)blockIdx.x % kXcds) * q.per + k;
  if (k >= q.per || i >= q.n) return;
  float* part = a.part + q.part;
  if constexpr (TS == 256) {
    if (q.op == FFN_DWGU) tile256<FFN_DWGU, 0>(a, lds, part, i, q.M, q.K, q.nr, q.nc, q.batch, q.splits);
    else if (q.op == FFN_DWD) tile256<FFN_DWD, 0>(a, lds, part, i, q.M, q.K, q.nr, q.nc, 1, q.splits);
    else tile256<FFN_DX, 0>(a, lds, part, i, q.M, q.K, q.nr, q.nc, 1, q.splits);
  } else {
    if (q.op == FFN_DWGU) tile128<FFN_DWGU, 0, S>(a, lds, part, i, q.M, q.K, q.nr, q.nc, q.batch, q.splits);
    else if (q.op == FFN_DWD) tile128<FFN_DWD, 0, S>(a, lds, part, i, q.M, q.K, q.nr, q.nc, 1, q.splits);
    else tile128<FFN_DX, 0, S>(a, lds, part, i, q.M, q.K, q.nr, q.nc, 1, q.splits);
  }
}
template <int TS>
__global__ __launch_bounds__(kThreads) void ffn_grads_join_kernel(mok_ffn_args a, GradsPlan g) {
  int t = (int)blockIdx.y, r = 0;
  if (t >= g.p[0].joins) { t -= g.p[0].joins; r = 1; }
  if (r == 1 && t >= g.p[1].joins) { t -= g.p[1].joins; r = 2; }
  const GradsPart q = r == 0 ? g.p[0] : r == 1 ? g.p[1] : g.p[2];
  const int idx = (int)blockIdx.x * kThreads + (int)threadIdx.x;
  const float* part = a.part + q.part;
  if (q.op == FFN_DWGU) join_tile<FFN_DWGU, 0, TS>(a, part, t, idx, q.M, q.nr, q.nc, q.batch, q.splits);
  else if (q.op == FFN_DWD) join_tile<FFN_DWD, 0, TS>(a, part, t, idx, q.M, q.nr, q.nc, 1, q.splits);
  else join_tile<FFN_DX, 0, TS>(a, part, t, idx, q.M, q.nr, q.nc, 1, q.splits);
}

// ------------------------------------------------------------------ few tokens
// One 16-row slice of the weights against every token (scheme in dense_core.h).
// A slot is 64 elements of K: two 16-byte pieces per lane and row.
template <int OP, int ACT, int NT>
__global__ __launch_bounds__(kFewThreads) void ffn_few_kernel(mok_ffn_args a) {
  static_assert(OP == FFN_GATEUP || OP == FFN_DOWN, "forward products");
  constexpr int U = NT <= 2 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) float red[kFewWaves * NT * 256];
  const int l = lane_id(), lr = l & 15, g = l >> 4;
  const int K = OP == FFN_GATEUP ? a.H : a.I;
  const bf16_t* wp;
  const bf16_t* xp[NT];
  const int c0 = (int)blockIdx.x * (OP == FFN_GATEUP ? 8 : 16);
  if constexpr (OP == FFN_GATEUP) wp = (lr < 8 ? a.wg : a.wu) + (int64_t)(c0 + (lr & 7)) * K;
  else wp = a.wd + (int64_t)min(c0 + lr, a.H - 1) * K;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = min(16 * n + lr, a.T - 1);
    xp[n] = OP == FFN_GATEUP ? a.x + t * a.ldx : a.h + (int64_t)t * a.I;
  }
  const int ns = (K + 63) / 64;
  const int b = ns * wave_id() / kFewWaves, e = ns * (wave_id() + 1) / kFewWaves;
  bf16x8_t wv[2][U][2], xv[2][U][2][NT];
  f4_t acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f4_t{0.f, 0.f, 0.f, 0.f};
  // element of K of piece p of slot j (clamped into the row where it is past K)
  const auto at = [&](int j, int p) { return min(64 * j + 32 * p + 8 * g, K - 8); };
  const auto load = [&](int s, int j) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u >= e) continue;                  // wave-uniform
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        wv[s][u][p] = *reinterpret_cast<const bf16x8_t*>(wp + at(j + u, p));
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[s][u][p][n] = *reinterpret_cast<const bf16x8_t*>(xp[n] + at(j + u, p));
      }
    }
  };
  const auto compute = [&](int s, int j) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u >= e) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // pieces past K: zeros on both sides
        const bool in = 64 * (j + u) + 32 * p + 8 * g < K;
        const bf16x8_t z = {};
        const bf16x8_t w = in ? wv[s][u][p] : z;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, in ? xv[s][u][p][n] : z, acc[n], 0, 0, 0);
      }
    }
  };
  few_pipeline<U>(b, e, load, compute);
  few_put<NT>(red, acc);
  if constexpr (OP == FFN_GATEUP) {
    for (int i = threadIdx.x; i < 8 * a.T; i += kFewThreads) {
      const int c = i & 7, t = i >> 3;
      const float v = few_get<NT>(red, c, t), w = few_get<NT>(red, c + 8, t);
      a.h[(int64_t)t * a.I + c0 + c] = f32_to_bf16(gate_act<ACT>(v) * w);
      if (a.ab) {
        a.ab[(int64_t)t * 2 * a.I + c0 + c] = f32_to_bf16(v);
        a.ab[(int64_t)t * 2 * a.I + a.I + c0 + c] = f32_to_bf16(w);
      }
    }
  } else {
    for (int i = threadIdx.x; i < 16 * a.T; i += kFewThreads) {
      const int c = i & 15, t = i >> 4;
      if (c0 + c >= a.H) continue;
      float v = few_get<NT>(red, c, t);
      if (a.res) v += bf16_to_f32(a.res[t * a.ldy + c0 + c]);
      a.y[t * a.ldy + c0 + c] = f32_to_bf16(v);
    }
  }
}

template <int OP, int ACT>
hipError_t launch_few(const mok_ffn_args& a, hipStream_t st) {
  const dim3 grid(OP == FFN_GATEUP ? a.I / 8 : (a.H + 15) / 16), block(kFewThreads);
  if (a.T <= 16) hipLaunchKernelGGL((ffn_few_kernel<OP, ACT, 1>), grid, block, 0, st, a);
  else if (a.T <= 32) hipLaunchKernelGGL((ffn_few_kernel<OP, ACT, 2>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((ffn_few_kernel<OP, ACT, 4>), grid, block, 0, st, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ host
struct Plan {
  Shape s;
  int tile, nr, nc, splits;                      // tile 0: few tokens
};

// (slots of 64)
constexpr dense_cost kCost = {13.0f, 2.11f, 2.2f, 1.62f, 0.36f, 3.5f, 2.65e6f};

Plan plan_of(const mok_ffn_args& a, mok_ffn_op op) {
  Plan p;
  p.s = shape_of(a, op);
  const float t = dense_plan(p.s.M, p.s.N, p.s.batch, (p.s.K + 63) / 64, kCost, &p.tile, &p.splits);
  if (a.T <= kFewRows && (op == FFN_GATEUP || op == FFN_DOWN) && few_time(a.T, p.s.N, p.s.K) < t) {
    p.tile = p.nr = p.nc = 0;
    p.splits = 1;
    return p;
  }
  p.nr = (p.s.M + p.tile - 1) / p.tile;
  p.nc = (p.s.N + p.tile - 1) / p.tile;
  return p;
}

template <int OP, int ACT>
hipError_t launch(const mok_ffn_args& a, const Plan& p, hipStream_t st) {
  if constexpr (OP == FFN_GATEUP || OP == FFN_DOWN)
    if (p.tile == 0) return a.T > 0 ? launch_few<OP, ACT>(a, st) : hipSuccess;
  const int64_t tiles = (int64_t)p.nr * p.nc * p.s.batch;
  if (tiles == 0) return hipSuccess;
  const dim3 grid(dense_grid(tiles * p.splits)), block(p.tile == 256 || tiles * p.splits <= 256 ? 512 : 256);
  const int nr = p.nr, nc = p.nc, nb = p.s.batch;
  if (p.splits > 1) {
    if (p.tile == 256)
      hipLaunchKernelGGL((ffn256_kernel<OP, 0, true>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, p.splits);
    else if (tiles * p.splits <= 256)
      hipLaunchKernelGGL((ffn128_kernel<OP, 0, true, 4>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, p.splits);
    else
      hipLaunchKernelGGL((ffn128_kernel<OP, 0, true, 2>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, p.splits);
    const int ch = p.tile * (OP == FFN_GATEUP ? p.tile / 2 : p.tile) / 8;
    const dim3 jgrid((ch + kThreads - 1) / kThreads, (unsigned)tiles);
    if (p.tile == 256)
      hipLaunchKernelGGL((ffn_join_kernel<OP, ACT, 256>), jgrid, dim3(kThreads), 0, st, a, p.s.M, nr, nc, nb, p.splits);
    else
      hipLaunchKernelGGL((ffn_join_kernel<OP, ACT, 128>), jgrid, dim3(kThreads), 0, st, a, p.s.M, nr, nc, nb, p.splits);
  } else if (p.tile == 256) {
    if (OP == FFN_DOWN && a.res)
      hipLaunchKernelGGL((ffn256_kernel<OP, OP == FFN_DOWN ? 1 : ACT, false>), grid, block, 0, st, a, p.s.M, p.s.K, nr,
                         nc, nb, 1);
    else
      hipLaunchKernelGGL((ffn256_kernel<OP, ACT, false>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, 1);
  } else if (tiles <= 256) {
    hipLaunchKernelGGL((ffn128_kernel<OP, ACT, false, 4>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, 1);
  } else {
    hipLaunchKernelGGL((ffn128_kernel<OP, ACT, false, 2>), grid, block, 0, st, a, p.s.M, p.s.K, nr, nc, nb, 1);
  }
  return hipGetLastError();
}

// Tile and splits of the three together, by the constants of dense_plan (weights that order the
// choices, not times): for each tile and
// each longest chunk of K (in slots) the time of all workgroups over the CUs, the half of a
// shortest one by which the CUs end apart, and the partial sums.
GradsPlan grads_plan(const mok_ffn_args& a) {
  constexpr mok_ffn_op kOps[3] = {FFN_DWD, FFN_DWGU, FFN_DX};
  constexpr int kChunks[] = {1 << 30, 192, 128, 96, 64, 48, 32, 24, 16, 12, 8, 6, 4};
  Shape sh[3];
  float read = 0.f;
  for (int i = 0; i < 3; ++i) {
    sh[i] = shape_of(a, kOps[i]);
    read += (float)(sh[i].M + (int64_t)sh[i].N * sh[i].batch) * ((sh[i].K + 63) / 64) * 128 / 4.6e6f;
  }
  GradsPlan best;
  float least = 0.f, took[3] = {0.f, 0.f, 0.f};
  best.tile = 0;
  for (int ts = 256; ts >= 128; ts -= 128)
    for (int chunk : kChunks) {
      GradsPlan g;
      float d[3], sum = 0.f, join = 0.f, longest = 0.f, shortest = 0.f;
      int64_t count = 0;
      g.tile = ts;
      g.joins = 0;
      g.part = 0;
      for (int i = 0; i < 3; ++i) {
        GradsPart& q = g.p[i];
        const int slots = (sh[i].K + 63) / 64;
        q.op = kOps[i];
        q.M = sh[i].M; q.K = sh[i].K; q.batch = sh[i].batch;
        q.nr = (int)(((int64_t)q.M + ts - 1) / ts);
        q.nc = (sh[i].N + ts - 1) / ts;
        q.splits = chunk >= slots ? 1 : (slots + chunk - 1) / chunk;
        if (q.splits > slots / 4) q.splits = slots / 4 > 1 ? slots / 4 : 1;
        const int64_t n = (int64_t)q.nr * q.nc * q.batch * q.splits;   // (may pass 32 bits where it is dropped below)
        q.n = (int)n;
        q.per = (int)((n + kXcds - 1) / kXcds);
        q.joins = q.splits > 1 ? q.nr * q.nc * q.batch : 0;
        q.part = g.part;
        g.joins += q.joins;
        if (q.joins) g.part += n * ts * ts;
        if (q.joins) join += (float)q.splits * q.M * sh[i].N * q.batch * 8 / kCost.rate;
        count += n;
      }
      if (g.joins && count > 1024) continue;     // partial tiles take at most 1024 * 256 KiB
      const bool alone = ts == 256 || count <= 256;
      for (int i = 0; i < 3; ++i) {
        const GradsPart& q = g.p[i];
        const int per = ((q.K + 63) / 64 + q.splits - 1) / q.splits;
        d[i] = ts == 256 ? kCost.fix256 + per * kCost.slot256
                         : kCost.fix128 + per * kCost.slot128 * (alone ? kCost.alone : 1.f);
        if (q.n == 0) continue;
        sum += q.n * d[i];
        if (d[i] > longest) longest = d[i];
        if (shortest == 0.f || d[i] < shortest) shortest = d[i];
      }
      const int cap = alone ? 256 : 512;
      float t = count <= cap ? longest : sum / cap + 0.5f * shortest;
      if (t < longest) t = longest;
      if (t < read) t = read;
      if (g.joins) t += kCost.join + join;
      if (best.tile == 0 || t < least) {
        best = g;
        least = t;
        for (int i = 0; i < 3; ++i) took[i] = d[i];
      }
    }
  for (int i = 0; i < 2; ++i)                    // longest first
    for (int j = 0; j < 2 - i; ++j)
      if (took[j] < took[j + 1]) {
        std::swap(took[j], took[j + 1]);
        std::swap(best.p[j], best.p[j + 1]);
      }
  best.blocks = 0;
  for (const GradsPart& q : best.p) best.blocks += q.per * kXcds;
  return best;
}

}  // namespace

size_t mok_ffn_part_bytes(const mok_ffn_args& a, mok_ffn_op op) {
  const Plan p = plan_of(a, op);
  return p.splits > 1 ? (size_t)p.splits * p.nr * p.nc * p.s.batch * p.tile * p.tile * 4 : 0;
}

hipError_t mok_launch_ffn(const mok_ffn_args& a, mok_ffn_op op, int act, hipStream_t st) {
  const Plan p = plan_of(a, op);
  switch (op) {
    case FFN_GATEUP: return act == 0 ? launch<FFN_GATEUP, 0>(a, p, st) : launch<FFN_GATEUP, 1>(a, p, st);
    case FFN_DOWN: return launch<FFN_DOWN, 0>(a, p, st);
    case FFN_DH: return act == 0 ? launch<FFN_DH, 0>(a, p, st) : launch<FFN_DH, 1>(a, p, st);
    default: return hipErrorInvalidValue;
  }
}

size_t mok_ffn_grads_part_bytes(const mok_ffn_args& a) { return (size_t)grads_plan(a).part * 4; }

hipError_t mok_launch_ffn_grads(const mok_ffn_args& a, hipStream_t st) {
  const GradsPlan g = grads_plan(a);
  const int count = g.p[0].n + g.p[1].n + g.p[2].n;
  const dim3 grid((unsigned)g.blocks);
  if (g.tile == 256)
    hipLaunchKernelGGL((ffn_grads_kernel<256, 0>), grid, dim3(kPpThreads), 0, st, a, g);
  else if (count <= 256)
    hipLaunchKernelGGL((ffn_grads_kernel<128, 4>), grid, dim3(kThreads128<4>), 0, st, a, g);
  else
    hipLaunchKernelGGL((ffn_grads_kernel<128, 2>), grid, dim3(kThreads128<2>), 0, st, a, g);
  if (g.joins) {
    const dim3 jgrid((unsigned)(g.tile * g.tile / 8 / kThreads), (unsigned)g.joins);
    if (g.tile == 256) hipLaunchKernelGGL((ffn_grads_join_kernel<256>), jgrid, dim3(kThreads), 0, st, a, g);
    else hipLaunchKernelGGL((ffn_grads_join_kernel<128>), jgrid, dim3(kThreads), 0, st, a, g);
  }
  return hipGetLastError();
}
