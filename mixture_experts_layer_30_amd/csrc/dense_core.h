// Tile machinery of the dense products (k_ffn.hip, k_mx.hip): operand copies
// for matrices that no schedule gathers, with tails in K, main loops of 128 x 128
// and 256 x 256 tiles, products of few rows, the choice among them, and the gates.
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
// All copies are buffer loads into LDS: a descriptor in scalar registers (base,
// bytes), one 32-bit offset per lane and a scalar offset per copy. What lies past
// the descriptor's bytes reads as zero, which covers rows past the last one and
// k-rows past K without a branch. Measured on gfx950 with four wavefronts that
// copy the panels of 256 x 256 tiles and four that multiply, nothing else and no
// barrier between them: copies alone 42 us, products alone 37 us, both 52 us; with
// global_load_lds and its 64-bit address per lane 43, 41 and 82 us: those
// copies and the matrix instructions ran one after the other.
typedef i32x4_t srd_t;
MOK_DEV int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
MOK_DEV srd_t make_srd(const void* p, int64_t bytes) {         // (0 <= bytes < 2^31)
  const uint64_t u = (uint64_t)p;
  return srd_t{uni((int)u), uni((int)(u >> 32) & 0xFFFF), uni((int)bytes), 0x00020000};
}
// Bounds: a lane's offset alone has to be past the descriptor's bytes where nothing
// may be read (the scalar offset, only ever a step along K inside a row, does not
// move the bound), and offsets stay below 2^31: row pitches are at most 2^23 bytes.
constexpr int kNowhere = 0x7ffffff0;             // past every descriptor's bytes
// (the five wait states cover a descriptor or offset written by v_readfirstlane
// right before, which the compiler does not see; m0 needs one of them)
MOK_DEV void buf16_to_lds(srd_t srd, int off, int soff, uint32_t lds) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %2, %3 offen lds" ::"v"(off), "{m0}"(lds), "s"(srd), "s"(soff)
               : "memory");
}
MOK_DEV void buf4_to_lds(srd_t srd, int off, int soff, uint32_t lds) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %2, %3 offen lds" ::"v"(off), "{m0}"(lds), "s"(srd), "s"(soff)
               : "memory");
}
MOK_DEV int copy_wave() { return wave_id() & 3; }  // four wavefronts share an operand's copies

// Rows of a K-contiguous operand: row r at base + r * ld bytes; or, with two
// bases, 32-row groups alternating between them (gate and up rows of the same
// columns side by side, as in gemm_core.h).
struct Rows1 {
  static constexpr bool kTwo = false;
  const void* p;
  int64_t ld;
  int n;                   // rows (>= 1)
};
struct Rows2 {
  static constexpr bool kTwo = true;
  const void* p;
  const void* p2;
  int64_t ld;
  int n;                   // rows of each (>= 1)
};

// K-contiguous operand of 128 rows, RB bytes of K per row and slot; bytes past
// kbytes read as zero, on both operands, so that nothing stored behind a row
// enters a product.
template <int RB, bool TWO>
struct CopyK {
  static_assert(RB == 64 || RB == 128, "bytes of K per row and slot");
  static constexpr int kDma = 128 * RB / 4096;   // 1 KiB windows per wavefront
  srd_t srd, srd2;
  int off, step, lcb, kbytes;
  template <class Rows>
  MOK_DEV CopyK(const Rows& r, int64_t kbytes_) : kbytes((int)kbytes_) {
    static_assert(Rows::kTwo == TWO, "row source");
    const int w = copy_wave(), l = lane_id();
    const int64_t bytes = (int64_t)(min(r.n, 128) - 1) * r.ld + kbytes_;
    int row, lc;
    if constexpr (RB == 128) {                   // copy q: rows 32 q .. +31
      row = swap03(8 * w + (l >> 3));
      lc = (l & 7) ^ (row & 7);
    } else {                                     // copy q: rows 64 q + 16 w .. +15
      row = 2 * swap02(8 * w + (l >> 3)) + ((l >> 2) & 1);
      lc = (l & 3) ^ ((row >> 1) & 3);
    }
    lcb = lc * 16;
    srd = make_srd(r.p, bytes);
    srd2 = srd;
    if constexpr (TWO) {
      srd2 = make_srd(r.p2, bytes);
      if (RB == 64 && (w & 2)) srd = srd2;       // wavefronts 2, 3 copy up rows
      row &= 31;
    }
    off = row * (int)r.ld + lcb;
    step = uni((RB == 64 && !TWO ? 64 : 32) * (int)r.ld);
  }
  MOK_DEV void dma(int j, uint32_t slot) const {
    const uint32_t mb = slot + copy_wave() * 1024;
    const bool past = (j + 1) * RB > kbytes && j * RB + lcb >= kbytes;
#pragma unroll
    for (int q = 0; q < kDma; ++q) {
      const bool alt = TWO && RB == 128;         // groups q = 0, 2 gate, 1, 3 up
      const int o = off + (alt ? q >> 1 : q) * step;
      buf16_to_lds(alt && (q & 1) ? srd2 : srd, past ? kNowhere : o, uni(j * RB), mb + q * 4096);
    }
  }
  // bf16 fragment of 32 rows from r0: 16-wide K step kk of half h
  MOK_DEV static bf16x8_t frag(const uint8_t* t, int r0, int h, int kk) {
    const int l = lane_id();
    return *reinterpret_cast<const bf16x8_t*>(t + lds_at(r0 + (l & 31), 4 * h + 2 * kk + (l >> 5)));
  }
};

// K-outer bf16 operand of 128 columns: element (k, n) at src0 + k*ld + 2n for the
// first segment of kseg k-rows (a multiple of 64) and at src1 + (k - kseg)*ld + 2n
// for the second; k-rows past kvalid in either segment read as zero. Columns past
// ncols read what follows them and land in output that is not stored.
struct CopyT {
  static constexpr int kDma = 4;
  const uint8_t* src0;
  const uint8_t* src1;
  int kseg, kvalid, ncols, off, ld;
  MOK_DEV CopyT(const void* s0, const void* s1, int kseg_, int kvalid_, int64_t ld_, int ncols_)
      : src0((const uint8_t*)s0), src1((const uint8_t*)s1), kseg(kseg_), kvalid(kvalid_), ncols(ncols_),
        ld((int)ld_) {
    const int l = lane_id(), kl = 4 * copy_wave() + (l >> 4);
    off = kl * ld + (((l & 15) ^ ((kl & 3) << 2)) << 4);
  }
  MOK_DEV void dma(int j, uint32_t slot) const {
    const bool second = j * 64 >= kseg;
    const int k0 = second ? j * 64 - kseg : j * 64, kr = min(kvalid - k0, 64);
    const srd_t srd = make_srd((second ? src1 : src0) + (int64_t)k0 * ld,
                               max((int64_t)(kr - 1) * ld + 2 * min(ncols, 128), (int64_t)0));
    const uint32_t mb = slot + copy_wave() * 1024;
#pragma unroll
    for (int q = 0; q < kDma; ++q) buf16_to_lds(srd, off + q * 16 * ld, 0, mb + q * 4096);
  }
  MOK_DEV static bf16x8_t frag(const uint8_t* t, int r0, int h, int kk) {
    const int l = lane_id(), g = l >> 4, L = l & 15;
    const int n = r0 + 16 * (g & 1) + 4 * (L & 3);
    const int k = 32 * h + 16 * kk + 8 * (g >> 1) + (L >> 2);
    typedef __attribute__((address_space(3))) v4i16_t* lds_v4_ptr;
    const auto at = [&](int kk_) {
      return (lds_v4_ptr)(t + kk_ * 256 + (((n >> 3) ^ ((kk_ & 3) << 2)) << 4) + ((2 * n) & 15));
    };
    const v4i16_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k));
    const v4i16_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(k + 4));
    typedef __attribute__((ext_vector_type(8))) short v8i16_t;
    const v8i16_t v = v8i16_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  }
};

// ------------------------------------------------------------------ 128 x 128 tile
// Four wavefronts of 64 x 64 (2 x 2 fragments of 32 x 32), and two ways to fill a CU:
//  S = 2: two slots of LDS and two workgroups a CU, each multiplying while the other
//         waits; for more than 256 tiles (with S = 4 those take 10% longer, mean of 200).
//  S = 4: one workgroup a CU, with four more wavefronts that only copy, three slots
//         ahead. A wavefront that copies waits for the address unit, and the multiplying
//         ones then do not: a bf16 slot takes 0.58 us, with four wavefronts doing both
//         and two slots 0.83 us, and with four slots 0.95 us.
using G128 = Geo<128, 128, 2, 2>;
constexpr int kPitch128 = 128 * 4 + 16;          // fp32 staging of the tile
constexpr int kLds128 = 128 * kPitch128;         // 67584 B, above two slots' 65536 B
template <int S>
constexpr int kThreads128 = S == 2 ? 256 : 512;
template <int S, int SLOT>
constexpr int lds128() { return S * SLOT > kLds128 ? S * SLOT : kLds128; }

// slots [j0, j1): issue(j, buffer) starts a wavefront's kD copies of slot j, compute(buffer)
// multiplies (S = 4: wavefronts 0 to 3)
template <int S, int kD, class Issue, class Compute>
MOK_DEV void ring128(int j0, int j1, Issue&& issue, Compute&& compute) {
  if constexpr (S == 2) {
    if (j0 < j1) issue(j0, 0);
    if (j0 + 1 < j1) issue(j0 + 1, 1);
    for (int j = j0; j < j1; ++j) {
      const int s = (j - j0) & 1;
      if (j + 1 < j1) wait_vm_lds<kD>();
      else wait_vm_lds<0>();
      barrier_lds();
      compute(s);
      barrier_lds_only();
      if (j + 2 < j1) issue(j + 2, s);
    }
  } else if (wave_id() >= 4) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (j0 + k < j1) issue(j0 + k, k);
    for (int j = j0; j < j1; ++j) {
      // slot j has arrived when at most the two slots after it are outstanding; behind the
      // barrier everyone is done with slot j - 1, whose buffer slot j + 3 takes
      if (j + 2 < j1) wait_vm_lds<2 * kD>();
      else wait_vm_lds<0>();
      barrier_lds();
      if (j + 3 < j1) issue(j + 3, (j - j0 + 3) & 3);
    }
    barrier_lds();
  } else {
    for (int j = j0; j < j1; ++j) {
      barrier_lds_only();                        // (with the reads of slot j - 1 complete)
      compute((j - j0) & 3);
    }
    barrier_lds_only();
  }
}

// bf16 product over slots [j0, j1)
template <int S, class LA, class LB>
MOK_DEV void loop128(uint8_t* lds, const LA& la, const LB& lb, int j0, int j1, Acc<2, 2>& acc) {
  constexpr int kSlot = 32768, kB = 16384;
  const uint32_t base = lds_addr(lds);
  acc.zero();
  ring128<S, LA::kDma + LB::kDma>(
      j0, j1,
      [&](int j, int s) {
        la.dma(j, base + s * kSlot);
        lb.dma(j, base + s * kSlot + kB);
      },
      [&](int s) {
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
      });
}

// stage the fp32 tile in LDS (the slots are free: every loop ends in a barrier)
template <int S>
MOK_DEV void stage128(uint8_t* lds, const Acc<2, 2>& acc) {
  if (S == 2 || wave_id() < 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          *reinterpret_cast<float*>(lds + G128::row(i, q) * kPitch128 + G128::col(n) * 4) = acc.c[i][n][q];
  }
  barrier_lds_only();
}

// ------------------------------------------------------------------ 256 x 256 tile
// Eight wavefronts in two groups of four, one of each group on every SIMD, that multiply in
// turns (a published scheme, known as ping-pong). Group g owns tile rows 128 g .. +127, its
// wavefront c columns 64 c .. +63 (4 x 2 fragments, 128 accumulators a lane; the products are
// formed transposed, so that a lane holds four adjacent columns of a row: element 4 q + e of
// fragment (i, n) is row 32 i + l % 32, column 32 n + 8 q + 4 (l / 32) + e). The groups run half a step apart: in each
// interval between two workgroup barriers one group reads fragments from LDS and
// issues copies while the other multiplies, so a copy that waits for the address
// unit or for the L1 never holds up a matrix instruction. (One wavefront per
// SIMD that does both in turn keeps the matrix cores half busy: the copies of
// a tile come in at 17-19 bytes per clock and CU, where the same copies alone
// reach 43-45.)
//
// A slot is 64 bf16 of K; a half operand (128 rows or columns of it) takes 16 KiB.
// Group g copies half g of both operands: of B into two buffers, of A, which only
// group g reads, into three.
//
//   interval  group 0                                   group 1
//   4s        read steps 0, 1 of s; copy B of s+1       multiply steps 2, 3 of s-1
//   4s+1      multiply                                  read steps 0, 1 of s; copy B of s+1
//   4s+2      read steps 2, 3; copy A of s+2            multiply
//   4s+3      multiply; wait for its B of s+1           read steps 2, 3; copy A of s+2;
//                                                       wait for its B of s+1
//
// with a workgroup barrier at the end of each. Every interval has a quarter of the
// copies (at the matrix cores' full rate 32 bytes per clock and CU). Both waits lie
// before the barrier that opens slot s+1; B has two or three intervals to arrive, A more
// than a slot, and no time goes into the waits. The last reads of slot s are complete
// before the barrier of 4s+3, B of s+2 is written over them from 4s+4 on, A of s+3 from
// 4s+6 on. (Copies between the matrix instructions of the multiplying group were 13 to
// 40% slower, all of B in interval 4s and two slots of each operand 5% each.) A down
// product of 4096 x 4096 x 8192 takes 203 us (1352 TFLOP/s; the library's 200 us); the same
// matrix instructions alone sustain 1801 TFLOP/s on random data, 2352 on constant data.
constexpr int kPpThreads = 512;
constexpr int kPpHalf = 16384;
constexpr int kPpLds = 10 * kPpHalf;             // 160 KiB: 3 + 3 half slots of A, 2 + 2 of B
MOK_DEV int pp_group() { return wave_id() >> 2; }
MOK_DEV int pp_col() { return wave_id() & 3; }

// The matrix instructions touch no memory, and the compiler would move them past the
// barriers into the next interval: these fix their operands and results in place.
template <class T>
MOK_DEV void pin(T& v) { asm volatile("" : "+v"(v)); }
MOK_DEV void pin_acc(Acc<4, 2>& acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n) pin(acc.c[i][n]);
}

// all copies but the last N have arrived (with `more`; without, all have)
template <int N>
MOK_DEV void pp_wait(bool more) {
  if (more) wait_vm_lds<N>();
  else wait_vm_lds<0>();
}

// slots [j0, ns); la, lb: this wavefront's group's halves
template <class LA, class LB>
MOK_DEV void pp_loop(uint8_t* lds, const LA& la, const LB& lb, int j0, int ns, Acc<4, 2>& acc) {
  static_assert(LA::kDma == 4 && LB::kDma == 4, "four copies per half and wavefront");
  const int grp = pp_group(), c = pp_col();
  const uint32_t base = lds_addr(lds), oa = grp * 3 * kPpHalf, ob = 6 * kPpHalf;
  acc.zero();
  if (ns <= j0) return;
  lb.dma(j0, base + ob + grp * kPpHalf);
  la.dma(j0, base + oa);
  if (ns > j0 + 1) {
    la.dma(j0 + 1, base + oa + kPpHalf);
    wait_vm_lds<4>();
  } else {
    wait_vm_lds<0>();
  }
  barrier_lds();
  if (grp) barrier_lds();
  bf16x8_t a[2][4], b[2][2];
  const auto read = [&](const uint8_t* ta, const uint8_t* tb, int h) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int n = 0; n < 2; ++n) b[kk][n] = LB::frag(tb, 64 * (c & 1) + 32 * n, h, kk);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[kk][i] = LA::frag(ta, 32 * i, h, kk);
    }
  };
  const auto multiply = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    pin(b[0][0]);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          acc.c[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[kk][n], a[kk][i], acc.c[i][n], 0, 0, 0);
    pin_acc(acc);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  uint32_t s0 = 0, s2 = 2 * kPpHalf;             // A's buffer of s, and of s + 2
  for (int s = j0; s < ns; ++s) {
    const int par = (s - j0) & 1;
    const uint8_t* ta = lds + oa + s0;
    const uint8_t* tb = lds + ob + (par * 2 + (c >> 1)) * kPpHalf;
    const bool more = s + 2 < ns;
    read(ta, tb, 0);
    if (s + 1 < ns) lb.dma(s + 1, base + ob + ((par ^ 1) * 2 + grp) * kPpHalf);
    barrier_lds_only();
    multiply();
    barrier_lds();
    read(ta, tb, 1);
    if (more) la.dma(s + 2, base + oa + s2);
    if (grp) pp_wait<4>(more);
    barrier_lds_only();
    multiply();
    if (!grp) pp_wait<4>(more);
    barrier_lds();
    s0 = s0 == 2 * kPpHalf ? 0 : s0 + kPpHalf;
    s2 = s2 == 2 * kPpHalf ? 0 : s2 + kPpHalf;
  }
  if (!grp) barrier_lds();
}

// Row of the tile of this lane's fragments i, and its first column of (n, q)
MOK_DEV int pp_row(int i) { return 128 * pp_group() + 32 * i + (lane_id() & 31); }
MOK_DEV int pp_col0(int n, int q) { return 64 * pp_col() + 32 * n + 8 * q + 4 * (lane_id() >> 5); }

// bf16 staging of 256 rows x W columns: 16-byte chunk c of row r at c ^ (r & 15) (the 32
// rows of a store instruction spread over all banks), 8 bytes a lane in, 16 out
template <int W>
MOK_DEV int pp_at16(int r, int c) { return r * 2 * W + (((c >> 3) ^ (r & 15)) << 4) + ((c & 7) << 1); }
MOK_DEV void pp_put4(uint8_t* p, float x, float y, float z, float w) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
}
// rows [0, nrows) of the staging, chunk by chunk: put(row, column, value) with eight columns
template <int W, class Put>
MOK_DEV void pp_rows16(const uint8_t* lds, int nrows, Put&& put) {
  constexpr int CH = W / 8;
#pragma unroll 4
  for (int idx = threadIdx.x; idx < 256 * CH; idx += kPpThreads) {
    const int r = idx / CH, c = (idx % CH) * 8;
    if (r < nrows) put(r, c, *reinterpret_cast<const uint4*>(lds + pp_at16<W>(r, c)));
  }
}
// c += the residual's row r at this lane's columns of a fragment from column c0 on (8 q + 0 .. 3;
// N a multiple of 8). Columns past N take others instead, and are not stored.
MOK_DEV void pp_add_residual(f32x16_t& c, const bf16_t* res, int64_t ld, int r, int c0, int N) {
  uint2 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint2*>(res + r * ld + min(c0 + 8 * q, N - 4));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    c[4 * q] += __uint_as_float(v[q].x << 16);
    c[4 * q + 1] += __uint_as_float(v[q].x & 0xFFFF0000u);
    c[4 * q + 2] += __uint_as_float(v[q].y << 16);
    c[4 * q + 3] += __uint_as_float(v[q].y & 0xFFFF0000u);
  }
  __builtin_amdgcn_sched_barrier(0);             // (all fragments' loads at once spill)
}
// fp32 staging of fragment columns n: 256 rows x 128 columns, column 32 k + x of it being
// tile column 64 k + 32 n + x
constexpr int kPpPitch = 128 * 4 + 16;
MOK_DEV void pp_stage32(uint8_t* lds, const Acc<4, 2>& acc, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(lds + pp_row(i) * kPpPitch + (32 * pp_col() + 8 * q + 4 * (lane_id() >> 5)) * 4) =
          make_float4(acc.c[i][n][4 * q], acc.c[i][n][4 * q + 1], acc.c[i][n][4 * q + 2], acc.c[i][n][4 * q + 3]);
}

// the tile as fp32 rows of 256 columns at p (rows [0, nrows)), for products split along K
MOK_DEV void pp_store32(uint8_t* lds, const Acc<4, 2>& acc, int nrows, float* p) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (n) barrier_lds_only();
    pp_stage32(lds, acc, n);
    barrier_lds_only();
#pragma unroll 4
    for (int idx = threadIdx.x; idx < 256 * 32; idx += kPpThreads) {
      const int r = idx >> 5, x = (idx & 31) * 4;
      if (r < nrows)
        *reinterpret_cast<float4*>(p + r * 256 + 64 * (x >> 5) + 32 * n + (x & 31)) =
            *reinterpret_cast<const float4*>(lds + r * kPpPitch + x * 4);
    }
  }
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

// v = the sum over the splits, in ascending order, of eight fp32 values at p, each split's
// `step` floats after the one before (four splits' loads in flight)
MOK_DEV void sum_splits(const float* p, int64_t step, int splits, float v[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = 0.f;
  int s = 0;
  for (; s + 4 <= splits; s += 4) {
    float q[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) load_f32<8>(p + (s + k) * step, q[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] += q[k][u];
  }
  for (; s < splits; ++s) {
    float q[8];
    load_f32<8>(p + s * step, q);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] += q[u];
  }
}

// ------------------------------------------------------------------ few rows
// Products with few rows of x (at most kFewRows) read the weights once and are bound by
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

// Tile and split of a product of M x N (x batch) over `slots` slots of K: the least
// estimated time. A pass of 256 workgroups of 256 x 256 tiles (one a CU), or of 512 of
// 128 x 128 (two a CU), takes a fixed part (launch, first copies, epilogue) and a part
// per slot, of which a 128 x 128 tile with a CU to itself needs the share `alone`; all
// slots take at least as long as reading the operands; partial sums add a launch and the
// traffic of writing and reading them. The constants are those that make the choice, not
// the times, come out best over 280 shapes of 33 to 8192 rows, each timed with both tiles
// and up to 8 splits: no single one of them is the time of its part (a lone MXFP4
// tile took about 5 us and 0.5 to 0.6 a slot; here 8.7 and 0.39). There the choice
// was within 1% of the fastest in the mean and 18% at worst; on 200 random products that were
// not fitted (bf16 120, MXFP8 and MXFP4 times MXFP4 40 each) within 2% and 24%.
struct dense_cost {
  float fix256, slot256, fix128, slot128, alone; // (us)
  float join, rate;                              // (us, bytes per us)
};
inline float dense_plan(int64_t M, int64_t N, int batch, int64_t slots, const dense_cost& c, int* tile, int* splits) {
  const float read = (float)(M + N * batch) * slots * 128 / 4.6e6f;   // the operands once, 4.6 TB/s
  float best = 0.f;
  *tile = 128;
  *splits = 1;
  for (int ts = 256; ts >= 128; ts -= 128) {
    const int64_t n = ((M + ts - 1) / ts) * ((N + ts - 1) / ts) * batch, fill = ts == 256 ? 256 : 512;
    for (int64_t s = 1; s == 1 || (n * s <= fill && slots >= 4 * s); ++s) {
      const int64_t passes = (n * s + fill - 1) / fill, per = (slots + s - 1) / s;
      float t = ts == 256 ? passes * per * c.slot256 : per * c.slot128 * (n * s <= 256 ? c.alone : (float)passes);
      t = passes * (ts == 256 ? c.fix256 : c.fix128) + (t > read ? t : read);
      if (s > 1) t += c.join + (float)s * M * N * batch * 8 / c.rate;
      if (best == 0.f || t < best) {
        best = t;
        *tile = ts;
        *splits = (int)s;
      }
    }
  }
  return best;
}
// The same for few rows of bf16: a launch, the weights (`rows` of K elements) once, and x in
// every workgroup of 16 weight rows, which each CU takes in at 37 bytes per ns (fitted to 1 to
// 64 rows at 4096 x 7168, 7168 x 2048, 1536 x 2048 and 2048 x 768). Both ways, gate/up and down
// of 7168 x 2048: one row 15.7 and 10.5 us against 19.3 and 12.0 as tiles, 16 rows 20.0 and 12.8
// against 19.9 and 13.5, 64 rows 40.5 and 25.6 against 22.9 and 15.1; of 2048 x 768: 16 rows
// 7.1 and 4.5 against 11.2 and 8.3, 64 rows 12.8 and 6.5 against 12.8 and 8.3.
inline float few_time(int64_t M, int64_t rows, int64_t K) {
  return 2.5f + (float)rows * K * 2 / 4.6e6f + (float)M * K * 2 * ((rows / 16 + 255) / 256) / 37e3f;
}
inline unsigned dense_grid(int64_t n) { return (unsigned)((n + kXcds - 1) / kXcds * kXcds); }

// A launch takes fewer than 2^32 threads along x: `blocks` workgroups as rows of 2^22.
inline dim3 flat_grid(int64_t blocks) {
  const int64_t row = (int64_t)1 << 22;
  return blocks <= row ? dim3((unsigned)blocks) : dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}
MOK_DEV int64_t flat_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

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
    // (from |a| = 16 on act or 1 - s is 0 in fp32: a*a, which passes the largest number at 1.8e19, is held there)
    const float p = __builtin_amdgcn_fmed3f(a, -16.0f, 16.0f);
    dact = s + act * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * p * p);
  }
}

}  // namespace mok
