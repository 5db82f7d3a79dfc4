// The tiled matrix product of linear.hip and linear_q8.hip: tiles straight into
// a swizzled LDS, matrix instructions, epilogues in registers, and the rules
// that choose a tile.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {

enum Mode { kFwd, kDx, kDw };

struct GemmArgs {
  WinTab a, b, out, bias, residual, preact;
  const int32_t* counts;  // [R][G] or null
  uint32_t* err;
  int R, G, rows;
  int M, N, K;            // kDw: M weight rows; else M is the group's rows. kDw: K is the group's rows
  int O;                  // columns of out (gated forward: N / 2)
  uint64_t lda, ldb;      // elements
  uint64_t b_group, out_group;
  int mt, nt;             // row tiles per rank (kDw: per group), column tiles
  int tile0;              // the launch's first tile
};

// A tile of ROWS rows and 128 bytes of the contraction axis, or of 128 bytes'
// elements of the contraction axis and ROWS columns, in 16-byte pieces:
//   KC (the contraction axis is contiguous): piece c of row r at position
//      c ^ (r & 7) of the row's 128 bytes, so that the 16 rows of a fragment
//      read fall on all banks;
//   otherwise rows of ROWS columns per k; pieces are exchanged so that the
//      rows of one read do: bf16, 4 rows for each 16 lanes, and the 4 rows 8
//      further on for the next 16 (with the first 4 alone, half the LDS's
//      cycles in dw were conflicts); fp32, the 4 row quarters.
template <int DT, bool KC, int ROWS>
struct Tile {
  static constexpr int kK = 128 / Elem<DT>::kSize;       // contraction elements
  static constexpr int kC = Elem<DT>::kChunk;
  static constexpr int kBytes = ROWS * 128;
  static constexpr int kPieces = ROWS * 8;
  static constexpr int kPerRow = KC ? 8 : ROWS / kC;     // pieces per stored row
  __device__ static int swz(int r) {
    if constexpr (KC) return r & 7;
    else if constexpr (DT == VR_DT_BF16) return ((r & 3) | (ROWS >= 128 ? (r >> 1) & 4 : 0)) << 1;
    else return ((r >> 2) & 3) << 2;
  }
  // Fragment of 16 rows (columns) from `base`, pieces ks: lane l holds
  // contraction elements ks * 4 pieces + (l / 16) of row base + l % 16.
  __device__ static v4u frag(const char* lds, int base, int ks, int lane) {
    const int i = lane & 15, q = lane >> 4;
    if constexpr (KC) {
      const int r = base + i;
      return *reinterpret_cast<const v4u*>(lds + r * 128 + (((ks * 4 + q) ^ swz(r)) << 4));
    } else if constexpr (DT == VR_DT_BF16) {
      // transposed 64-bit reads: 16 lanes name 4 rows of 16 columns, lane i gets column i of the 4 rows
      const int k = ks * 32 + q * 8 + (i >> 2);
      const int c = (base >> 3) + ((i >> 1) & 1);
      const char* p = lds + ((k * kPerRow + (c ^ swz(k))) << 4) + ((i & 1) << 3);
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * kPerRow * 16));
      const v2u a = __builtin_bit_cast(v2u, lo), b = __builtin_bit_cast(v2u, hi);
      return v4u{a[0], a[1], b[0], b[1]};
    } else {
      v4u v;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = ks * 16 + q * 4 + s, col = base + i;
        v[s] = *reinterpret_cast<const uint32_t*>(lds + ((k * kPerRow + ((col >> 2) ^ swz(k))) << 4) + ((col & 3) << 2));
      }
      return v;
    }
  }
};

// Epilogue of 4 consecutive columns of one row.
template <int DT>
__device__ inline void load4(const char* p, uint64_t i, int n, float* f) {
  if (n >= 4) {
    load_n<DT, 4>(p, i, f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < n ? Elem<DT>::load(p, i + j) : 0.0f;
  }
}
template <int DT>
__device__ inline void store4(char* p, uint64_t i, int n, const float* f) {
  if (n >= 4) {
    store_n<DT, 4>(p, i, f);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) Elem<DT>::store(p, i + j, f[j]);
  }
}

template <int DT, int ACT, bool gated>  // DT: of out
__device__ inline void epilogue(const GemmArgs& a, int r, int g, int row, int col, v4f z0, v4f z1) {
  const int n = a.O - col;
  if (n <= 0) return;
  float g4[4], u4[4], y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g4[j] = z0[j];
    u4[j] = z1[j];
  }
  if (a.bias.p[r]) {
    float b[4];
    load4<DT>(a.bias.p[r], (uint64_t)g * a.N + col, n, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) g4[j] += b[j];
    if (gated) {
      load4<DT>(a.bias.p[r], (uint64_t)g * a.N + a.O + col, n, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) u4[j] += b[j];
    }
  }
  if (a.preact.p[r]) {
    store4<DT>(a.preact.p[r], (uint64_t)row * a.N + col, n, g4);
    if (gated) store4<DT>(a.preact.p[r], (uint64_t)row * a.N + a.O + col, n, u4);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = act_value<DT, ACT>(g4[j]);
    if (gated) y[j] *= u4[j];
  }
  if (a.residual.p[r]) {
    float b[4];
    load4<DT>(a.residual.p[r], (uint64_t)row * a.O + col, n, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += b[j];
  }
  store4<DT>(a.out.p[r], (uint64_t)row * a.O + col, n, y);
}

// 4 elements as they lie in memory.
template <int DT> struct Raw4 { typedef v4u T; };
template <> struct Raw4<VR_DT_BF16> { typedef v2u T; };
template <int DT>
__device__ inline typename Raw4<DT>::T load_raw4(const char* p) {
  typename Raw4<DT>::T v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, Elem<DT>::kSize), sizeof(v));
  return v;
}
template <int DT>
__device__ inline v4f from_raw4(typename Raw4<DT>::T v) {
  if constexpr (DT == VR_DT_F32) return __builtin_bit_cast(v4f, v);
  else return v4f{bf16lo(v[0]), bf16hi(v[0]), bf16lo(v[1]), bf16hi(v[1])};
}

// sum * scale of the row * scale of the channel. A sum, below 2^31, times a scale above
// 2^64 might pass binary32 where a small second scale brings it back: such a scale
// is taken in two parts.
struct RowScale {
  float s, after;
  bool large;
  __device__ explicit RowScale(float scale) : large(fabsf(scale) > 0x1p64f) {
    s = large ? scale * 0x1p-64f : scale;
    after = large ? 0x1p64f : 1.0f;
  }
  __device__ float operator()(int sum, float w) const { return static_cast<float>(sum) * s * w * after; }
};

// Epilogue of a wave's part of a tile that has all its columns: NF x MF
// fragments from column c0 and row m0 (of the group; rows up to mEnd). Loads
// are issued many rows ahead: out might be residual's own slice, so the
// compiler keeps their order, and a fragment at a time each load's latency was
// waited for in turn (82 of the 300 us of a dense 8192 x 4096 x 4096
// product).
// large: rows' second parts of scales are left, their scales in the LDS at row_scales.
// PAIRS: fragments 2 p and 2 p + 1 hold the columns 32 p + 8 q + 0..3 and + 4..7 of
// lane quarter q, not 16 each: 16-byte stores of bf16 rather than 8.
// BARE: no bias, residual, preact or large scale. A tensor that may be absent costs a branch at
// every use, and where the branches meet a wait for loads that were not issued,
// which then waits for the stores and for the next tile's loads: the experts'
// 8 x 32768 rows (15/16 used), 512 -> 512 gated, in 8 bits 302 to 275 us, in bf16 from 256
// elements 271 to 257.
template <int DT, int ACT, bool GATED, int NF, int MF, bool PAIRS, bool BARE>
__device__ inline void epilogue_whole(const GemmArgs& a, int r, int g, int row0, int m0, int mEnd, int c0, int lane,
                                      v4f (*acc)[MF], [[maybe_unused]] bool large,
                                      [[maybe_unused]] const float* row_scales) {
  constexpr int kES = Elem<DT>::kSize, NO = GATED ? NF / 2 : NF, S = GATED ? 2 : 1;
  const int m1 = m0 + (lane & 15), col = c0 + (lane >> 4) * (PAIRS ? 8 : 4);
  const auto off = [](int i) { return PAIRS ? (i >> 1) * 32 + (i & 1) * 4 : i * 16; };
  // rows whose residual is held at once: all of a small tile's, 32 registers
  constexpr int kRows = MF <= 4 ? MF : 4;
  typename Raw4<DT>::T bias[NO][S], res[kRows][NO];
  const char* pb = BARE ? nullptr : a.bias.p[r];
  const char* pr = BARE ? nullptr : a.residual.p[r];
  char* pz = BARE ? nullptr : a.preact.p[r];
  char* po = a.out.p[r];
  if (pb) {
    pb += ((uint64_t)g * a.N + col) * kES;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int h = 0; h < S; ++h) bias[i][h] = load_raw4<DT>(pb + (uint64_t)(h * a.O + off(i)) * kES);
  }
#pragma unroll
  for (int j0 = 0; j0 < MF; j0 += kRows) {
    if (pr) {
#pragma unroll
      for (int v = 0; v < kRows; ++v)
#pragma unroll
        for (int i = 0; i < NO; ++i)
          res[v][i] = load_raw4<DT>(pr + ((uint64_t)(row0 + min(m1 + (j0 + v) * 16, mEnd - 1)) * a.O + col + off(i)) * kES);
    }
#pragma unroll
    for (int v = 0; v < kRows; ++v) {
      const uint64_t row = row0 + m1 + (j0 + v) * 16;
      if (!BARE && large) {
        const float after = RowScale(row_scales[(j0 + v) * 16 + (lane & 15)]).after;
#pragma unroll
        for (int i = 0; i < NF; ++i) acc[i][j0 + v] *= after;
      }
      if (m1 + (j0 + v) * 16 < mEnd) {
        float pair[8];
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          float z[S][4], *y = pair + (PAIRS ? (i & 1) * 4 : 0);
#pragma unroll
          for (int h = 0; h < S; ++h) {
#pragma unroll
            for (int q = 0; q < 4; ++q) z[h][q] = acc[i * S + h][j0 + v][q];
            if (pb) {
              const v4f f = from_raw4<DT>(bias[i][h]);
#pragma unroll
              for (int q = 0; q < 4; ++q) z[h][q] += f[q];
            }
            if (pz) store_n<DT, 4>(pz, row * a.N + h * a.O + col + off(i), z[h]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[q] = act_value<DT, ACT>(z[0][q]);
            if (GATED) y[q] *= z[S - 1][q];
          }
          if (pr) {
            const v4f f = from_raw4<DT>(res[v][i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] += f[q];
          }
          if (!PAIRS) store_n<DT, 4>(po, row * a.O + col + off(i), y);
          else if (i & 1) store_n<DT, 8>(po, row * a.O + col + off(i - 1), pair);
        }
      }
    }
  }
}

// 16 bytes per lane from base + off straight into the LDS at `to` + 16 * lane
// (`to` the same in all lanes). In asm so that the compiler, which cannot tell
// the two halves of the LDS apart across a loop, does not wait for it before
// every LDS read: the caller waits for vmcnt and meets at a barrier instead.
// There is no output register, and the address is read when it issues. m0 is
// reserved: the compiler keeps nothing in it between instructions. Five wait
// states have to lie between a vector instruction that writes a scalar
// register (v_readfirstlane, or v_readlane of a spilled one) and a vector memory
// instruction that reads it; the compiler keeps this in its own code but does
// not look into asm, so all five are here: s_mov and s_nop 3.
__device__ inline void load_lds16(const char* base, uint32_t off, char* to) {
  const uint32_t lds = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(to)));
  const uint64_t at = reinterpret_cast<uintptr_t>(base);
  const uint64_t uniform = (static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32))) << 32) |
                           static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform) : "memory");
}

// 4 bytes per lane from p straight into the LDS at `to` + lane (`to` the same in
// all lanes); as load_lds16 otherwise, but the address is a vector's: one wait
// state between m0's write and its use.
__device__ inline void load_lds4(const char* p, float* to) {
  const uint32_t lds = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) float*)(to)));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory");
}

// Workgroups of consecutive numbers run on the XCDs in turn; give each XCD
// consecutive tiles, which share rows of a and b in its L2.
__device__ inline int xcd_order(int b, int n) {
  const int x = b & 7, q = n >> 3, rem = n & 7;
  return x * q + min(x, rem) + (b >> 3);
}

// One BM x BN tile of out per workgroup; the waves' WM x WN parts stay in
// registers. The matrix instructions take the b side (columns of out) as
// their first operand, so a lane's four sums are four consecutive columns of
// one row of out. While one 128-byte step of the contraction axis is
// multiplied, the next is on its way into the other half of the LDS: straight
// from global memory where rows start on 16 bytes (DIRECT), else through
// registers, zero-filled past the ends.
template <int DT, int MODE, bool GATED, bool DIRECT, int BM, int BN, int WM, int WN, int STAGES>
struct Gemm {
  static constexpr int kThreads = 64 * (BM / WM) * (BN / WN);
  using TA = Tile<DT, MODE != kDw, BM>;
  using TB = Tile<DT, MODE == kFwd, BN>;
  static constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kK = TA::kK;
  static constexpr int kPA = TA::kPieces / kThreads, kPB = TB::kPieces / kThreads;
  static constexpr int kMF = WM / 16, kNF = WN / 16;
  static constexpr bool kPairs = kInt8<DT> && (GATED ? kNF / 2 : kNF) % 2 == 0;
  static constexpr int kStage = TA::kBytes + TB::kBytes, kStages = !DIRECT || kThreads == 512 ? 2 : STAGES;

  struct Where {
    const char *pa, *pb;  // the tile's rows of a and b at contraction index 0
    uint64_t lda, ldb;    // bytes
    int m0, mEnd, n0, N, O, K, width_a, width_b;
  };

  struct Spot {
    Where t;
    int r, g, row0;
  };
  // Tile b: tiles of a group (kDw) or rank, then groups and
  // ranks. False when there is no such tile. find(r, slot): the group of a row tile.
  template <class F>
  __device__ static __forceinline__ bool locate(const GemmArgs& a, int b, Spot* s, F find) {
    Where& t = s->t;
    int nti = b % a.nt, slot = b / a.nt % a.mt;
    b /= a.nt * a.mt;
    if (MODE == kDw || !a.counts) {
      // a band of 8 row tiles, column by column: the tiles that run on one XCD at a time are 8 by 4
      const int band = slot / 8 * 8, high = min(8, a.mt - band), in = (slot - band) * a.nt + nti;
      slot = band + in % high;
      nti = in / high;
    }
    if constexpr (MODE == kDw) {
      s->g = b % a.G;
      s->r = b / a.G;
      const GroupTile q = find_group<true>(a.counts ? a.counts + (size_t)s->r * a.G : nullptr, a.G, a.rows, 1, s->g, a.err);
      s->row0 = q.first;
      t.K = q.count;
      t.m0 = slot * BM;
      t.mEnd = a.M;
    } else {
      s->r = b;
      const GroupTile q = find(s->r, slot);
      if (q.g < 0) return false;
      s->g = q.g;
      s->row0 = q.first;
      t.K = a.K;
      t.m0 = (slot - q.tile0) * BM;
      t.mEnd = q.count;
    }
    t.n0 = nti * BN;  // tile's first column of b; gated: BN / 2 columns of either half
    t.N = a.N;
    t.O = a.O;
    t.lda = a.lda * kES;
    t.ldb = a.ldb * kES;
    t.width_a = static_cast<int>(a.lda);
    t.width_b = static_cast<int>(a.ldb);
    t.pa = a.a.p[s->r] + (uint64_t)s->row0 * t.lda + (MODE != kDw ? (uint64_t)t.m0 * t.lda : 0);
    t.pb = a.b.p[s->r] + (MODE == kDw ? (uint64_t)s->row0 * t.ldb : (uint64_t)s->g * a.b_group * kES) +
           (MODE == kFwd ? (uint64_t)(GATED ? t.n0 / 2 : t.n0) * t.ldb : 0);
    return true;
  }

  __device__ static __forceinline__ bool locate(const GemmArgs& a, int b, Spot* s) {
    return locate(a, b, s, [&](int r, int slot) {
      return find_group<false>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, BM, slot, a.err);
    });
  }

  template <int ACT>
  __device__ static __forceinline__ void finish(const GemmArgs& a, const Spot& s, int wm, int wn, int lane, v4f (*acc)[kMF],
                                                bool large = false, const float* row_scales = nullptr) {
    const Where& t = s.t;
    if constexpr (MODE == kFwd) {
      if (GATED ? t.n0 / 2 + BN / 2 <= a.O : t.n0 + BN <= a.N) {
        const int c0 = GATED ? (t.n0 + wn) / 2 : t.n0 + wn;
        if (a.bias.p[s.r] || a.residual.p[s.r] || a.preact.p[s.r] || large)
          epilogue_whole<kOutOf<DT>, ACT, GATED, kNF, kMF, kPairs, false>(a, s.r, s.g, s.row0, t.m0 + wm, t.mEnd, c0, lane, acc,
                                                                          large, row_scales);
        else
          epilogue_whole<kOutOf<DT>, ACT, GATED, kNF, kMF, kPairs, true>(a, s.r, s.g, s.row0, t.m0 + wm, t.mEnd, c0, lane, acc,
                                                                          large, row_scales);
        return;
      }
    }
    const int cq = (lane >> 4) * 4;
#pragma unroll
    for (int j = 0; j < kMF; ++j) {
      const int m = t.m0 + wm + j * 16 + (lane & 15);
      if (m >= t.mEnd) continue;
      if (large) {
        const float after = RowScale(row_scales[j * 16 + (lane & 15)]).after;
#pragma unroll
        for (int i = 0; i < kNF; ++i) acc[i][j] *= after;
      }
#pragma unroll
      for (int i = 0; i < kNF; i += GATED ? 2 : 1) {
        if constexpr (MODE == kFwd) {
          const int io = GATED ? i / 2 : i, c0 = GATED ? (t.n0 + wn) / 2 : t.n0 + wn;
          const int col = c0 + (kPairs ? (io >> 1) * 32 + cq * 2 + (io & 1) * 4 : io * 16 + cq);
          epilogue<kOutOf<DT>, ACT, GATED>(a, s.r, s.g, s.row0 + m, col, acc[i][j], acc[i + (GATED ? 1 : 0)][j]);
        } else {
          const int col = t.n0 + wn + i * 16 + cq;
          float y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = acc[i][j][q];
          const uint64_t row = MODE == kDw ? (uint64_t)m : (uint64_t)(s.row0 + m);
          if (col < a.N) store4<DT>(a.out.p[s.r] + (uint64_t)s.g * a.out_group * kES, row * a.N + col, a.N - col, y);
        }
      }
    }
  }

  // The scales of a tile's rows of a and b, the last 4 bytes of each, on their
  // way into the LDS before anything else is, so that the first step's wait
  // covers them. (Read from memory by the epilogue they took up to 45 us of 233 at
  // 8 x 32768 rows (15/16 used), 128 -> 512 gated.) kThreads >= BM and >= BN.
  static constexpr int kScales = kInt8<DT> ? BM + BN : 0;  // floats
  __device__ static __forceinline__ void fetch_scales(const Where& t, int tid, int wave, float* to) {
    if (wave < BM / 64)
      load_lds4(t.pa + (uint64_t)(min(t.m0 + tid, t.mEnd - 1) - t.m0 + 1) * t.lda - 4, to + wave * 64);
    if (wave < BN / 64) {
      bool in;
      const int n = b_row(t, tid, &in);  // where there is no such row, the tile's first: not stored
      load_lds4(t.pb + (in ? n - (GATED ? t.n0 / 2 : t.n0) + 1 : 1) * (int64_t)t.ldb - 4, to + BM + wave * 64);
    }
  }
  // The sums scaled; second parts of large scales are taken too or, kLate, left to the general epilogue, a row at a time
  // (true: there are some). All of a gated bf16 tile at once put 46 registers into scratch, the experts' 8 x 32768 rows,
  // 512 -> 512 gated, 236 to 262 us, and a branch for it in the bare epilogue took 245; fp32 has no registers left there.
  static constexpr bool kLate = GATED && DT == kI8ToBf16;
  __device__ static __forceinline__ bool scaled(const float* scales, int wm, int wn, int lane, const Acc<DT> (*acc)[kMF], v4f (*z)[kMF]) {
    float sx[kMF];
    bool large = false;
#pragma unroll
    for (int j = 0; j < kMF; ++j) {
      const RowScale by(scales[wm + j * 16 + (lane & 15)]);
      sx[j] = by.s;
      large |= by.large;
    }
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const v4f sw = *reinterpret_cast<const v4f*>(scales + BM + wn + i * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int j = 0; j < kMF; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) z[i][j][q] = static_cast<float>(acc[i][j][q]) * sx[j] * sw[q];
    }
    const bool any = ballot(large) != 0;
    if (kLate || !any) return any;
#pragma unroll
    for (int j = 0; j < kMF; ++j) {
      const float after = RowScale(scales[wm + j * 16 + (lane & 15)]).after;
#pragma unroll
      for (int i = 0; i < kNF; ++i) z[i][j] *= after;
    }
    return false;
  }

  // Row of b behind tile row j (forward): gated, 16 gate columns, then the same 16
  // of the other half. kPairs: the columns as epilogue_whole's PAIRS has them.
  __device__ static __forceinline__ int b_row(const Where& t, int j, bool* in) {
    const int at = ((j >> 2) & 3) * 8 + (j & 3);
    if constexpr (GATED) {
      const int o = t.n0 / 2 + (kPairs ? (j >> 6) * 32 + at + ((j >> 5) & 1) * 4 : (j >> 5) * 16 + (j & 15));
      *in = o < t.O;
      return o + ((j >> 4) & 1) * t.O;
    } else {
      const int n = t.n0 + (kPairs ? (j & ~31) + at + ((j >> 4) & 1) * 4 : j);
      *in = n < t.N;
      return n;
    }
  }

  // Byte offsets of a thread's pieces from pa, pb; pieces outside are taken
  // from a valid row or column (their products are not stored).
  __device__ static __forceinline__ void offsets(const Where& t, int tid, uint32_t* oa, uint32_t* ob) {
#pragma unroll
    for (int i = 0; i < kPA; ++i) {
      const int id = i * kThreads + tid, sr = id / TA::kPerRow, c = (id % TA::kPerRow) ^ TA::swz(sr);
      if constexpr (MODE != kDw) oa[i] = static_cast<uint32_t>(min(t.m0 + sr, t.mEnd - 1) - t.m0) * static_cast<uint32_t>(t.lda) + (c << 4);
      else oa[i] = sr * static_cast<uint32_t>(t.lda) + min(t.m0 + c * kC, t.width_a - kC) * kES;
    }
#pragma unroll
    for (int i = 0; i < kPB; ++i) {
      const int id = i * kThreads + tid, sr = id / TB::kPerRow, c = (id % TB::kPerRow) ^ TB::swz(sr);
      if constexpr (MODE == kFwd) {
        bool in;
        const int n = b_row(t, sr, &in);
        ob[i] = 0;
        if constexpr (GATED) {
          const int o = min(n - ((sr >> 4) & 1) * t.O, t.O - 1);  // the second half's rows are t.O rows further on
          ob[i] = static_cast<uint32_t>(o - t.n0 / 2) * static_cast<uint32_t>(t.ldb) + (c << 4);
        } else {
          ob[i] = static_cast<uint32_t>(min(n, t.N - 1) - t.n0) * static_cast<uint32_t>(t.ldb) + (c << 4);
        }
      } else {
        ob[i] = sr * static_cast<uint32_t>(t.ldb) + min(t.n0 + c * kC, t.width_b - kC) * kES;
      }
    }
  }

  // Pieces of step k0 by registers, zero past the ends.
  __device__ static __forceinline__ void load(const Where& t, int tid, int k0, v4u* ra, v4u* rb) {
#pragma unroll
    for (int i = 0; i < kPA; ++i) {
      const int id = i * kThreads + tid, sr = id / TA::kPerRow, c = (id % TA::kPerRow) ^ TA::swz(sr);
      if constexpr (MODE != kDw) {
        const int m = t.m0 + sr, k = k0 + c * kC;
        ra[i] = load_piece<DT>(t.pa + (uint64_t)sr * t.lda + (uint64_t)k * kES, m < t.mEnd ? t.K - k : 0);
      } else {
        const int k = k0 + sr, m = t.m0 + c * kC;
        ra[i] = load_piece<DT>(t.pa + (uint64_t)k * t.lda + (uint64_t)m * kES, k < t.K ? t.mEnd - m : 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kPB; ++i) {
      const int id = i * kThreads + tid, sr = id / TB::kPerRow, c = (id % TB::kPerRow) ^ TB::swz(sr);
      if constexpr (MODE == kFwd) {
        const int k = k0 + c * kC;
        bool in;
        const int n = b_row(t, sr, &in);
        const int64_t from = n - (GATED ? t.n0 / 2 : t.n0);
        rb[i] = load_piece<DT>(t.pb + from * static_cast<int64_t>(t.ldb) + (int64_t)k * kES, in ? t.K - k : 0);
      } else {
        const int k = k0 + sr, n = t.n0 + c * kC;
        rb[i] = load_piece<DT>(t.pb + (uint64_t)k * t.ldb + (uint64_t)n * kES, k < t.K ? t.N - n : 0);
      }
    }
  }
  __device__ static __forceinline__ void store(int tid, char* la, char* lb, const v4u* ra, const v4u* rb) {
#pragma unroll
    for (int i = 0; i < kPA; ++i) *reinterpret_cast<v4u*>(la + ((i * kThreads + tid) << 4)) = ra[i];
#pragma unroll
    for (int i = 0; i < kPB; ++i) *reinterpret_cast<v4u*>(lb + ((i * kThreads + tid) << 4)) = rb[i];
  }

  // Half ks of a step: the fragments, and their products.
  __device__ static __forceinline__ void frags(const char* la, const char* lb, int ks, int wm, int wn, int lane,
                                               v4u* fa, v4u* fb) {
#pragma unroll
    for (int i = 0; i < kNF; ++i) fb[i] = TB::frag(lb, wn + i * 16, ks, lane);
#pragma unroll
    for (int j = 0; j < kMF; ++j) fa[j] = TA::frag(la, wm + j * 16, ks, lane);
  }
  __device__ static __forceinline__ void products(const v4u* fa, const v4u* fb, Acc<DT> (*acc)[kMF]) {
#pragma unroll
    for (int j = 0; j < kMF; ++j)
#pragma unroll
      for (int i = 0; i < kNF; ++i) acc[i][j] = mfma_piece<DT>(fb[i], fa[j], acc[i][j]);
  }
  __device__ static __forceinline__ void multiply(const char* la, const char* lb, int wm, int wn, int lane, Acc<DT> (*acc)[kMF]) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v4u fa[kMF], fb[kNF];
      frags(la, lb, ks, wm, wn, lane, fa, fb);
      products(fa, fb, acc);
    }
  }

  // Start the loads of the whole step k1 into `to`.
  __device__ static __forceinline__ void fetch(const Where& t, int k1, int tid, int wave, const uint32_t* oa,
                                               const uint32_t* ob, char* to) {
    const char* pa = t.pa + (MODE != kDw ? (uint64_t)k1 * kES : (uint64_t)k1 * t.lda);
    const char* pb = t.pb + (MODE == kFwd ? (uint64_t)k1 * kES : (uint64_t)k1 * t.ldb);
#pragma unroll
    for (int i = 0; i < kPA; ++i) load_lds16(pa, oa[i], to + ((i * kThreads + wave * 64) << 4));
#pragma unroll
    for (int i = 0; i < kPB; ++i) {
      const char* half = pb;
      // gated: 8 pieces of a wave's 8 rows are in one block of 16, so in one half of the columns
      if constexpr (GATED)
        half += ((((i * kThreads + wave * 64) / TB::kPerRow) >> 4) & 1) ? (uint64_t)t.O * t.ldb : 0;
      load_lds16(half, ob[i], to + TA::kBytes + ((i * kThreads + wave * 64) << 4));
    }
  }

  // Multiply what is in `cur` while step k1 goes to `nxt` by registers.
  __device__ static __forceinline__ void step(const Where& t, int k1, int tid, const char* cur, char* nxt, int wm, int wn, int lane, Acc<DT> (*acc)[kMF]) {
    v4u ra[kPA], rb[kPB];
    load(t, tid, k1, ra, rb);  // nothing past the end
    multiply(cur, cur + TA::kBytes, wm, wn, lane, acc);
    store(tid, nxt, nxt + TA::kBytes, ra, rb);
    __syncthreads();
  }
  // All whole steps through a ring of kStages steps in the LDS: kStages - 1 are
  // on their way or there while one is multiplied. A tile of few waves has
  // nothing else to cover the loads' latency with.
  __device__ static __forceinline__ void ring(const Where& t, int steps, int tid, int wave, const uint32_t* oa,
                                              const uint32_t* ob, char* s, int wm, int wn, int lane, Acc<DT> (*acc)[kMF]) {
    int to = 0;  // bytes: the stage that is loaded next
    const auto next = [](int at) { return at == (kStages - 1) * kStage ? 0 : at + kStage; };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i, to = next(to))
      if (i < steps) fetch(t, i * kK, tid, wave, oa, ob, s + to);
    int at = 0;
    for (int i = 0; i < steps; ++i, at = next(at)) {
      // step i has landed, in every wave, and step i - 1 has been read
      if (i + kStages - 2 < steps) meet<(kStages - 2) * (kPA + kPB)>();
      else meet<0>();
      if (i + kStages - 1 < steps) fetch(t, (i + kStages - 1) * kK, tid, wave, oa, ob, s + to);
      to = next(to);
      multiply(s + at, s + at + TA::kBytes, wm, wn, lane, acc);
    }
    meet<0>();
  }
  // Two groups of four waves, one wave of each per SIMD, a phase apart: while
  // one reads its fragments of a half step from the LDS the other multiplies,
  // so that the matrix units do not wait for the LDS. Phases end at barriers:
  //   first group    R0(t) M0(t) R1(t) M1(t)  R0(t+1) ...
  //   second group   M1(t-1) R0(t) M0(t) R1(t)  M1(t) ...
  // In the phase of the first group's R0(t) every read of step t-1 is done:
  // both groups then start loading step t+1 over it, and wait for it at the
  // end of the phase of M1(t), before the first group's R0(t+1).
  // AHEAD: step 1 is on its way already; both groups load the others behind the
  // reads of their R0, where waiting to issue holds up no matrix instruction
  // (8192 x 4096 x 4096 in 8 bits with gelu, bias and residual: 172 to 160 us).
  template <bool FIRST, bool AHEAD>
  __device__ static __forceinline__ void phases(const Where& t, int steps, int tid, int wave, const uint32_t* oa,
                                                const uint32_t* ob, char* s0, char* s1, int wm, int wn, int lane,
                                                Acc<DT> (*acc)[kMF]) {
    if (!FIRST) {
      if (!AHEAD && steps > 1) fetch(t, kK, tid, wave, oa, ob, s1);
      barrier();
    }
    for (int i = 0; i < steps; ++i) {
      char* cur = (i & 1) ? s1 : s0;
      char* nxt = (i & 1) ? s0 : s1;
      v4u fa[kMF], fb[kNF];
      if (!AHEAD && FIRST && i + 1 < steps) fetch(t, (i + 1) * kK, tid, wave, oa, ob, nxt);
      frags(cur, cur + TA::kBytes, 0, wm, wn, lane, fa, fb);
      if (AHEAD && i > 0 && i + 1 < steps) fetch(t, (i + 1) * kK, tid, wave, oa, ob, nxt);
      lds_done();
      barrier();
      __builtin_amdgcn_s_setprio(1);
      products(fa, fb, acc);
      __builtin_amdgcn_s_setprio(0);
      barrier();
      frags(cur, cur + TA::kBytes, 1, wm, wn, lane, fa, fb);
      lds_done();
      if (!FIRST) wait_vmem();
      barrier();
      if (!AHEAD && !FIRST && i + 2 < steps) fetch(t, (i + 2) * kK, tid, wave, oa, ob, cur);
      __builtin_amdgcn_s_setprio(1);
      products(fa, fb, acc);
      __builtin_amdgcn_s_setprio(0);
      if (FIRST) wait_vmem();
      barrier();
    }
    if (FIRST) barrier();
  }
  __device__ static __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
  __device__ static __forceinline__ void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  // Own loads but the last LATER have landed and own reads are done, in every wave.
  template <int LATER = 0>
  __device__ static __forceinline__ void meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LATER) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
};

// One tile. (A 256 x 256 tile's workgroup has its compute unit to itself; one
// that took tile after tile, the next one's first step loading during the
// epilogue, was slower: 302 us beside 275 for 8192 x 4096 x 4096, 259 beside
// 249 for the experts' 32768 rows, since a tile then waits for the stores of
// the one before.)
template <int DT, int MODE, int ACT, bool GATED, bool DIRECT, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_gemm(const GemmArgs a) {
  using G = Gemm<DT, MODE, GATED, DIRECT, BM, BN, WM, WN, STAGES>;
  constexpr int kK = G::kK, kMF = G::kMF, kNF = G::kNF;
  __shared__ __align__(16) char s0[G::kStages * G::kStage + G::kScales * 4];
  char* s1 = s0 + G::kStage;
  float* scales = reinterpret_cast<float*>(s0 + G::kStages * G::kStage);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave % (BM / WM)) * WM, wn = (wave / (BM / WM)) * WN;
  typename G::Spot at;
  if (!G::locate(a, a.tile0 + xcd_order(blockIdx.x, gridDim.x), &at)) return;
  const typename G::Where& t = at.t;
  if constexpr (kInt8<DT>) G::fetch_scales(t, tid, wave, scales);

  Acc<DT> acc[kNF][kMF];
#pragma unroll
  for (int i = 0; i < kNF; ++i)
#pragma unroll
    for (int j = 0; j < kMF; ++j) acc[i][j] = Acc<DT>{0, 0, 0, 0};
  // whole steps (DIRECT; the others zero-fill and take every step here)
  const int steps = DIRECT ? t.K / kK : (t.K + kK - 1) / kK;
  if (steps > 0) {
    if constexpr (DIRECT) {
      uint32_t oa[G::kPA], ob[G::kPB];
      G::offsets(t, tid, oa, ob);
      if constexpr (G::kThreads == 512) {
        G::fetch(t, 0, tid, wave, oa, ob, s0);
        G::meet();
        if (wave < 4) G::template phases<true, false>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
        else G::template phases<false, false>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
      } else {
        G::ring(t, steps, tid, wave, oa, ob, s0, wm, wn, lane, acc);
      }
    } else {
      v4u ra[G::kPA], rb[G::kPB];
      G::load(t, tid, 0, ra, rb);
      G::store(tid, s0, s0 + G::TA::kBytes, ra, rb);
      if constexpr (kInt8<DT>) wait_vmem();  // the scales too
      __syncthreads();
      for (int i = 0; i < steps; ++i)
        G::step(t, (i + 1) * kK, tid, (i & 1) ? s1 : s0, (i & 1) ? s0 : s1, wm, wn, lane, acc);
    }
  }
  if (DIRECT && steps * kK < t.K) {  // the last, partial step: by registers, zero-filled
    v4u ra[G::kPA], rb[G::kPB];
    G::load(t, tid, steps * kK, ra, rb);
    G::store(tid, s0, s0 + G::TA::kBytes, ra, rb);
    if constexpr (kInt8<DT>) wait_vmem();  // the scales too, where no whole step was
    __syncthreads();
    G::multiply(s0, s0 + G::TA::kBytes, wm, wn, lane, acc);
  }
  if constexpr (kInt8<DT>) {
    v4f z[kNF][kMF];
    const bool large = G::scaled(scales, wm, wn, lane, acc, z);
    G::template finish<ACT>(a, at, wm, wn, lane, z, large, scales + wm);
  } else {
    G::template finish<ACT>(a, at, wm, wn, lane, acc);
  }
}

// The groups of a rank in the LDS, for a workgroup that takes many of its tiles:
// past the last row tile (of bm rows) and the first row of each group. What
// find_group finds by itself for every tile, about 3000 cycles, is a read and a
// ballot here.
struct GroupTable {
  int32_t *end, *first;  // [G], [G + 1]
  // By one wave. Counts as find_group takes them, all of them looked at.
  __device__ void build(const int32_t* counts, int G, int rows, int bm, uint32_t* err) const {
    const int lane = static_cast<int>(lane_id());
    int row0 = 0, tile0 = 0;
    bool bad = false;
    for (int g0 = 0; g0 < G; g0 += 64) {
      const int g = g0 + lane, c = g < G ? counts[g] : 0, pos = max(c, 0);
      int64_t s = pos;  // sums of 64 counts pass 32 bits
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const int64_t o = __shfl_up(s, m);
        if (lane >= m) s += o;
      }
      const int64_t last = s + row0;
      const int lo = static_cast<int>(last - pos < rows ? last - pos : rows);
      const int hi = static_cast<int>(last < rows ? last : rows);
      bad |= c < 0 || last > rows;
      int k = (hi - lo + bm - 1) / bm;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(k, m);
        if (lane >= m) k += o;
      }
      if (g < G) {
        end[g] = tile0 + k;
        first[g] = lo;
        if (g == G - 1) first[G] = hi;
      }
      row0 = __builtin_amdgcn_readlane(hi, 63);
      tile0 += __builtin_amdgcn_readlane(k, 63);
    }
    if (ballot(bad) && lane == 0) atomic_or_u32(err, VR_ASYNC_CAPACITY);
  }
  // The group that holds row tile `want`.
  __device__ GroupTile find(int G, int want) const {
    const int lane = static_cast<int>(lane_id());
    for (int g0 = 0; g0 < G; g0 += 64) {
      const uint64_t past = ballot(g0 + lane < G && end[min(g0 + lane, G - 1)] > want);
      if (!past) continue;
      const int g = g0 + __builtin_ctzll(past);
      const int lo = __builtin_amdgcn_readfirstlane(first[g]), hi = __builtin_amdgcn_readfirstlane(first[g + 1]);
      return {g, lo, hi - lo, g ? __builtin_amdgcn_readfirstlane(end[g - 1]) : 0};
    }
    return {-1, 0, 0, 0};
  }
};

// 256 x 256 tiles of rows in 8 bits, one workgroup to a compute unit that takes
// tile after tile: while it finishes one, the next one's first two steps and its
// scales are on their way. They were issued before the stores, and vector memory
// operations count down in order, so that the next tile waits for them and not
// for the stores, where the number of these is known (a whole tile).
//
// Four steps of 128 bytes and a silu epilogue (8 x 32768 rows, 15/16 used, by 32 experts,
// 512 -> 512 gated, 244 us), cycles of a tile, at its median: 14600 for the steps
// (8200 at the matrix units' rate; each step's loads have one step's time),
// 6700 for the next tile's loads to be taken (128 KB), 5000 for the epilogue, 3600 until
// the waves meet, 1400 to find the next tile. With 32 steps (8192 x 4096 x 4096,
// gelu, bias, residual, 149 us) the matrix units are 42 % busy and the card's
// power matters: zeros take 112 us where random values take 131.
//
// fp32 results are slower than their bytes: without a gate 27 to 37 registers lie in
// scratch and are read back behind the next tile's loads (the dense case 231 us, bf16
// 152), gated 3 at most (the experts 338 and 247, of which 250 MB more take about 40).
//
// Tiles are dealt out by the buffers' capacity, as the used rows are known on the
// device alone: where a rank's buffer is only partly used, so are the XCDs. The same
// 32768 used rows of one rank, 32 experts, 512 -> 512 gated, take 41, 63, 102, 185 us
// in a buffer of 1, 2, 4, 8 times as many; 2 ranks 68, 106, 188, 207; of 4 ranks 16384
// rows each 67, 108, 108, 114, of 8 ranks 114, 127, 125, 140.
template <int DT, int ACT, bool GATED>
__global__ __launch_bounds__(512) void k_gemm_run(const GemmArgs a, int tiles) {
  using G = Gemm<DT, kFwd, GATED, true, 256, 256, 128, 64, 2>;
  constexpr int kK = G::kK, kMF = G::kMF, kNF = G::kNF;
  // stores of a wave's part of a whole tile, at least (fp32: twice as many)
  constexpr int kLoads = G::kPA + G::kPB, kStores = kMF * (GATED ? kNF / 2 : kNF) / 2;
  static_assert(G::kPairs && kLoads + kStores < 64, "what a wait counts");
  __shared__ __align__(16) char s0[2 * G::kStage + 2 * G::kScales * 4 + (2 * 1024 + 1) * 4];
  char* s1 = s0 + G::kStage;
  float* scales = reinterpret_cast<float*>(s0 + 2 * G::kStage);
  int32_t* words = reinterpret_cast<int32_t*>(scales + 2 * G::kScales);
  const GroupTable table = {words, words + 1024};
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave % 2) * 128, wn = (wave / 2) * 64;
  // an XCD's tiles are consecutive, and so are those that run on it at a time
  const int x = blockIdx.x & 7, q = tiles >> 3, rem = tiles & 7, stride = gridDim.x >> 3;
  const int end = (x + 1) * q + min(x + 1, rem);
  int b = x * q + min(x, rem) + (blockIdx.x >> 3), rank = -1;
  const auto next = [&](typename G::Spot* s) {  // the same in all waves, and none is in the table's use when it is built
    for (; b < end; b += stride) {
      if (G::locate(a, b, s, [&](int r, int slot) {
            if (!a.counts) return find_group<false>(nullptr, a.G, a.rows, 256, slot, a.err);
            if (r != rank) {
              rank = r;
              __syncthreads();
              if (wave == 0) table.build(a.counts + (size_t)r * a.G, a.G, a.rows, 256, a.err);
              __syncthreads();
            }
            return table.find(a.G, slot);
          }))
        return true;
    }
    return false;
  };
  const int steps = a.K / kK;
  uint32_t oa[G::kPA], ob[G::kPB];
  const auto issue = [&](const typename G::Where& t, float* to) {
    G::fetch_scales(t, tid, wave, to);
    G::offsets(t, tid, oa, ob);
    if (steps > 0) G::fetch(t, 0, tid, wave, oa, ob, s0);
    if (steps > 1) G::fetch(t, kK, tid, wave, oa, ob, s1);
  };
  typename G::Spot at;
  if (!next(&at)) return;
  issue(at.t, scales);
  bool whole = false;  // the tile before was
  for (int flip = 0;; flip ^= 1) {
    const typename G::Where& t = at.t;
    Acc<DT> acc[kNF][kMF];
#pragma unroll
    for (int i = 0; i < kNF; ++i)
#pragma unroll
      for (int j = 0; j < kMF; ++j) acc[i][j] = Acc<DT>{0, 0, 0, 0};
    if (steps > 0) {
      if (steps > 1 && whole) G::template meet<kLoads + kStores>();  // step 0 has landed, all that is older too
      else G::template meet<0>();
      if (wave < 4) G::template phases<true, true>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
      else G::template phases<false, true>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
    }
    if (steps * kK < t.K) {
      v4u ra[G::kPA], rb[G::kPB];
      G::load(t, tid, steps * kK, ra, rb);
      G::store(tid, s0, s0 + G::TA::kBytes, ra, rb);
      wait_vmem();  // the scales too, where no whole step was
      __syncthreads();
      G::multiply(s0, s0 + G::TA::kBytes, wm, wn, lane, acc);
      __syncthreads();
    }
    b += stride;
    typename G::Spot then;
    const bool more = next(&then);
    // every wave is past its reads of the steps, and of the other scales: a tile's barriers lie between
    if (more) issue(then.t, scales + (flip ^ 1) * G::kScales);
    v4f z[kNF][kMF];
    const bool large = G::scaled(scales + flip * G::kScales, wm, wn, lane, acc, z);
    G::template finish<ACT>(a, at, wm, wn, lane, z, large, scales + flip * G::kScales + wm);
    if (!more) return;
    whole = t.m0 + 256 <= t.mEnd && (GATED ? t.n0 / 2 + 128 <= t.O : t.n0 + 256 <= t.N);
    at = then;
  }
}

// Few rows (MT * 16 at a time) against many weights: bound by the weights'
// bytes. A workgroup takes 16 columns of out (gated: 16 of either half), its 8
// waves an eighth of the contraction axis each; weights and rows go straight
// to registers, and the waves' sums meet in the LDS once, at the end. One row of
// 4096 x 4096 bf16 weights: 128-column tiles, of which there are only 32, took
// 45 us.
template <int DT, int ACT, bool GATED, int MT>
__global__ __launch_bounds__(512) void k_few(const GemmArgs a) {
  constexpr int kES = Elem<DT>::kSize, kStep = 4 * Elem<DT>::kChunk, NW = GATED ? 2 : 1, BM = MT * 16;
  constexpr int U = 16 / (NW + MT);  // 64 registers of loads in flight
  __shared__ __align__(16) Acc<DT> part[8][NW][BM][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, q = lane >> 4;
  int b = a.tile0 + blockIdx.x;
  const int slot = b % a.mt;
  b /= a.mt;
  const int c0 = b % a.nt * 16, r = b / a.nt;
  const GroupTile g = find_group<false>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, BM, slot, a.err);
  if (g.g < 0) return;
  const int m0 = (slot - g.tile0) * BM, rows = min(g.count - m0, BM), first = g.first + m0;
  const char *w[NW], *x[MT];
  const int col = min(c0 + i, a.O - 1);
#pragma unroll
  for (int h = 0; h < NW; ++h) w[h] = a.b.p[r] + ((uint64_t)g.g * a.b_group + (uint64_t)(h * a.O + col) * a.ldb) * kES;
#pragma unroll
  for (int j = 0; j < MT; ++j) x[j] = a.a.p[r] + (uint64_t)(first + min(j * 16 + i, rows - 1)) * a.lda * kES;
  Acc<DT> z[NW][MT];
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j) z[h][j] = Acc<DT>{0, 0, 0, 0};
  // what the epilogue reads, in 8 bits, on its way with the weights: one latency less
  const int m = tid >> 2, p = tid & 3;
  [[maybe_unused]] float sx = 0.0f, sw[NW][4], bias[NW][4], res[4];
  if constexpr (kInt8<DT>) {
    constexpr int kOut = kOutOf<DT>;
    if (m < rows) {
      const int at = c0 + p * 4, n = a.O - at;
      sx = *reinterpret_cast<const float*>(a.a.p[r] + (uint64_t)(first + m + 1) * a.lda - 4);
#pragma unroll
      for (int h = 0; h < NW; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t row = (uint64_t)g.g * a.N + h * a.O + min(at + j, a.O - 1);
          sw[h][j] = *reinterpret_cast<const float*>(a.b.p[r] + (row + 1) * a.ldb - 4);
        }
        if (a.bias.p[r]) load4<kOut>(a.bias.p[r], (uint64_t)g.g * a.N + h * a.O + at, n, bias[h]);
      }
      if (a.residual.p[r]) load4<kOut>(a.residual.p[r], (uint64_t)(first + m) * a.O + at, n, res);
    }
  }
  const int per = (a.K + 8 * kStep - 1) / (8 * kStep) * kStep;
  stream_products<DT, NW, MT, U>(w, x, wave * per, min(a.K, (wave + 1) * per), a.K, z);
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][h][j * 16 + i][q] = z[h][j];
  __syncthreads();
  if (m >= rows) return;
  Acc<DT> s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int v = 0; v < 8; ++v) s[h] += part[v][h][m][p];
  if constexpr (kInt8<DT>) {
    const int n = a.O - (c0 + p * 4);
    if (n <= 0) return;
    float y[4];
    const RowScale by(sx);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float z[NW];
#pragma unroll
      for (int h = 0; h < NW; ++h) {
        z[h] = by(s[h][j], sw[h][j]);
        if (a.bias.p[r]) z[h] += bias[h][j];
      }
      y[j] = act_value<kOutOf<DT>, ACT>(z[0]);
      if (GATED) y[j] *= z[NW - 1];
      if (a.residual.p[r]) y[j] += res[j];
    }
    store4<kOutOf<DT>>(a.out.p[r], (uint64_t)(first + m) * a.O + c0 + p * 4, n, y);
  } else {
    epilogue<DT, ACT, GATED>(a, r, g.g, first + m, c0 + p * 4, s[0], s[1]);
  }
}

// A launch holds fewer than 2^32 threads in a direction; 2^22 workgroups of up to
// 512 do. More tiles (a thousand groups of 128 thousand columns, say) take more
// launches: launch(workgroups) with a.tile0 set, a multiple of 8 for xcd_order.
template <class F>
vrResult_t launch_parts(GemmArgs& a, uint64_t tiles, F launch) {
  constexpr uint64_t kMost = 1u << 22;
  if (tiles > 0x7FFFFFFFull) return VR_ERR_INVALID_ARGUMENT;
  for (uint64_t at = 0; at < tiles; at += kMost) {
    a.tile0 = static_cast<int>(at);
    launch(dim3(static_cast<uint32_t>(std::min(tiles - at, kMost))));
  }
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

template <int DT, int ACT, bool GATED, int MT>
vrResult_t launch_few(GemmArgs& a, hipStream_t st) {
  a.mt = a.counts ? a.rows / (MT * 16) + a.G : (a.rows + MT * 16 - 1) / (MT * 16);
  a.nt = (a.O + 15) / 16;
  return launch_parts(a, (uint64_t)a.R * a.mt * a.nt, [&](dim3 grid) {
    hipLaunchKernelGGL((k_few<DT, ACT, GATED, MT>), grid, dim3(512), 0, st, a);
  });
}

// Whether every row of the present parts of both operands starts on 16 bytes.
bool rows_aligned(const GemmArgs& a, int es) {
  uintptr_t v = (a.lda * es) | (a.ldb * es) | (a.b_group * es);
  for (int r = 0; r < a.R; ++r) v |= reinterpret_cast<uintptr_t>(a.a.p[r]) | reinterpret_cast<uintptr_t>(a.b.p[r]);
  return v % 16 == 0;
}

template <int DT, int MODE, int ACT, bool GATED, bool DIRECT, int BM, int BN, int WM, int WN, int STAGES>
vrResult_t launch_tiles(GemmArgs& a, hipStream_t st) {
  if (MODE == kDw) a.mt = (a.M + BM - 1) / BM;
  else a.mt = a.counts ? a.rows / BM + a.G : (a.rows + BM - 1) / BM;
  a.nt = GATED ? (a.O + BN / 2 - 1) / (BN / 2) : (a.N + BN - 1) / BN;
  return launch_parts(a, (uint64_t)a.R * (MODE == kDw ? a.G : 1) * a.mt * a.nt, [&](dim3 grid) {
    hipLaunchKernelGGL((k_gemm<DT, MODE, ACT, GATED, DIRECT, BM, BN, WM, WN, STAGES>), grid,
                       dim3(64 * (BM / WM) * (BN / WN)), 0, st, a);
  });
}

template <int DT, int ACT, bool GATED>
vrResult_t launch_run(GemmArgs& a, hipStream_t st) {
  a.mt = a.counts ? a.rows / 256 + a.G : (a.rows + 255) / 256;
  a.nt = GATED ? (a.O + 127) / 128 : (a.N + 255) / 256;
  const uint64_t tiles = (uint64_t)a.R * a.mt * a.nt;
  if (tiles > 0x7FFFFFFFull - 256) return VR_ERR_INVALID_ARGUMENT;
  hipLaunchKernelGGL((k_gemm_run<DT, ACT, GATED>), dim3(256), dim3(512), 0, st, a, static_cast<int>(tiles));
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

// Tiles of size n x n to expect: a group's last row tile is half empty.
template <int MODE, bool GATED>
uint64_t expected_tiles(const GemmArgs& a, int n) {
  const uint64_t cols = GATED ? (a.O + n / 2 - 1) / (n / 2) : (a.N + n - 1) / n;
  if (MODE == kDw) return (uint64_t)a.R * a.G * ((a.M + n - 1) / n) * cols;
  return a.R * (a.counts ? (uint64_t)a.rows / n + (a.G + 1) / 2 : (a.rows + n - 1) / n) * cols;
}

// The tile. 256 x 256 tiles take a compute unit each, 128 x 128 tiles share
// one by two; a round of the latter, half the products, takes 0.59 of a round
// of the former (81 and 137 us of 8192 x 4096 x 4096 bf16), and whichever
// needs the less time in whole rounds is taken. 128 x 128 tiles need to give
// every compute unit one; below that, bf16 4096 x 4096 weights take at 128,
// 512, 1024 rows: 64 x 64 tiles with two steps in the LDS 34, 42, 62 us, with
// three 23, 42, 79; 128 x 128 tiles 50, 52, 56. By expert the rule counts the
// rows' capacity, since the used rows are known on the device alone: 16384 rows
// of 8 groups, 1024 -> 512 gated bf16, take 71 us where they fill it and 241 where
// they fill an eighth (the tiles' order gives each XCD a part of the capacity,
// so the used ones are on few of them). Nothing splits the contraction: dw of
// 300 x 300 fp32 weights over 4096 rows, 25 tiles, takes 109 us.
template <int DT, int MODE, int ACT, bool GATED, bool DIRECT>
vrResult_t launch_any(GemmArgs& a, hipStream_t st) {
  const uint64_t n128 = expected_tiles<MODE, GATED>(a, 128);
  if constexpr (DT != VR_DT_F32 && DIRECT) {
    const uint64_t n256 = expected_tiles<MODE, GATED>(a, 256);
    if ((n256 + 255) / 256 * 100 <= (n128 + 511) / 512 * 59) {
      if constexpr (kInt8<DT>) return launch_run<DT, ACT, GATED>(a, st);
      else return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 256, 256, 128, 64, 2>(a, st);
    }
  }
  // Experts of few rows each in 8 bits are bound by the weights' bytes: 64 x 128 tiles
  // with three steps in the LDS take 83, 92, 94 us at 32, 128, 256 rows of 32
  // experts on 8 ranks, 2048 -> 512 gated; 64 x 64 ones 86, 94, 96, 128 x 128 ones
  // 94, 98, 100.
  if constexpr (kInt8<DT> && DIRECT) {
    if (a.G > 1 && a.rows / a.G < 64) return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 64, 128, 32, 64, 3>(a, st);
  }
  if (n128 >= 256) return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 128, 128, 64, 64, 2>(a, st);
  if constexpr (DIRECT) {
    if (expected_tiles<MODE, GATED>(a, 64) <= 512)
      return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 64, 64, 32, 32, 3>(a, st);
  }
  return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 64, 64, 32, 32, 2>(a, st);
}

template <int DT, int MODE, int ACT, bool GATED>
vrResult_t launch_gemm(GemmArgs& a, hipStream_t st) {
  if constexpr (MODE == kFwd) {
    // Few rows: against 64 x 64 tiles, us at 1, 32, 64 rows of bf16 4096 x 4096
    // weights 11, 15, 25 to 22; at 64, 256 rows of fp32 2048 x 2048 weights, whose
    // tiles are bound by the matrix units, 16, 47 to 45. Groups are ragged.
    // 8 bits: of a single group alone, at 32, 64 rows of 4096 x 4096 weights 10, 15 to
    // 14.4, 14.5, at 64, 128 rows of 2048 x 2048 weights 7.2, 11 to 9.5, 9.6; by expert
    // tiles are as fast from the first row on (8 x 32 rows of 32 experts, 2048 ->
    // 512 gated: 98 to 83).
    const int few8 = a.G > 1 ? -1 : (uint64_t)a.N * a.K <= 4u << 20 ? 64 : 32;
    const int most = kInt8<DT> ? few8 : (DT == VR_DT_F32 ? 128 : 32) / (a.G > 1 ? 2 : 1), rows = a.rows / a.G;
    if (rows <= 16 && rows <= most) return launch_few<DT, ACT, GATED, 1>(a, st);
    if (rows <= most) return launch_few<DT, ACT, GATED, 2>(a, st);
  }
  return rows_aligned(a, Elem<DT>::kSize) ? launch_any<DT, MODE, ACT, GATED, true>(a, st)
                                          : launch_any<DT, MODE, ACT, GATED, false>(a, st);
}

}  // namespace
}  // namespace vr
