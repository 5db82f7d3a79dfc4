// Matrix products with their epilogues over window rows, dense or by expert:
// vr_linear and vr_linear_backward.
//
//   forward   z = x w^T + bias;  out = act(z) (gated: act(z_g) * z_u) + residual
//   backward  dz = dout * act'(z) (gated: [dout z_u act'(z_g), dout act(z_g)]);
//             dx = dz w;  dw = dz^T x;  dbias = sum over rows of dz
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

template <int DT, int ACT, bool gated>
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

// Epilogue of a wave's part of a tile that has all its columns: NF x MF
// fragments from column c0 and row m0 (of the group; rows up to mEnd). Loads
// are issued many rows ahead: out might be residual's own slice, so the
// compiler keeps their order, and a fragment at a time each load's latency was
// waited for in turn (82 of the 300 us of a dense 8192 x 4096 x 4096
// product).
template <int DT, int ACT, bool GATED, int NF, int MF>
__device__ inline void epilogue_whole(const GemmArgs& a, int r, int g, int row0, int m0, int mEnd, int c0, int lane,
                                      const v4f (*acc)[MF]) {
  constexpr int kES = Elem<DT>::kSize, NO = GATED ? NF / 2 : NF, S = GATED ? 2 : 1;
  const int m1 = m0 + (lane & 15), col = c0 + (lane >> 4) * 4;
  // rows whose residual is held at once: all of a small tile's, 32 registers
  constexpr int kRows = MF <= 4 ? MF : 4;
  typename Raw4<DT>::T bias[NO][S], res[kRows][NO];
  const char* pb = a.bias.p[r];
  const char* pr = a.residual.p[r];
  char* pz = a.preact.p[r];
  if (pb) {
    pb += ((uint64_t)g * a.N + col) * kES;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int h = 0; h < S; ++h) bias[i][h] = load_raw4<DT>(pb + (uint64_t)(h * a.O + i * 16) * kES);
  }
#pragma unroll
  for (int j0 = 0; j0 < MF; j0 += kRows) {
    if (pr) {
#pragma unroll
      for (int v = 0; v < kRows; ++v)
#pragma unroll
        for (int i = 0; i < NO; ++i)
          res[v][i] = load_raw4<DT>(pr + ((uint64_t)(row0 + min(m1 + (j0 + v) * 16, mEnd - 1)) * a.O + col + i * 16) * kES);
    }
#pragma unroll
    for (int v = 0; v < kRows; ++v) {
      const uint64_t row = row0 + m1 + (j0 + v) * 16;
      if (m1 + (j0 + v) * 16 < mEnd) {
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          float z[S][4], y[4];
#pragma unroll
          for (int h = 0; h < S; ++h) {
#pragma unroll
            for (int q = 0; q < 4; ++q) z[h][q] = acc[i * S + h][j0 + v][q];
            if (pb) {
              const v4f f = from_raw4<DT>(bias[i][h]);
#pragma unroll
              for (int q = 0; q < 4; ++q) z[h][q] += f[q];
            }
            if (pz) store_n<DT, 4>(pz, row * a.N + h * a.O + col + i * 16, z[h]);
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
          store_n<DT, 4>(a.out.p[r], row * a.O + col + i * 16, y);
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
  // ranks. False when there is no such tile.
  __device__ static __forceinline__ bool locate(const GemmArgs& a, int b, Spot* s) {
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
      const GroupTile q = find_group<false>(a.counts ? a.counts + (size_t)s->r * a.G : nullptr, a.G, a.rows, BM, slot, a.err);
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

  template <int ACT>
  __device__ static __forceinline__ void finish(const GemmArgs& a, const Spot& s, int wm, int wn, int lane, const v4f (*acc)[kMF]) {
    const Where& t = s.t;
    if constexpr (MODE == kFwd) {
      if (GATED ? t.n0 / 2 + BN / 2 <= a.O : t.n0 + BN <= a.N) {
        epilogue_whole<DT, ACT, GATED, kNF, kMF>(a, s.r, s.g, s.row0, t.m0 + wm, t.mEnd, GATED ? (t.n0 + wn) / 2 : t.n0 + wn, lane, acc);
        return;
      }
    }
    const int cq = (lane >> 4) * 4;
#pragma unroll
    for (int j = 0; j < kMF; ++j) {
      const int m = t.m0 + wm + j * 16 + (lane & 15);
      if (m >= t.mEnd) continue;
#pragma unroll
      for (int i = 0; i < kNF; i += GATED ? 2 : 1) {
        if constexpr (MODE == kFwd) {
          const int col = GATED ? t.n0 / 2 + (wn + i * 16) / 2 + cq : t.n0 + wn + i * 16 + cq;
          epilogue<DT, ACT, GATED>(a, s.r, s.g, s.row0 + m, col, acc[i][j], acc[i + (GATED ? 1 : 0)][j]);
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

  // Row of b behind tile row j (forward): gated, 16 gate columns, then the same 16 of the other half.
  __device__ static __forceinline__ int b_row(const Where& t, int j, bool* in) {
    if constexpr (GATED) {
      const int o = t.n0 / 2 + (j >> 5) * 16 + (j & 15);
      *in = o < t.O;
      return o + ((j >> 4) & 1) * t.O;
    } else {
      *in = t.n0 + j < t.N;
      return t.n0 + j;
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
  __device__ static __forceinline__ void products(const v4u* fa, const v4u* fb, v4f (*acc)[kMF]) {
#pragma unroll
    for (int j = 0; j < kMF; ++j)
#pragma unroll
      for (int i = 0; i < kNF; ++i) acc[i][j] = mfma_piece<DT>(fb[i], fa[j], acc[i][j]);
  }
  __device__ static __forceinline__ void multiply(const char* la, const char* lb, int wm, int wn, int lane, v4f (*acc)[kMF]) {
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
  __device__ static __forceinline__ void step(const Where& t, int k1, int tid, const char* cur, char* nxt, int wm, int wn, int lane, v4f (*acc)[kMF]) {
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
                                              const uint32_t* ob, char* s, int wm, int wn, int lane, v4f (*acc)[kMF]) {
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
  template <bool FIRST>
  __device__ static __forceinline__ void phases(const Where& t, int steps, int tid, int wave, const uint32_t* oa,
                                                const uint32_t* ob, char* s0, char* s1, int wm, int wn, int lane,
                                                v4f (*acc)[kMF]) {
    if (!FIRST) {
      if (steps > 1) fetch(t, kK, tid, wave, oa, ob, s1);
      barrier();
    }
    for (int i = 0; i < steps; ++i) {
      char* cur = (i & 1) ? s1 : s0;
      char* nxt = (i & 1) ? s0 : s1;
      v4u fa[kMF], fb[kNF];
      if (FIRST && i + 1 < steps) fetch(t, (i + 1) * kK, tid, wave, oa, ob, nxt);
      frags(cur, cur + TA::kBytes, 0, wm, wn, lane, fa, fb);
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
      if (!FIRST && i + 2 < steps) fetch(t, (i + 2) * kK, tid, wave, oa, ob, cur);
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
  __shared__ __align__(16) char s0[G::kStages * G::kStage];
  char* s1 = s0 + G::kStage;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave % (BM / WM)) * WM, wn = (wave / (BM / WM)) * WN;
  typename G::Spot at;
  if (!G::locate(a, a.tile0 + xcd_order(blockIdx.x, gridDim.x), &at)) return;
  const typename G::Where& t = at.t;

  v4f acc[kNF][kMF];
#pragma unroll
  for (int i = 0; i < kNF; ++i)
#pragma unroll
    for (int j = 0; j < kMF; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  // whole steps (DIRECT; the others zero-fill and take every step here)
  const int steps = DIRECT ? t.K / kK : (t.K + kK - 1) / kK;
  if (steps > 0) {
    if constexpr (DIRECT) {
      uint32_t oa[G::kPA], ob[G::kPB];
      G::offsets(t, tid, oa, ob);
      if constexpr (G::kThreads == 512) {
        G::fetch(t, 0, tid, wave, oa, ob, s0);
        G::meet();
        if (wave < 4) G::template phases<true>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
        else G::template phases<false>(t, steps, tid, wave, oa, ob, s0, s1, wm, wn, lane, acc);
      } else {
        G::ring(t, steps, tid, wave, oa, ob, s0, wm, wn, lane, acc);
      }
    } else {
      v4u ra[G::kPA], rb[G::kPB];
      G::load(t, tid, 0, ra, rb);
      G::store(tid, s0, s0 + G::TA::kBytes, ra, rb);
      __syncthreads();
      for (int i = 0; i < steps; ++i)
        G::step(t, (i + 1) * kK, tid, (i & 1) ? s1 : s0, (i & 1) ? s0 : s1, wm, wn, lane, acc);
    }
  }
  if (DIRECT && steps * kK < t.K) {  // the last, partial step: by registers, zero-filled
    v4u ra[G::kPA], rb[G::kPB];
    G::load(t, tid, steps * kK, ra, rb);
    G::store(tid, s0, s0 + G::TA::kBytes, ra, rb);
    __syncthreads();
    G::multiply(s0, s0 + G::TA::kBytes, wm, wn, lane, acc);
  }
  G::template finish<ACT>(a, at, wm, wn, lane, acc);
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
  __shared__ __align__(16) v4f part[8][NW][BM][4];
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
  v4f z[NW][MT];
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j) z[h][j] = v4f{0, 0, 0, 0};
  const int per = (a.K + 8 * kStep - 1) / (8 * kStep) * kStep;
  stream_products<DT, NW, MT, U>(w, x, wave * per, min(a.K, (wave + 1) * per), a.K, z);
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][h][j * 16 + i][q] = z[h][j];
  __syncthreads();
  const int m = tid >> 2, p = tid & 3;
  if (m >= rows) return;
  v4f s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int h = 0; h < NW; ++h)
#pragma unroll
    for (int v = 0; v < 8; ++v) s[h] += part[v][h][m][p];
  epilogue<DT, ACT, GATED>(a, r, g.g, first + m, c0 + p * 4, s[0], s[1]);
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
  if constexpr (DT == VR_DT_BF16 && DIRECT) {
    const uint64_t n256 = expected_tiles<MODE, GATED>(a, 256);
    if ((n256 + 255) / 256 * 100 <= (n128 + 511) / 512 * 59)
      return launch_tiles<DT, MODE, ACT, GATED, DIRECT, 256, 256, 128, 64, 2>(a, st);
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
    const int most = (DT == VR_DT_F32 ? 128 : 32) / (a.G > 1 ? 2 : 1), rows = a.rows / a.G;
    if (rows <= 16 && rows <= most) return launch_few<DT, ACT, GATED, 1>(a, st);
    if (rows <= most) return launch_few<DT, ACT, GATED, 2>(a, st);
  }
  return rows_aligned(a, Elem<DT>::kSize) ? launch_any<DT, MODE, ACT, GATED, true>(a, st)
                                          : launch_any<DT, MODE, ACT, GATED, false>(a, st);
}

// ---- the gradient of z, and of the bias ---------------------------------------------------
constexpr int kDzRows = 32;  // rows per workgroup

struct DzArgs {
  WinTab dout, preact, dbias;
  char* dz;         // [R][rows][ldz], or null: dz is dout
  float* partial;   // [R][slots][N] column sums of each row tile, or null
  const int32_t* counts;
  uint32_t* err;
  int R, G, rows, N, O, slots;
  uint64_t ldz, dz_rank;  // elements per row, bytes per rank
  uint32_t act;
};

// bf16: dz is rounded to bf16 once, since it is an operand of two bf16 products;
// in two bf16 parts it would double them, most of the call's time. Against
// binary64 the gradients are off by 0.0023 (relative, in the norm) where their
// own rounding alone makes 0.0017. The bias' sums take it unrounded.
//
// A workgroup takes kDzRows rows of one group and 64 * V columns; its four
// waves take every fourth row, kAhead rows' loads in flight (64 rows of 4096
// columns, few workgroups: 13.8 us a row at a time, 10.0 this way).
constexpr int kAhead = 4;
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void k_dz(const DzArgs a) {
  constexpr int V = Elem<DT>::kChunk;
  const int r = blockIdx.z, slot = blockIdx.x;
  const GroupTile t = find_group<false>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, kDzRows, slot, a.err);
  if (t.g < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (blockIdx.y * 64 + lane) * V, n = a.O - col;
  const int first = (slot - t.tile0) * kDzRows, last = min(first + kDzRows, t.count);
  float sg[V], su[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sg[j] = su[j] = 0.0f;
  const bool whole = (blockIdx.y + 1) * 64 * V <= static_cast<uint32_t>(a.O);  // the same in all lanes: no branch at a load
  const auto get = [&](const char* base, uint64_t at) {
    const char* q = base + at * Elem<DT>::kSize;
    return whole ? load_whole<DT>(q) : load_piece<DT>(q, n);
  };
  const auto put = [&](uint64_t at, const float* f) {
    char* base = a.dz + (uint64_t)r * a.dz_rank;
    if (n >= V) {
      store_n<DT, V>(base, at, f);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < n) Elem<DT>::store(base, at + j, f[j]);
    }
  };
  for (int i0 = first + wave; i0 < last && n > 0; i0 += 4 * kAhead) {
    v4u dv[kAhead], gv[kAhead], uv[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint64_t row = t.first + min(i0 + 4 * k, last - 1);
      dv[k] = get(a.dout.p[r], row * a.O + col);
      if (a.preact.p[r]) {
        gv[k] = get(a.preact.p[r], row * a.N + col);
        if (GATED) uv[k] = get(a.preact.p[r], row * a.N + a.O + col);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i0 + 4 * k >= last) break;
      const uint64_t row = t.first + i0 + 4 * k;
      float g[V], u[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = piece_f32<DT>(dv[k], j);
        g[j] = d;
        if (a.preact.p[r]) {
          float y, slope;
          act_both<DT>(piece_f32<DT>(gv[k], j), a.act, &y, &slope);
          if (GATED) {
            g[j] = d * piece_f32<DT>(uv[k], j) * slope;
            u[j] = d * y;
          } else {
            g[j] = d * slope;
          }
        }
      }
      if (a.dz) {
        put(row * a.ldz + col, g);
        if (GATED) put(row * a.ldz + a.O + col, u);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sg[j] += g[j];
        if (GATED) su[j] += u[j];
      }
    }
  }
  if (!a.partial) return;
  __shared__ float sum[4][GATED ? 2 : 1][64 * V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    sum[wave][0][lane * V + j] = sg[j];
    if (GATED) sum[wave][GATED ? 1 : 0][lane * V + j] = su[j];
  }
  __syncthreads();
  float* out = a.partial + ((uint64_t)r * a.slots + slot) * a.N;
  for (int i = threadIdx.x; i < 64 * V * (GATED ? 2 : 1); i += 256) {
    const int h = i / (64 * V), c = i % (64 * V), at = blockIdx.y * 64 * V + c;
    if (at < a.O) out[h * a.O + at] = (sum[0][h][c] + sum[1][h][c]) + (sum[2][h][c] + sum[3][h][c]);
  }
}

// dbias[g][n] of 64 columns: four waves sum a quarter of the group's row tiles
// each, in order. (A thread for a whole column, 4096 columns and 128 tiles:
// 7.5 us, bound by the loads' latency; this way about 5.)
template <int DT>
__global__ __launch_bounds__(256) void k_dbias(const DzArgs a) {
  const int r = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x * 64 + lane;
  const GroupTile t = find_group<true>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, kDzRows, g, a.err);
  const int tiles = (t.count + kDzRows - 1) / kDzRows, per = (tiles + 3) / 4, last = min(tiles, (wave + 1) * per);
  const float* p = a.partial + ((uint64_t)r * a.slots + t.tile0) * a.N + min(n, a.N - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int i = wave * per; i < last; ++i) s += p[(uint64_t)i * a.N];
  __shared__ float part[4][64];
  part[wave][lane] = s;
  __syncthreads();
  if (wave || n >= a.N) return;
  Elem<DT>::store(a.dbias.p[r], (uint64_t)g * a.N + n, (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

bool gated(const vrLinearShape& s) { return (s.act & VR_ACT_GATED) != 0; }
int width(const vrLinearShape& s) { return gated(s) ? 2 * s.out : s.out; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct BackwardLayout {
  uint64_t ldz, dz_rank;  // dz rows are padded to 16 bytes
  size_t dz, partial, total;
  int slots;
};
BackwardLayout backward_layout(int R, const vrLinearShape& s) {
  BackwardLayout l;
  const size_t es = s.dtype == VR_DT_F32 ? 4 : 2;
  l.ldz = (width(s) + 16 / es - 1) / (16 / es) * (16 / es);
  l.dz_rank = s.act == VR_ACT_NONE ? 0 : align256((uint64_t)s.rows * l.ldz * es);
  l.slots = s.rows / kDzRows + s.groups;
  l.dz = 0;
  l.partial = R * l.dz_rank;
  l.total = l.partial + align256((size_t)R * l.slots * width(s) * sizeof(float));
  return l;
}

template <int DT>
vrResult_t linear(vrComm* c, const vrLinearShape& s, const vrSlice& x, const vrSlice& w, const vrSlice& bias,
                  const vrSlice& residual, const int32_t* group_rows, const vrSlice& out, const vrSlice& preact,
                  hipStream_t st) {
  GemmArgs a = {};
  a.a = slice_tab(x);
  a.b = slice_tab(w);
  a.bias = slice_tab(bias);
  a.residual = slice_tab(residual);
  a.out = slice_tab(out);
  a.preact = slice_tab(preact);
  a.counts = group_rows;
  a.err = c->err;
  a.R = c->nranks;
  a.G = s.groups;
  a.rows = s.rows;
  a.N = width(s);
  a.K = s.in;
  a.O = s.out;
  a.lda = a.ldb = s.in;
  a.b_group = (uint64_t)a.N * s.in;
  vrResult_t e = VR_OK;
  with_act(s.act, [&](auto act) {
    e = gated(s) ? launch_gemm<DT, kFwd, act(), true>(a, st) : launch_gemm<DT, kFwd, act(), false>(a, st);
  });
  return e;
}

template <int DT>
vrResult_t linear_backward(vrComm* c, const vrLinearShape& s, const vrSlice& dout, const vrSlice& x, const vrSlice& w,
                           const vrSlice& preact, const int32_t* group_rows, const vrSlice& dx, const vrSlice& dw,
                           const vrSlice& dbias, char* ws, hipStream_t st) {
  const BackwardLayout l = backward_layout(c->nranks, s);
  const int R = c->nranks, N = width(s);
  DzArgs z = {};
  z.dout = slice_tab(dout);
  z.preact = slice_tab(s.act == VR_ACT_NONE ? vrSlice{nullptr, 0} : preact);
  z.dbias = slice_tab(dbias);
  z.dz = l.dz_rank && (dx.window || dw.window) ? ws + l.dz : nullptr;
  z.partial = dbias.window ? reinterpret_cast<float*>(ws + l.partial) : nullptr;
  z.counts = group_rows;
  z.err = c->err;
  z.R = R;
  z.G = s.groups;
  z.rows = s.rows;
  z.N = N;
  z.O = s.out;
  z.slots = l.slots;
  z.ldz = l.ldz;
  z.dz_rank = l.dz_rank;
  z.act = s.act;
  if ((z.dz || z.partial) && s.rows) {
    constexpr int kCols = 64 * Elem<DT>::kChunk;
    const dim3 grid(l.slots, (s.out + kCols - 1) / kCols, R);
    if (gated(s)) hipLaunchKernelGGL((k_dz<DT, true>), grid, dim3(256), 0, st, z);
    else hipLaunchKernelGGL((k_dz<DT, false>), grid, dim3(256), 0, st, z);
  }
  if (z.partial) hipLaunchKernelGGL((k_dbias<DT>), dim3((N + 63) / 64, s.groups, R), dim3(256), 0, st, z);
  if (hipGetLastError() != hipSuccess) return VR_ERR_HIP;

  GemmArgs a = {};
  a.a = slice_tab(dout);
  a.lda = s.out;
  if (l.dz_rank) {
    a.lda = l.ldz;
    for (int r = 0; r < R; ++r) a.a.p[r] = ws + l.dz + r * l.dz_rank;
  }
  a.counts = group_rows;
  a.err = c->err;
  a.R = R;
  a.G = s.groups;
  a.rows = s.rows;
  a.N = a.O = s.in;
  a.ldb = s.in;
  if (dx.window) {
    a.b = slice_tab(w);
    a.b_group = (uint64_t)N * s.in;
    a.out = slice_tab(dx);
    a.K = N;
    const vrResult_t e = launch_gemm<DT, kDx, VR_ACT_NONE, false>(a, st);
    if (e != VR_OK) return e;
  }
  if (dw.window) {
    a.b = slice_tab(x);
    a.out = slice_tab(dw);
    a.out_group = (uint64_t)N * s.in;
    a.M = N;
    const vrResult_t e = launch_gemm<DT, kDw, VR_ACT_NONE, false>(a, st);
    if (e != VR_OK) return e;
  }
  return VR_OK;
}

}  // namespace

size_t linear_backward_workspace_bytes(int R, const vrLinearShape& s) { return backward_layout(R, s).total; }

vrResult_t launch_linear(vrComm* c, const vrLinearShape& s, const vrSlice& x, const vrSlice& w, const vrSlice& bias,
                         const vrSlice& residual, const int32_t* group_rows, const vrSlice& out,
                         const vrSlice& preact, hipStream_t st) {
  return s.dtype == VR_DT_F32 ? linear<VR_DT_F32>(c, s, x, w, bias, residual, group_rows, out, preact, st)
                              : linear<VR_DT_BF16>(c, s, x, w, bias, residual, group_rows, out, preact, st);
}

vrResult_t launch_linear_backward(vrComm* c, const vrLinearShape& s, const vrSlice& dout, const vrSlice& x,
                                  const vrSlice& w, const vrSlice& preact, const int32_t* group_rows,
                                  const vrSlice& dx, const vrSlice& dw, const vrSlice& dbias, char* ws,
                                  hipStream_t st) {
  return s.dtype == VR_DT_F32
             ? linear_backward<VR_DT_F32>(c, s, dout, x, w, preact, group_rows, dx, dw, dbias, ws, st)
             : linear_backward<VR_DT_BF16>(c, s, dout, x, w, preact, group_rows, dx, dw, dbias, ws, st);
}

}  // namespace vr
