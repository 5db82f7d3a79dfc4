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
  uint32_t act;
};

// A tile of ROWS rows and 128 bytes of the contraction axis, or of 128 bytes'
// elements of the contraction axis and ROWS columns, in 16-byte pieces:
//   KC (the contraction axis is contiguous): piece c of row r at position
//      c ^ (r & 7) of the row's 128 bytes, so that the 16 rows of a fragment
//      read fall on all banks;
//   otherwise rows of ROWS columns per k; pieces are exchanged so that the 4
//      rows (bf16) or the 4 row quarters (fp32) of one read do.
template <int DT, bool KC, int ROWS>
struct Tile {
  static constexpr int kK = 128 / Elem<DT>::kSize;       // contraction elements
  static constexpr int kC = Elem<DT>::kChunk;
  static constexpr int kBytes = ROWS * 128;
  static constexpr int kPieces = ROWS * 8;
  static constexpr int kPerRow = KC ? 8 : ROWS / kC;     // pieces per stored row
  __device__ static int swz(int r) {
    if constexpr (KC) return r & 7;
    else if constexpr (DT == VR_DT_BF16) return (r & 3) << 1;
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

template <int DT>
__device__ inline void epilogue(const GemmArgs& a, int r, int g, int row, int col, v4f z0, v4f z1, bool gated) {
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
    y[j] = act_value(g4[j], a.act);
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

// One BM x BN tile of out per workgroup; the waves' WM x WN parts stay in
// registers. The matrix instructions take the b side (columns of out) as
// their first operand, so a lane's four sums are four consecutive columns of
// one row of out.
template <int DT, int MODE, bool GATED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_gemm(const GemmArgs a) {
  constexpr int kThreads = 64 * (BM / WM) * (BN / WN);
  using TA = Tile<DT, MODE != kDw, BM>;
  using TB = Tile<DT, MODE == kFwd, BN>;
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kK = TA::kK;
  __shared__ __align__(16) char la[TA::kBytes];
  __shared__ __align__(16) char lb[TB::kBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave % (BM / WM)) * WM, wn = (wave / (BM / WM)) * WN;

  // the tile: rank, group, rows and columns
  int b = blockIdx.x;
  const int nti = b % a.nt;
  b /= a.nt;
  int r, g, m0, mEnd, row0, K;
  if constexpr (MODE == kDw) {
    const int mti = b % a.mt;
    b /= a.mt;
    g = b % a.G;
    r = b / a.G;
    const GroupTile t = find_group<true>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, 1, g, a.err);
    row0 = t.first;
    K = t.count;
    m0 = mti * BM;
    mEnd = a.M;
  } else {
    const int slot = b % a.mt;
    r = b / a.mt;
    const GroupTile t = find_group<false>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, BM, slot, a.err);
    if (t.g < 0) return;
    g = t.g;
    row0 = t.first;
    K = a.K;
    m0 = (slot - t.tile0) * BM;
    mEnd = t.count;
  }
  const int n0 = nti * BN;  // tile's first column of b; gated: BN / 2 columns of either half
  const char* pa = a.a.p[r] + (uint64_t)row0 * a.lda * kES;
  const char* pb = a.b.p[r] + (MODE == kDw ? (uint64_t)row0 * a.ldb : (uint64_t)g * a.b_group) * kES;

  v4f acc[WN / 16][WM / 16];
#pragma unroll
  for (int i = 0; i < WN / 16; ++i)
#pragma unroll
    for (int j = 0; j < WM / 16; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  for (int k0 = 0; k0 < K; k0 += kK) {
    // stage: registers, then LDS
#pragma unroll
    for (int i = 0; i < TA::kPieces / kThreads; ++i) {
      const int id = i * kThreads + tid, sr = id / TA::kPerRow, c = (id % TA::kPerRow) ^ TA::swz(sr);
      v4u v;
      if constexpr (MODE != kDw) {
        const int m = m0 + sr, k = k0 + c * kC;
        v = load_piece<DT>(pa + ((uint64_t)m * a.lda + k) * kES, m < mEnd ? K - k : 0);
      } else {
        const int k = k0 + sr, m = m0 + c * kC;
        v = load_piece<DT>(pa + ((uint64_t)k * a.lda + m) * kES, k < K ? mEnd - m : 0);
      }
      *reinterpret_cast<v4u*>(la + (id << 4)) = v;
    }
#pragma unroll
    for (int i = 0; i < TB::kPieces / kThreads; ++i) {
      const int id = i * kThreads + tid, sr = id / TB::kPerRow, c = (id % TB::kPerRow) ^ TB::swz(sr);
      v4u v;
      if constexpr (MODE == kFwd) {
        const int k = k0 + c * kC;
        int n = n0 + sr;
        bool in = n < a.N;
        if constexpr (GATED) {  // 16 gate columns, then the same 16 of the other half
          const int o = n0 / 2 + (sr >> 5) * 16 + (sr & 15);
          in = o < a.O;
          n = o + ((sr >> 4) & 1) * a.O;
        }
        v = load_piece<DT>(pb + ((uint64_t)n * a.ldb + k) * kES, in ? K - k : 0);
      } else {
        const int k = k0 + sr, n = n0 + c * kC;
        v = load_piece<DT>(pb + ((uint64_t)k * a.ldb + n) * kES, k < K ? a.N - n : 0);
      }
      *reinterpret_cast<v4u*>(lb + (id << 4)) = v;
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v4u fa[WM / 16], fb[WN / 16];
#pragma unroll
      for (int j = 0; j < WM / 16; ++j) fa[j] = TA::frag(la, wm + j * 16, ks, lane);
#pragma unroll
      for (int i = 0; i < WN / 16; ++i) fb[i] = TB::frag(lb, wn + i * 16, ks, lane);
#pragma unroll
      for (int i = 0; i < WN / 16; ++i)
#pragma unroll
        for (int j = 0; j < WM / 16; ++j) acc[i][j] = mfma_piece<DT>(fb[i], fa[j], acc[i][j]);
    }
    __syncthreads();
  }

  const int cq = (lane >> 4) * 4;
#pragma unroll
  for (int j = 0; j < WM / 16; ++j) {
    const int m = m0 + wm + j * 16 + (lane & 15);
    if (m >= mEnd) continue;
#pragma unroll
    for (int i = 0; i < WN / 16; i += GATED ? 2 : 1) {
      if constexpr (MODE == kFwd) {
        const int col = GATED ? n0 / 2 + (wn + i * 16) / 2 + cq : n0 + wn + i * 16 + cq;
        epilogue<DT>(a, r, g, row0 + m, col, acc[i][j], acc[i + (GATED ? 1 : 0)][j], GATED);
      } else {
        const int col = n0 + wn + i * 16 + cq;
        float y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = acc[i][j][q];
        const uint64_t row = MODE == kDw ? (uint64_t)m : (uint64_t)(row0 + m);
        store4<DT>(a.out.p[r] + (uint64_t)g * a.out_group * kES, row * a.N + col, a.N - col, y);
      }
    }
  }
}

template <int DT, int MODE, bool GATED>
vrResult_t launch_gemm(GemmArgs& a, hipStream_t st) {
  constexpr int BM = 128, BN = 128;
  if (MODE == kDw) a.mt = (a.M + BM - 1) / BM;
  else a.mt = a.counts ? a.rows / BM + a.G : (a.rows + BM - 1) / BM;
  a.nt = GATED ? (a.O + BN / 2 - 1) / (BN / 2) : (a.N + BN - 1) / BN;
  const uint64_t grid = (uint64_t)a.R * (MODE == kDw ? a.G : 1) * a.mt * a.nt;
  if (!grid) return VR_OK;
  if (grid > 0x7FFFFFFFull) return VR_ERR_INVALID_ARGUMENT;
  hipLaunchKernelGGL((k_gemm<DT, MODE, GATED, BM, BN, 64, 64>), dim3(static_cast<uint32_t>(grid)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
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

// A workgroup takes kDzRows rows of one group and 64 * V columns; its four
// waves take every fourth row.
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
  for (int i = first + wave; i < last && n > 0; i += 4) {
    const uint64_t row = t.first + i;
    float d[V], g[V], u[V];
    auto get = [&](const char* base, uint64_t at, float* f) {
      if (n >= V) {
        load_n<DT, V>(base, at, f);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = j < n ? Elem<DT>::load(base, at + j) : 0.0f;
      }
    };
    auto put = [&](uint64_t at, const float* f) {
      char* base = a.dz + (uint64_t)r * a.dz_rank;
      if (n >= V) {
        store_n<DT, V>(base, at, f);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j < n) Elem<DT>::store(base, at + j, f[j]);
      }
    };
    get(a.dout.p[r], row * a.O + col, d);
    if (a.preact.p[r]) {
      get(a.preact.p[r], row * a.N + col, g);
      if (GATED) get(a.preact.p[r], row * a.N + a.O + col, u);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float y, s;
        act_both(g[j], a.act, &y, &s);
        if (GATED) {
          g[j] = d[j] * u[j] * s;
          u[j] = d[j] * y;
        } else {
          g[j] = d[j] * s;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = d[j];
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

// dbias[g][n]: the group's row tiles in order.
template <int DT>
__global__ __launch_bounds__(256) void k_dbias(const DzArgs a) {
  const int r = blockIdx.z, g = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  const GroupTile t = find_group<true>(a.counts ? a.counts + (size_t)r * a.G : nullptr, a.G, a.rows, kDzRows, g, a.err);
  if (n >= a.N) return;
  const int tiles = (t.count + kDzRows - 1) / kDzRows;
  const float* p = a.partial + ((uint64_t)r * a.slots + t.tile0) * a.N + n;
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < tiles; ++i) s += p[(uint64_t)i * a.N];
  Elem<DT>::store(a.dbias.p[r], (uint64_t)g * a.N + n, s);
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
  a.act = s.act;
  return gated(s) ? launch_gemm<DT, kFwd, true>(a, st) : launch_gemm<DT, kFwd, false>(a, st);
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
  if (z.partial) hipLaunchKernelGGL((k_dbias<DT>), dim3((N + 255) / 256, s.groups, R), dim3(256), 0, st, z);
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
    const vrResult_t e = launch_gemm<DT, kDx, false>(a, st);
    if (e != VR_OK) return e;
  }
  if (dw.window) {
    a.b = slice_tab(x);
    a.out = slice_tab(dw);
    a.out_group = (uint64_t)N * s.in;
    a.M = N;
    const vrResult_t e = launch_gemm<DT, kDw, false>(a, st);
    if (e != VR_OK) return e;
  }
  return VR_OK;
}

}  // namespace

size_t linear_workspace_bytes(int, const vrLinearShape&) { return 0; }
size_t linear_backward_workspace_bytes(int R, const vrLinearShape& s) { return backward_layout(R, s).total; }

vrResult_t launch_linear(vrComm* c, const vrLinearShape& s, const vrSlice& x, const vrSlice& w, const vrSlice& bias,
                         const vrSlice& residual, const int32_t* group_rows, const vrSlice& out,
                         const vrSlice& preact, char*, hipStream_t st) {
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
