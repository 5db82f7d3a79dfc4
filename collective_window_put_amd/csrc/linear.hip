// Matrix products with their epilogues over window rows, dense or by expert:
// vr_linear and vr_linear_backward.
//
//   forward   z = x w^T + bias;  out = act(z) (gated: act(z_g) * z_u) + residual
//   backward  dz = dout * act'(z) (gated: [dout z_u act'(z_g), dout act(z_g)]);
//             dx = dz w;  dw = dz^T x;  dbias = sum over rows of dz
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_gemm.hpp"

namespace vr {
namespace {

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
