// Gradient of the MoE combine (vr_combine_backward). The combine mixes
//   out[s][t] = sum over k of weights[s][t][k] * y[d][p]
// with p = send_pos[s][t][k] the entry's row at rank d = expert / (E/R), so
//   dy[d][p] = weights[s][t][k] * dout[s][t]     (a put to the row's rank)
//   dweights[s][t][k] = dout[s][t] . y[d][p]     (a get from it)
//
// Bound by memory: for each entry one row is read and one written; a token's
// own row is read once for up to kBatch entries. A group of 2^LOG lanes takes a
// token; all its entries' loads of a column chunk are in flight together.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {

constexpr int kBatch = 8;  // entries of a token at a time

struct GradArgs {
  WinTab dout, y, dy;
  const int32_t *topk, *pos;  // [R][T][K]
  const float* weights;
  float* dweights;            // or null
  uint32_t* err;
  uint64_t row_bytes, cap;
  int R, T, K, per, E;        // per: experts of a rank
};

template <int DT, int LOG>
__global__ __launch_bounds__(256) void k_combine_back(const GradArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kL = 1 << LOG, kTok = 256 / kL;
  const int s = blockIdx.x % a.R, l = threadIdx.x & (kL - 1);
  const int t = blockIdx.x / a.R * kTok + threadIdx.x / kL;
  if (t >= a.T) return;
  const int H = static_cast<int>(a.row_bytes / Elem<DT>::kSize);
  const char* d = a.dout.p[s] + (uint64_t)t * a.row_bytes;
  const uint64_t e0 = ((uint64_t)s * a.T + t) * a.K;
  const bool whole = H % kC == 0;
  for (int k0 = 0; k0 < a.K; k0 += kBatch) {
    const int n = min(kBatch, a.K - k0);
    uint64_t at[kBatch];  // the entry's row: byte offset in its rank's part, all ones without one
    int rank[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const uint64_t g = e0 + k0 + min(q, n - 1);
      const int e = a.topk[g], p = a.pos[g];
      w[q] = a.weights[g];
      at[q] = ~0ull;
      rank[q] = 0;
      dot[q] = 0.0f;
      if (q >= n) continue;
      if (e != -1 && (e < 0 || e >= a.E)) {
        if (l == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_EXPERT);
      } else if (e >= 0 && p != -1) {
        if (p < 0 || (uint64_t)p >= a.cap) {
          if (l == 0) atomic_or_u32(a.err, VR_ASYNC_CAPACITY);
        } else {
          at[q] = (uint64_t)p * a.row_bytes;
          rank[q] = e / a.per;
        }
      }
    }
    for (int col = l * kC; col < H; col += kL * kC) {
      const uint64_t off = (uint64_t)col * Elem<DT>::kSize;
      const v4u dv = whole ? load_whole<DT>(d + off) : load_piece<DT>(d + off, H - col);
      v4u yv[kBatch];
      if (a.dweights) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          yv[q] = v4u{0, 0, 0, 0};
          if (at[q] != ~0ull) {
            const char* p = a.y.p[rank[q]] + at[q] + off;
            yv[q] = whole ? load_whole<DT>(p) : load_piece<DT>(p, H - col);
          }
        }
      }
      float f[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) f[j] = piece_f32<DT>(dv, j);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (at[q] == ~0ull) continue;
        if (a.dweights) {
#pragma unroll
          for (int j = 0; j < kC; ++j) dot[q] = fmaf(f[j], piece_f32<DT>(yv[q], j), dot[q]);
        }
        if (a.dy.p[0]) {
          float g[kC];
#pragma unroll
          for (int j = 0; j < kC; ++j) g[j] = w[q] * f[j];
          char* p = a.dy.p[rank[q]] + at[q];
          if (H - col >= kC) {
            store_n<DT, kC>(p, col, g);
          } else {
#pragma unroll
            for (int j = 0; j < kC - 1; ++j)
              if (j < H - col) Elem<DT>::store(p, col + j, g[j]);
          }
        }
      }
    }
    if (a.dweights) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const float v = lane_reduce<LOG>(dot[q], [](float x, float y) { return x + y; });
        if (l == 0 && q < n) a.dweights[e0 + k0 + q] = v;
      }
    }
  }
}

template <int DT, int LOG>
vrResult_t start(const GradArgs& a, hipStream_t st) {
  constexpr int kTok = 256 >> LOG;
  hipLaunchKernelGGL((k_combine_back<DT, LOG>), dim3(a.R * ((a.T + kTok - 1) / kTok)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}
template <int DT>
vrResult_t start_any(const GradArgs& a, hipStream_t st) {
  const uint64_t pieces = (a.row_bytes + 15) / 16;
  if (pieces <= 8) return start<DT, 3>(a, st);
  if (pieces <= 16) return start<DT, 4>(a, st);
  if (pieces <= 32) return start<DT, 5>(a, st);
  return start<DT, 6>(a, st);
}

}  // namespace

vrResult_t launch_combine_backward(vrComm* c, const vrSlice& dout, const vrSlice& y, size_t cap, size_t row_bytes,
                                   int dtype, const int32_t* topk, const float* weights, const int32_t* pos, int T,
                                   int K, int E, const vrSlice& dy, float* dweights, hipStream_t st) {
  GradArgs a = {};
  a.dout = slice_tab(dout);
  a.y = slice_tab(y);
  a.dy = slice_tab(dy);
  a.topk = topk;
  a.pos = pos;
  a.weights = weights;
  a.dweights = dweights;
  a.err = c->err;
  a.row_bytes = row_bytes;
  a.cap = cap;
  a.R = c->nranks;
  a.T = T;
  a.K = K;
  a.E = E;
  a.per = E / c->nranks;
  return dtype == VR_DT_F32 ? start_any<VR_DT_F32>(a, st) : start_any<VR_DT_BF16>(a, st);
}

}  // namespace vr
