// Router: softmax over each token's expert logits, the K largest, and the
// gradient.
//
//   p[j] = exp(x[j] - max x) / sum_j exp(x[j] - max x)
//   w[k] = p[e_k], or p[e_k] / sum_k p[e_k]
//   with m = sum_k dw[k] w[k]:  dx[j] = p[j] (sum_{k: e_k = j} dw[k] - m), or
//   renormalized  dx[e_k] = w[k] (dw[k] - m), 0 elsewhere
//
// One wave takes a token. Lane l holds the V = ceil(E / 64) (rounded to a
// power of two) logits of columns l * V ..., so among equal logits the lowest
// lane, and in it the lowest register, is the lowest expert. Each of the K
// rounds takes the wave's maximum, finds its owner with a ballot and removes
// it there; lane k keeps round k's expert.
#include <hip/hip_runtime.h>

#include "vr_layers.hpp"

namespace vr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct RouteArgs {
  WinTab logits, dlogits;
  int32_t* topk;         // [R][T][K]
  float* weights;        // [R][T][K]
  const int32_t* topk_in;
  const float* weights_in;
  const float* dweights;
  uint32_t* err;
  int R, T, K, E, renorm;
  uint32_t tokens;  // R * T
};

// Logits of columns lane * V ... of a row; columns past E are -inf. NaN and
// +inf become -inf (*bad is set).
template <int DT, int V>
__device__ inline void load_logits(const char* row, int E, int lane, float* x, bool* bad) {
  const int c0 = lane * V;
  if (c0 + V <= E) {
    constexpr int N = V < Elem<DT>::kChunk ? V : Elem<DT>::kChunk;
#pragma unroll
    for (int j = 0; j < V; j += N) load_n<DT, N>(row, c0 + j, x + j);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = c0 + j < E ? Elem<DT>::load(row, c0 + j) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (!(x[j] < INFINITY)) {
      x[j] = -INFINITY;
      *bad = true;
    }
}

template <int DT, int V>
__global__ __launch_bounds__(kThreads) void k_route(const RouteArgs a) {
  const uint32_t tok = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (tok >= a.tokens) return;
  const int lane = threadIdx.x & 63;
  const uint32_t s = tok / a.T, t = tok - s * a.T;
  float x[V];
  bool bad = false;
  load_logits<DT, V>(a.logits.p[s] + (uint64_t)t * a.E * Elem<DT>::kSize, a.E, lane, x, &bad);
  if (ballot(bad) && lane == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
  float best = x[0];
#pragma unroll
  for (int j = 1; j < V; ++j) best = fmaxf(best, x[j]);
  const float top = wave_max(best);
  float whole = 0.0f;
  if (!a.renorm) {
    if (top > -INFINITY) {
#pragma unroll
      for (int j = 0; j < V; ++j) whole += expf(x[j] - top);
    }
    whole = wave_sum(whole);
  }
  float m = top, mine = -INFINITY;
  int id = -1;
  for (int k = 0; k < a.K; ++k) {
    if (k) m = wave_max(best);
    if (!(m > -INFINITY)) break;
    const int owner = __builtin_ctzll(ballot(best == m));
    int j0 = 0;
#pragma unroll
    for (int j = V - 1; j >= 0; --j) j0 = x[j] == m ? j : j0;
    const int col = owner * V + __builtin_amdgcn_readlane(j0, owner);
    if (lane == k) {
      id = col;
      mine = m;
    }
    if (lane == owner) {
      best = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[j] = j == j0 ? -INFINITY : x[j];
        best = fmaxf(best, x[j]);
      }
    }
  }
  const float part = id >= 0 ? expf(mine - top) : 0.0f;
  if (a.renorm) whole = wave_sum(part);
  if (lane < a.K) {
    const uint64_t at = (uint64_t)tok * a.K + lane;
    a.topk[at] = id;
    a.weights[at] = id >= 0 ? part / whole : 0.0f;
  }
}

template <int DT, int V>
__global__ __launch_bounds__(kThreads) void k_route_backward(const RouteArgs a) {
  const uint32_t tok = blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (tok >= a.tokens) return;
  const int lane = threadIdx.x & 63;
  const uint32_t s = tok / a.T, t = tok - s * a.T;
  const uint64_t row = (uint64_t)t * a.E * Elem<DT>::kSize;
  int e = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < a.K) {
    const uint64_t at = (uint64_t)tok * a.K + lane;
    e = a.topk_in[at];
    if (e < -1 || e >= a.E) {
      atomic_or_u32(a.err, VR_ASYNC_BAD_EXPERT);
      e = -1;
    }
    if (e >= 0) {
      w = a.weights_in[at];
      dw = a.dweights[at];
    }
  }
  const float mean = wave_sum(w * dw);
  float p[V];
  float val = dw;  // what entry k adds at its column
  if (a.renorm) {
    val = w * (dw - mean);
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = 0.0f;
  } else {
    bool bad = false;
    load_logits<DT, V>(a.logits.p[s] + row, a.E, lane, p, &bad);
    if (ballot(bad) && lane == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
    float best = p[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = fmaxf(best, p[j]);
    const float top = wave_max(best);
    float whole = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = top > -INFINITY ? expf(p[j] - top) : 0.0f;
      whole += p[j];
    }
    whole = wave_sum(whole);
    const float inv = whole > 0.0f ? 1.0f / whole : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] *= inv;
  }
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    const int c = __builtin_amdgcn_readlane(e, k) - lane * V;
    const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(val), k));
    if (__builtin_amdgcn_readlane(e, k) < 0) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] += c == j ? v : 0.0f;
  }
  if (!a.renorm) {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = p[j] * (d[j] - mean);
  }
  char* out = a.dlogits.p[s] + row;
  const int c0 = lane * V;
  if (c0 + V <= a.E) {
    constexpr int N = V < Elem<DT>::kChunk ? V : Elem<DT>::kChunk;
#pragma unroll
    for (int j = 0; j < V; j += N) store_n<DT, N>(out, c0 + j, d + j);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c0 + j < a.E) Elem<DT>::store(out, c0 + j, d[j]);
  }
}

template <int DT, int V>
void launch_v(const RouteArgs& a, bool backward, hipStream_t st) {
  const dim3 grid((a.tokens + kWaves - 1) / kWaves);
  if (backward) hipLaunchKernelGGL((k_route_backward<DT, V>), grid, dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((k_route<DT, V>), grid, dim3(kThreads), 0, st, a);
}
template <int DT>
void launch_dt(const RouteArgs& a, bool backward, hipStream_t st) {
  if (a.E <= 64) launch_v<DT, 1>(a, backward, st);
  else if (a.E <= 128) launch_v<DT, 2>(a, backward, st);
  else if (a.E <= 256) launch_v<DT, 4>(a, backward, st);
  else if (a.E <= 512) launch_v<DT, 8>(a, backward, st);
  else launch_v<DT, 16>(a, backward, st);
}

vrResult_t launch(RouteArgs& a, vrComm* c, int dtype, bool backward, hipStream_t st) {
  a.R = c->nranks;
  a.err = c->err;
  a.tokens = static_cast<uint32_t>(a.R) * a.T;
  if (!a.tokens) return VR_OK;
  if (dtype == VR_DT_F32) launch_dt<VR_DT_F32>(a, backward, st);
  else launch_dt<VR_DT_BF16>(a, backward, st);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

}  // namespace

vrResult_t launch_route(vrComm* c, const vrSlice& logits, int dtype, int T, int K, int E, int32_t* topk,
                        float* weights, bool renorm, hipStream_t st) {
  RouteArgs a = {};
  a.logits = slice_tab(logits);
  a.topk = topk;
  a.weights = weights;
  a.T = T;
  a.K = K;
  a.E = E;
  a.renorm = renorm;
  return launch(a, c, dtype, false, st);
}

vrResult_t launch_route_backward(vrComm* c, const vrSlice& logits, int dtype, int T, int K, int E,
                                 const int32_t* topk, const float* weights, const float* dweights,
                                 const vrSlice& dlogits, bool renorm, hipStream_t st) {
  RouteArgs a = {};
  if (!renorm) {
    a.logits = slice_tab(logits);
  }
  a.dlogits = slice_tab(dlogits);
  a.topk_in = topk;
  a.weights_in = weights;
  a.dweights = dweights;
  a.T = T;
  a.K = K;
  a.E = E;
  a.renorm = renorm;
  return launch(a, c, dtype, true, st);
}

}  // namespace vr
