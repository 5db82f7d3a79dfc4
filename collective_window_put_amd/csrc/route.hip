// Router: softmax over each token's expert logits, the K largest, and the
// gradient.
//
//   p[j] = exp(x[j] - max x) / sum_j exp(x[j] - max x)
//   w[k] = p[e_k], or p[e_k] / sum_k p[e_k]
//   with m = sum_k dw[k] w[k]:  dx[j] = p[j] (sum_{k: e_k = j} dw[k] - m), or
//   renormalized  dx[e_k] = w[k] (dw[k] - m), 0 elsewhere
//
// Two forms. K up to 16 and E up to 512: 16 lanes to a token, four tokens to a
// wave (k_route_rows, below). Else one wave takes a token: lane l holds the
// V = ceil(E / 64) (rounded to a power of two) logits of columns l * V ..., so
// among equal logits the lowest lane, and in it the lowest register, is the
// lowest expert. Each of the K rounds takes the wave's maximum, finds its owner
// with a ballot and removes it there; lane k keeps round k's expert.
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

// ---- 16 lanes to a token --------------------------------------------------------------
// Lane s of a row of 16 holds V columns of its token in pieces of P, the row's
// lanes side by side. 32768 tokens of 256 fp32 logits, K = 8: 25.7 us with a
// wave to a token, whose K rounds of maximum, ballot and removal are bound by
// the vector units; 10.2 us this way (5.4 us at a large copy's 6.55 TB/s). The
// gradient of 32768 x 256 bf16 logits: 20.7 and 11.5 us (5.6); half the active
// LDS cycles of k_route_backward_rows are bank conflicts, since the four rows of
// a wave in `adds` lie a multiple of all banks apart.
template <int DT, int V> struct Cols {
  static constexpr int P = V < Elem<DT>::kChunk ? V : Elem<DT>::kChunk;
  __device__ static int at(int j, int s) { return (j / P * 16 + s) * P + j % P; }
};
template <int DT, int V>
__device__ inline void load_row(const char* row, int E, int s, float* x) {
  constexpr int P = Cols<DT, V>::P;
  if (16 * V <= E) {
#pragma unroll
    for (int j = 0; j < V; j += P) load_n<DT, P>(row, Cols<DT, V>::at(j, s), x + j);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += P) {
      const int c = Cols<DT, V>::at(j, s);
      if (c + P <= E) {
        load_n<DT, P>(row, c, x + j);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) x[j + i] = c + i < E ? Elem<DT>::load(row, c + i) : -INFINITY;
      }
    }
  }
}
// NaN and +inf become -inf and set the error bit.
template <int V>
__device__ inline void drop_bad(float* x, uint32_t* err) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (!(x[j] < INFINITY)) {
      x[j] = -INFINITY;
      bad = true;
    }
  if (bad) atomic_or_u32(err, VR_ASYNC_BAD_VALUE);
}
__device__ inline float row_max(float v) {
  return lane_reduce<4>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float row_min(float v) {
  return lane_reduce<4>(v, [](float a, float b) { return fminf(a, b); });
}
__device__ inline float row_sum(float v) {
  return lane_reduce<4>(v, [](float a, float b) { return a + b; });
}
// The value of the lane N to the left, going round in the row of 16.
template <int N>
__device__ inline float row_turn(float v) {
  const int b = static_cast<int>(__float_as_uint(v));
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(b, b, 0x120 + N, 0xF, 0xF, false)));
}
// How many of the row's other lanes hold more.
template <int N = 1>
__device__ inline int lanes_above(float v) {
  if constexpr (N < 16) return (row_turn<N>(v) > v ? 1 : 0) + lanes_above<N + 1>(v);
  else return 0;
}
// The value of the lane N to the left in the row, 0 past its start.
template <int N>
__device__ inline int row_left(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x110 + N, 0xF, 0xF, true);
}
// LDS of one wave: its operations run in order, the compiler keeps them so.
__device__ inline void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// No rounds: the K-th largest of the 16 lanes' maxima bounds the K-th largest
// logit from below, so only what reaches it (11 of 256 logits for K = 8, on
// average) goes to a list in the LDS, and each entry's place is the number of
// entries above it. An entry is the logit's order-preserving bits over the
// complement of its column: equal logits fall by column. Ties at the bound are
// all listed: a row of E equal logits compares E entries with E, and 32768 such
// tokens of 256 logits take 256 us.
template <int DT, int V>
__global__ __launch_bounds__(kThreads) void k_route_rows(const RouteArgs a) {
  __shared__ uint64_t lists[kWaves * 4][16 * V];
  __shared__ uint64_t chosen[kWaves * 4][16];
  const int lane = threadIdx.x & 63, s = lane & 15, row = threadIdx.x >> 4;
  const int rank = blockIdx.y, t0 = blockIdx.x * kWaves * 4 + row, t = min(t0, a.T - 1);
  uint64_t* list = lists[row];
  float x[V];
  load_row<DT, V>(a.logits.p[rank] + (uint64_t)t * a.E * Elem<DT>::kSize, a.E, s, x);
  drop_bad<V>(x, a.err);
  float best = x[0];
#pragma unroll
  for (int j = 1; j < V; ++j) best = fmaxf(best, x[j]);
  const float top = row_max(best);
  float whole = 0.0f;
  if (!a.renorm) {
    const float from = top > -INFINITY ? top : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) whole += expf(x[j] - from);
    whole = row_sum(whole);
  }
  const float least = fmaxf(row_min(lanes_above(best) < a.K ? best : INFINITY), -3.402823466e38f);  // never a masked one
  int n = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) n += x[j] >= least;
  int end = n;
  end += row_left<1>(end);
  end += row_left<2>(end);
  end += row_left<4>(end);
  end += row_left<8>(end);
  int at = end - n;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (x[j] >= least) {
      const uint32_t b = __float_as_uint(x[j] + 0.0f);  // -0 as 0
      const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
      list[at++] = static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(Cols<DT, V>::at(j, s));
    }
  wave_lds();
  const int count = __shfl(end, lane | 15);
  for (int i = s; i < count; i += 16) {
    const uint64_t mine = list[i];
    int above = 0;
#pragma unroll 4
    for (int o = 0; o < count; ++o) above += list[o] > mine;
    if (above < a.K) chosen[row][above] = mine;
  }
  wave_lds();
  int id = -1;
  float part = 0.0f;
  if (s < min(count, a.K)) {
    const uint64_t c = chosen[row][s];
    const uint32_t key = static_cast<uint32_t>(c >> 32);
    id = static_cast<int>(~static_cast<uint32_t>(c));
    part = expf(__uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu)) - top);
  }
  if (a.renorm) whole = row_sum(part);
  if (t0 < a.T && s < a.K) {
    const uint64_t to = ((uint64_t)rank * a.T + t) * a.K + s;
    a.topk[to] = id;
    a.weights[to] = id >= 0 ? part / whole : 0.0f;
  }
}

// What the entries add goes through the LDS to the lanes that hold the columns.
template <int DT, int V>
__global__ __launch_bounds__(kThreads) void k_route_backward_rows(const RouteArgs a) {
  constexpr int P = Cols<DT, V>::P;
  __shared__ __align__(16) float adds[kWaves * 4][16 * V];
  const int lane = threadIdx.x & 63, s = lane & 15, row = threadIdx.x >> 4;
  const int rank = blockIdx.y, t0 = blockIdx.x * kWaves * 4 + row, t = min(t0, a.T - 1);
  const uint64_t from = (uint64_t)t * a.E * Elem<DT>::kSize;
  float p[V];
  // rows past the last token load nothing: dlogits may be the logits, already overwritten
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = -INFINITY;
  if (!a.renorm && t0 < a.T) load_row<DT, V>(a.logits.p[rank] + from, a.E, s, p);
  int e = -1;
  float w = 0.0f, dw = 0.0f;
  if (s < a.K && t0 < a.T) {
    const uint64_t at = ((uint64_t)rank * a.T + t) * a.K + s;
    e = a.topk_in[at];
    w = a.weights_in[at];
    dw = a.dweights[at];
    if (e < -1 || e >= a.E) {
      atomic_or_u32(a.err, VR_ASYNC_BAD_EXPERT);
      e = -1;
    }
    if (e < 0) w = dw = 0.0f;
  }
  const float mean = row_sum(w * dw);
  float* add = adds[row];
  // entries that name one expert twice are added in their order; others, all at once
  if (e >= 0) add[e] = __uint_as_float(s);
  wave_lds();
  const bool twice = ballot(e >= 0 && __float_as_uint(add[e]) != static_cast<uint32_t>(s)) != 0;
  wave_lds();
#pragma unroll
  for (int j = 0; j < V; j += P)
#pragma unroll
    for (int i = 0; i < P; ++i) add[Cols<DT, V>::at(j + i, s)] = 0.0f;
  wave_lds();
  const float val = a.renorm ? w * (dw - mean) : dw;
  if (!twice) {
    if (e >= 0) add[e] = val;
  } else {
    for (int k = 0; k < a.K; ++k) {
      if (s == k && e >= 0) add[e] += val;
      wave_lds();
    }
  }
  wave_lds();
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = add[Cols<DT, V>::at(j, s)];
  if (!a.renorm) {
    drop_bad<V>(p, a.err);
    float best = p[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = fmaxf(best, p[j]);
    const float top = row_max(best), base = top > -INFINITY ? top : 0.0f;
    float whole = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      p[j] = expf(p[j] - base);
      whole += p[j];
    }
    whole = row_sum(whole);
    const float inv = whole > 0.0f ? 1.0f / whole : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = p[j] * inv * (d[j] - mean);
  }
  if (t0 >= a.T) return;
  char* out = a.dlogits.p[rank] + from;
#pragma unroll
  for (int j = 0; j < V; j += P) {
    const int c = Cols<DT, V>::at(j, s);
    if (c + P <= a.E) {
      store_n<DT, P>(out, c, d + j);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (c + i < a.E) Elem<DT>::store(out, c + i, d[j + i]);
    }
  }
}

template <int DT, int V>
void launch_rows(const RouteArgs& a, bool backward, hipStream_t st) {
  const dim3 grid((a.T + kWaves * 4 - 1) / (kWaves * 4), a.R);
  if (backward) hipLaunchKernelGGL((k_route_backward_rows<DT, V>), grid, dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((k_route_rows<DT, V>), grid, dim3(kThreads), 0, st, a);
}

template <int DT, int V>
void launch_v(const RouteArgs& a, bool backward, hipStream_t st) {
  const dim3 grid((a.tokens + kWaves - 1) / kWaves);
  if (backward) hipLaunchKernelGGL((k_route_backward<DT, V>), grid, dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((k_route<DT, V>), grid, dim3(kThreads), 0, st, a);
}
template <int DT>
void launch_dt(const RouteArgs& a, bool backward, hipStream_t st) {
  if (a.K <= 16 && a.E <= 512) {
    if (a.E <= 64) launch_rows<DT, 4>(a, backward, st);
    else if (a.E <= 128) launch_rows<DT, 8>(a, backward, st);
    else if (a.E <= 256) launch_rows<DT, 16>(a, backward, st);
    else launch_rows<DT, 32>(a, backward, st);
    return;
  }
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
