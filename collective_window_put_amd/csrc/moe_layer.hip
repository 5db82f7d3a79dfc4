// A whole mixture-of-experts layer for a few tokens (vr_moe_layer).
//
//   logits = x router^T (binary64), the routing as vr_route;
//   h = act(w_up x) (gated: act(gate) * up) per routing entry;
//   out = residual + sum_k weights[k] * (w_down h_k), in k order
//
// Bound by the bytes of the used experts' weights. The weights' rows are the
// first operand of the matrix instructions, 16 rows to a wave, read straight
// from HBM into registers; an expert's tokens, up to 16 at a time, are the
// second, so an expert's weights are read once for its first 16 tokens.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {

constexpr int kMaxPairs = VR_MOE_LAYER_MAX_TOKENS * 64;

struct Plan {              // written by k_moe_plan
  int used;                // experts with at least one entry
  int pad[3];
  int expert[1024];        // slot -> expert, ascending
  int first[1025];         // slot -> first of its entries in pair[]
  int pair[kMaxPairs];     // entry (token * K + k), by expert, ascending
};

struct MoeArgs {
  WinTab x, up, down, residual, out;
  const char* router;
  int32_t* topk;   // [R * T][K]
  float* weights;  // [R * T][K]
  uint32_t* err;
  double* logits;  // [N][E]
  Plan* plan;
  float* h;        // [N * K][I]
  float* y;        // [N * K][H]
  int R, T, N, H, I, E, K, renorm;
  uint32_t act;
};

__device__ inline double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ inline double wave_max_f64(double v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = fmax(v, __shfl_xor(v, m));
  return v;
}
template <int DT>
__device__ inline double piece_f64(v4u v, int j) {
  if constexpr (DT == VR_DT_F32) return __uint_as_float(v[j]);
  else return __uint_as_float((j & 1) ? (v[j / 2] & 0xFFFF0000u) : (v[j / 2] << 16));
}

// logits[n][e]: a wave takes one expert and 4 tokens. Products of two
// elements are exact in binary64; the choice of the K largest is then that of
// the exact logits except within a few 2^-53.
template <int DT>
__global__ __launch_bounds__(256) void k_moe_logits(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize;
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6), n0 = blockIdx.y * 4;
  if (e >= a.E) return;
  const char* w = a.router + (uint64_t)e * a.H * kES;
  const char* x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, a.N - 1);
    x[i] = a.x.p[n / a.T] + (uint64_t)(n % a.T) * a.H * kES;
  }
  double s[4] = {0, 0, 0, 0};
  for (int c = lane * kC; c < a.H; c += 64 * kC) {
    const v4u wv = load_piece<DT>(w + (uint64_t)c * kES, a.H - c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4u xv = load_piece<DT>(x[i] + (uint64_t)c * kES, a.H - c);
#pragma unroll
      for (int j = 0; j < kC; ++j) s[i] = fma(piece_f64<DT>(wv, j), piece_f64<DT>(xv, j), s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[i] = wave_sum_f64(s[i]);
    if (lane == 0 && n0 + i < a.N) a.logits[(uint64_t)(n0 + i) * a.E + e] = s[i];
  }
}

// The routing of every token (a wave each, as in vr_route), then the experts'
// entry lists. One workgroup.
template <int V>
__global__ __launch_bounds__(1024) void k_moe_plan(const MoeArgs a) {
  __shared__ short ids[kMaxPairs];
  __shared__ int offset[1024], slot[1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int n = wave; n < a.N; n += 16) {
    double x[V], best = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = lane * V + j;
      x[j] = c < a.E ? a.logits[(uint64_t)n * a.E + c] : -INFINITY;
      if (!(x[j] < INFINITY)) {
        x[j] = -INFINITY;
        bad = true;
      }
      best = fmax(best, x[j]);
    }
    if (ballot(bad) && lane == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
    const double top = wave_max_f64(best);
    double whole = 0.0;
    if (!a.renorm) {
      if (top > -INFINITY) {
#pragma unroll
        for (int j = 0; j < V; ++j) whole += exp(x[j] - top);
      }
      whole = wave_sum_f64(whole);
    }
    double mine = -INFINITY;
    int id = -1;
    for (int k = 0; k < a.K; ++k) {
      const double m = k ? wave_max_f64(best) : top;
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
          best = fmax(best, x[j]);
        }
      }
    }
    const double part = id >= 0 ? exp(mine - top) : 0.0;
    if (a.renorm) whole = wave_sum_f64(part);
    if (lane < a.K) {
      const int at = n * a.K + lane;
      a.topk[at] = id;
      a.weights[at] = id >= 0 ? static_cast<float>(part / whole) : 0.0f;
      ids[at] = static_cast<short>(id);
    }
  }
  __syncthreads();
  // thread e counts expert e's entries; then two sums over the experts
  const int pairs = a.N * a.K;
  int cnt = 0;
  for (int i = 0; i < pairs; ++i) cnt += ids[i] == tid;
  offset[tid] = cnt;
  slot[tid] = cnt > 0;
  __syncthreads();
  for (int m = 1; m < 1024; m <<= 1) {
    const int o = tid >= m ? offset[tid - m] : 0, s = tid >= m ? slot[tid - m] : 0;
    __syncthreads();
    offset[tid] += o;
    slot[tid] += s;
    __syncthreads();
  }
  if (cnt) {
    const int u = slot[tid] - 1, first = offset[tid] - cnt;
    a.plan->expert[u] = tid;
    a.plan->first[u] = first;
    for (int i = 0, k = first; i < pairs; ++i)
      if (ids[i] == tid) a.plan->pair[k++] = i;
  }
  if (tid == 1023) {
    a.plan->used = slot[1023];
    a.plan->first[slot[1023]] = offset[1023];
  }
}

// h of 16 columns of one expert: 4 waves split the hidden axis.
template <int DT, int ACT, bool GATED>
__global__ __launch_bounds__(256) void k_moe_up(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kStep = 4 * kC;
  const int u = blockIdx.x;
  if (u >= a.plan->used) return;
  const int e = a.plan->expert[u], first = a.plan->first[u], count = a.plan->first[u + 1] - first;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int c0 = blockIdx.y * 16, epr = a.E / a.R;
  const int U = GATED ? 2 * a.I : a.I;
  const char* w = a.up.p[e / epr] + (uint64_t)(e % epr) * U * a.H * kES;
  const int col = min(c0 + i, a.I - 1);
  const char* wg = w + (uint64_t)col * a.H * kES;
  const char* wu = w + (uint64_t)(GATED ? a.I + col : col) * a.H * kES;
  const int per = ((a.H + 4 * kStep - 1) / (4 * kStep)) * kStep;  // of the hidden axis, per wave
  const int k1 = min(a.H, (wave + 1) * per);
  __shared__ float part[4][GATED ? 2 : 1][16][17];
  for (int t0 = 0; t0 < count; t0 += 16) {
    const int pr = a.plan->pair[first + min(t0 + i, count - 1)], n = pr / a.K;
    const char* x = a.x.p[n / a.T] + (uint64_t)(n % a.T) * a.H * kES;
    v4f g = {0, 0, 0, 0}, v = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = wave * per + q * kC; k - q * kC < k1; k += kStep) {
      const v4u xv = load_piece<DT>(x + (uint64_t)k * kES, a.H - k);
      g = mfma_piece<DT>(load_piece<DT>(wg + (uint64_t)k * kES, a.H - k), xv, g);
      if (GATED) v = mfma_piece<DT>(load_piece<DT>(wu + (uint64_t)k * kES, a.H - k), xv, v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      part[wave][0][q * 4 + j][i] = g[j];
      if (GATED) part[wave][GATED ? 1 : 0][q * 4 + j][i] = v[j];
    }
    __syncthreads();
    const int c = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t0 + t < count && c0 + c < a.I) {
      const float zg = (part[0][0][c][t] + part[1][0][c][t]) + (part[2][0][c][t] + part[3][0][c][t]);
      float y = act_value<DT, ACT>(zg);
      if (GATED) {
        constexpr int h = GATED ? 1 : 0;
        y *= (part[0][h][c][t] + part[1][h][c][t]) + (part[2][h][c][t] + part[3][h][c][t]);
      }
      a.h[(uint64_t)a.plan->pair[first + t0 + t] * a.I + c0 + c] = y;
    }
    __syncthreads();
  }
}

// 8 binary32 values as the sum of two bf16 pieces (their error, 2^-16 of the
// value, is far below the outputs' rounding).
__device__ inline void split_piece(const float* f, v4u* hi, v4u* lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    (*hi)[j] = bf16_pack(f[2 * j], f[2 * j + 1]);
    (*lo)[j] = bf16_pack(f[2 * j] - bf16lo((*hi)[j]), f[2 * j + 1] - bf16hi((*hi)[j]));
  }
}

// y of 16 columns of one expert: 4 waves split the inner axis.
template <int DT>
__global__ __launch_bounds__(256) void k_moe_down(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kStep = 4 * kC;
  const int u = blockIdx.x;
  if (u >= a.plan->used) return;
  const int e = a.plan->expert[u], first = a.plan->first[u], count = a.plan->first[u + 1] - first;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int c0 = blockIdx.y * 16, epr = a.E / a.R;
  const char* w = a.down.p[e / epr] + ((uint64_t)(e % epr) * a.H + min(c0 + i, a.H - 1)) * a.I * kES;
  const int per = ((a.I + 4 * kStep - 1) / (4 * kStep)) * kStep;
  const int k1 = min(a.I, (wave + 1) * per);
  __shared__ float part[4][16][17];
  for (int t0 = 0; t0 < count; t0 += 16) {
    const float* h = a.h + (uint64_t)a.plan->pair[first + min(t0 + i, count - 1)] * a.I;
    v4f s = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = wave * per + q * kC; k - q * kC < k1; k += kStep) {
      const v4u wv = load_piece<DT>(w + (uint64_t)k * kES, a.I - k);
      if constexpr (DT == VR_DT_F32) {
        s = mfma_piece<DT>(wv, load_piece<VR_DT_F32>(reinterpret_cast<const char*>(h + k), a.I - k), s);
      } else {
        v4u p[2], hi, lo;
        p[0] = load_piece<VR_DT_F32>(reinterpret_cast<const char*>(h + k), a.I - k);
        p[1] = load_piece<VR_DT_F32>(reinterpret_cast<const char*>(h + k + 4), a.I - k - 4);
        split_piece(reinterpret_cast<const float*>(p), &hi, &lo);
        s = mfma_piece<DT>(wv, hi, s);
        s = mfma_piece<DT>(wv, lo, s);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[wave][q * 4 + j][i] = s[j];
    __syncthreads();
    const int c = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t0 + t < count && c0 + c < a.H)
      a.y[(uint64_t)a.plan->pair[first + t0 + t] * a.H + c0 + c] =
          (part[0][c][t] + part[1][c][t]) + (part[2][c][t] + part[3][c][t]);
    __syncthreads();
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_moe_sum(const MoeArgs a) {
  const int n = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  const int s = n / a.T;
  float acc = 0.0f;
  for (int k = 0; k < a.K; ++k)
    if (a.topk[n * a.K + k] >= 0) acc += a.weights[n * a.K + k] * a.y[(uint64_t)(n * a.K + k) * a.H + c];
  const uint64_t at = (uint64_t)(n % a.T) * a.H + c;
  if (a.residual.p[s]) acc += Elem<DT>::load(a.residual.p[s], at);
  Elem<DT>::store(a.out.p[s], at, acc);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
struct MoeLayout {
  size_t logits, plan, h, y, total;
};
MoeLayout layout(int R, const vrMoeShape& s) {
  MoeLayout l;
  const size_t N = (size_t)R * s.tokens;
  l.logits = 0;
  l.plan = align256(N * s.num_experts * sizeof(double));
  l.h = l.plan + align256(sizeof(Plan));
  l.y = l.h + align256(N * s.topk * s.inner * sizeof(float));
  l.total = l.y + align256(N * s.topk * s.hidden * sizeof(float));
  return l;
}

template <int DT>
void launch_dt(const MoeArgs& a, hipStream_t st) {
  const int slots = std::min(a.N * a.K, a.E);
  hipLaunchKernelGGL((k_moe_logits<DT>), dim3((a.E + 3) / 4, (a.N + 3) / 4), dim3(256), 0, st, a);
  if (a.E <= 64) hipLaunchKernelGGL((k_moe_plan<1>), dim3(1), dim3(1024), 0, st, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_moe_plan<4>), dim3(1), dim3(1024), 0, st, a);
  else hipLaunchKernelGGL((k_moe_plan<16>), dim3(1), dim3(1024), 0, st, a);
  const dim3 up(slots, (a.I + 15) / 16), down(slots, (a.H + 15) / 16);
  with_act(a.act, [&](auto act) {
    if (a.act & VR_ACT_GATED) hipLaunchKernelGGL((k_moe_up<DT, act(), true>), up, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_moe_up<DT, act(), false>), up, dim3(256), 0, st, a);
  });
  hipLaunchKernelGGL((k_moe_down<DT>), down, dim3(256), 0, st, a);
  hipLaunchKernelGGL((k_moe_sum<DT>), dim3((a.H + 255) / 256, a.N), dim3(256), 0, st, a);
}

}  // namespace

size_t moe_layer_workspace_bytes(int R, const vrMoeShape& s) { return layout(R, s).total; }

vrResult_t launch_moe_layer(vrComm* c, const vrMoeShape& s, const vrSlice& x, const void* router, const vrSlice& w_up,
                            const vrSlice& w_down, const vrSlice& residual, const vrSlice& out, int32_t* topk,
                            float* weights, char* ws, hipStream_t st) {
  const MoeLayout l = layout(c->nranks, s);
  MoeArgs a = {};
  a.x = slice_tab(x);
  a.up = slice_tab(w_up);
  a.down = slice_tab(w_down);
  a.residual = slice_tab(residual);
  a.out = slice_tab(out);
  a.router = static_cast<const char*>(router);
  a.topk = topk;
  a.weights = weights;
  a.err = c->err;
  a.logits = reinterpret_cast<double*>(ws + l.logits);
  a.plan = reinterpret_cast<Plan*>(ws + l.plan);
  a.h = reinterpret_cast<float*>(ws + l.h);
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.R = c->nranks;
  a.T = s.tokens;
  a.N = a.R * s.tokens;
  a.H = s.hidden;
  a.I = s.inner;
  a.E = s.num_experts;
  a.K = s.topk;
  a.renorm = (s.flags & VR_ROUTE_RENORM) != 0;
  a.act = s.act;
  if (!a.N) return VR_OK;
  if (s.dtype == VR_DT_F32) launch_dt<VR_DT_F32>(a, st);
  else launch_dt<VR_DT_BF16>(a, st);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

}  // namespace vr
