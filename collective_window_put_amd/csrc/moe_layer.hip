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
// Launches: the routing (a workgroup per token; its logits apart where there
// are many), the up products, the down products and the weighted sum (one, for
// a single token). What a product needs of the routing it works out again from
// the chosen ids: a plan made by a launch of its own, one workgroup, took 7 us
// for one token and 33 us for 32. The sum has a launch of its own: by the last
// workgroup of each column group to arrive at a counter it took 8 us more for
// one token and 30 us more for 32 (coherent stores, an atomic and an acquire
// for every workgroup of the down products).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {

constexpr int kMaxPairs = VR_MOE_LAYER_MAX_TOKENS * 64;

struct MoeArgs {
  WinTab x, up, down, residual, out;
  const char* router;
  int32_t* topk;   // [R * T][K]
  float* weights;  // [R * T][K]
  uint32_t* err;
  double* logits;  // [N][E], or null: k_moe_route computes them
  char* h;         // [N * K][ldh] binary32; bf16: two such arrays, of the value and of what its rounding left out
  float* y;        // [N * K][H]
  uint64_t h_part; // bytes from the first array to the second
  int R, T, N, H, I, E, K, ldh, renorm;
  uint32_t act;
};

// A token's logits of experts e0 .. e0 + 3 into out[0 .. 3], by one wave.
// Products of two elements are exact in binary64; the choice of the K largest
// is then that of the exact logits except within a few 2^-53.
template <int DT>
__device__ inline void expert_logits(const MoeArgs& a, int n, int e0, double* out) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize;
  const int lane = static_cast<int>(lane_id());
  const char* x = a.x.p[n / a.T] + (uint64_t)(n % a.T) * a.H * kES;
  const char* w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = a.router + (uint64_t)min(e0 + i, a.E - 1) * a.H * kES;
  double s[4] = {0, 0, 0, 0};
  // four pieces a lane of each row in flight: the rows come from another
  // XCD's L2 or from HBM, and a workgroup is alone with its token
  for (int c0 = 0; c0 < a.H; c0 += 4 * 64 * kC) {
    v4u xv[4], wv[4][4];
    const int c = c0 + lane * kC;
    if (c0 + 4 * 64 * kC <= a.H) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint64_t at = (uint64_t)(c + u * 64 * kC) * kES;
        xv[u] = load_whole<DT>(x + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[u][i] = load_whole<DT>(w[i] + at);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint64_t at = (uint64_t)(c + u * 64 * kC) * kES;
        const int n = a.H - c - u * 64 * kC;
        xv[u] = load_piece<DT>(x + at, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[u][i] = load_piece<DT>(w[i] + at, n);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const double xj = piece_f32<DT>(xv[u], j);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = fma(piece_f32<DT>(wv[u][i], j), xj, s[i]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[i] = wave_sum(s[i]);
    if (lane == 0 && e0 + i < a.E) out[i] = s[i];
  }
}

// The logits of 16 experts and one token.
template <int DT>
__global__ __launch_bounds__(256) void k_moe_logits(const MoeArgs a) {
  const int n = blockIdx.y, e0 = blockIdx.x * 16 + (threadIdx.x >> 6) * 4;
  if (e0 < a.E) expert_logits<DT>(a, n, e0, a.logits + (uint64_t)n * a.E + e0);
}

// A workgroup routes one token: its waves compute the logits (unless
// k_moe_logits has), the first chooses.
template <int DT, int V>
__global__ __launch_bounds__(1024) void k_moe_route(const MoeArgs a) {
  __shared__ double own[64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.x;
  const double* logits = own;
  if (a.logits) {
    logits = a.logits + (uint64_t)n * a.E;
  } else {
    for (int e0 = wave * 4; e0 < a.E; e0 += 64) expert_logits<DT>(a, n, e0, own + e0);
    __syncthreads();
    if (wave) return;
  }
  // as vr_route, in binary64
  double x_[V], best = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = lane * V + j;
    x_[j] = c < a.E ? logits[c] : -INFINITY;
    if (!(x_[j] < INFINITY)) {
      x_[j] = -INFINITY;
      bad = true;
    }
    best = fmax(best, x_[j]);
  }
  if (ballot(bad) && lane == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
  const double top = wave_max(best);
  double whole = 0.0;
  if (!a.renorm) {
    if (top > -INFINITY) {
#pragma unroll
      for (int j = 0; j < V; ++j) whole += exp(x_[j] - top);
    }
    whole = wave_sum(whole);
  }
  double mine = -INFINITY;
  int id = -1;
  for (int k = 0; k < a.K; ++k) {
    const double m = k ? wave_max(best) : top;
    if (!(m > -INFINITY)) break;
    const int owner = __builtin_ctzll(ballot(best == m));
    int j0 = 0;
#pragma unroll
    for (int j = V - 1; j >= 0; --j) j0 = x_[j] == m ? j : j0;
    const int col = owner * V + __builtin_amdgcn_readlane(j0, owner);
    if (lane == k) {
      id = col;
      mine = m;
    }
    if (lane == owner) {
      best = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x_[j] = j == j0 ? -INFINITY : x_[j];
        best = fmax(best, x_[j]);
      }
    }
  }
  const double part = id >= 0 ? exp(mine - top) : 0.0;
  if (a.renorm) whole = wave_sum(part);
  if (lane < a.K) {
    const int at = n * a.K + lane;
    a.topk[at] = id;
    a.weights[at] = id >= 0 ? static_cast<float>(part / whole) : 0.0f;
  }
}

// The entries of the slot-th expert that has any, in order, into list (LDS; a
// token names an expert once at most); returns their count, 0 when there is no
// such expert. All threads of the workgroup call it.
__device__ inline int find_expert(const MoeArgs& a, int slot, short* ids, uint32_t* bits, short* list, int* expert) {
  const int tid = threadIdx.x, lane = tid & 63, pairs = a.N * a.K;
  if (a.N == 1) {  // one token's experts all differ: the slot is the entry
    *expert = a.topk[slot];
    list[0] = static_cast<short>(slot);
    __syncthreads();
    return *expert >= 0;
  }
  if (tid < 32) bits[tid] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += blockDim.x) {
    const int id = a.topk[i];
    ids[i] = static_cast<short>(id);
    if (id >= 0) atomicOr(&bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const uint32_t word = lane < 32 ? bits[lane] : 0;
  int sum = __popc(word);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up(sum, m);
    if (lane >= m) sum += o;
  }
  const uint64_t past = ballot(lane < 32 && sum > slot);
  if (!past) return 0;
  const int at = __builtin_ctzll(past);
  uint32_t w = __builtin_amdgcn_readlane(word, at);
  for (int skip = slot - (__builtin_amdgcn_readlane(sum, at) - __popc(w)); skip > 0; --skip) w &= w - 1;
  const int e = at * 32 + __builtin_ctz(w);
  int count = 0;  // each wave writes the whole list, all the same
  for (int i0 = 0; i0 < pairs; i0 += 64) {
    const bool hit = i0 + lane < pairs && ids[i0 + lane] == e;
    const uint64_t m = ballot(hit);
    if (hit) list[count + __popcll(m & ((1ull << lane) - 1))] = static_cast<short>(i0 + lane);
    count += __popcll(m);
  }
  __syncthreads();
  *expert = e;
  return count;
}

__device__ inline char* h_row(const MoeArgs& a, int pair, int es) { return a.h + (uint64_t)pair * a.ldh * es; }

// h of 16 columns of one expert: 8 waves split the hidden axis.
template <int DT, int ACT, bool GATED>
__global__ __launch_bounds__(512) void k_moe_up(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kStep = 4 * kC, NW = GATED ? 2 : 1;
  __shared__ short ids[kMaxPairs], list[VR_MOE_LAYER_MAX_TOKENS];
  __shared__ uint32_t bits[32];
  __shared__ float part[8][NW][16][17];
  int e;
  const int count = find_expert(a, blockIdx.y, ids, bits, list, &e);
  if (!count) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
  const int c0 = blockIdx.x * 16, epr = a.E / a.R;
  const char* w = a.up.p[e / epr] + (uint64_t)(e % epr) * (GATED ? 2 : 1) * a.I * a.H * kES;
  const int col = min(c0 + i, a.I - 1);
  const char* wr[NW];
#pragma unroll
  for (int h = 0; h < NW; ++h) wr[h] = w + ((uint64_t)h * a.I + col) * a.H * kES;
  const int per = (a.H + 8 * kStep - 1) / (8 * kStep) * kStep;  // of the hidden axis, per wave
  for (int t0 = 0; t0 < count; t0 += 16) {
    const int n = list[min(t0 + i, count - 1)] / a.K;
    const char* x[1] = {a.x.p[n / a.T] + (uint64_t)(n % a.T) * a.H * kES};
    v4f z[NW][1];
#pragma unroll
    for (int h = 0; h < NW; ++h) z[h][0] = v4f{0, 0, 0, 0};
    stream_products<DT, NW, 1, 4>(wr, x, wave * per, min(a.H, (wave + 1) * per), a.H, z);
#pragma unroll
    for (int h = 0; h < NW; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wave][h][q * 4 + j][i] = z[h][0][j];
    __syncthreads();
    const int c = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t < 16 && t0 + t < count && c0 + c < a.I) {
      float s[NW];
#pragma unroll
      for (int h = 0; h < NW; ++h) {
        s[h] = 0.0f;
#pragma unroll
        for (int v = 0; v < 8; ++v) s[h] += part[v][h][c][t];
      }
      float y = act_value<DT, ACT>(s[0]);
      if (GATED) y *= s[NW - 1];
      char* to = h_row(a, list[t0 + t], kES);
      Elem<DT>::store(to, c0 + c, y);
      // bf16: what the rounding left out; the two hold the value to 2^-16, far below the outputs' rounding
      if (DT == VR_DT_BF16) {
        const float hi = Elem<DT>::round(y);
        Elem<DT>::store(to + a.h_part, c0 + c, fabsf(hi) < INFINITY ? y - hi : 0.0f);
      }
    }
    __syncthreads();
  }
}

// y of CG * 16 columns of one expert. 8 waves: CG groups of 16 columns by 8 / CG parts
// of the inner axis. h goes through the LDS, once for all waves (read by each
// wave from memory, it took two loads for every load of weights and the
// kernel reached 2.8 TB/s); the weights go straight to registers, the first of
// them already while h is staged.
template <int DT, int CG>
__global__ __launch_bounds__(512, 4) void k_moe_down(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kStep = 4 * kC, kPart = 8 / CG;
  constexpr int kArr = DT == VR_DT_BF16 ? 2 : 1;       // arrays of h
  constexpr int kRow = 2048 / kArr;                    // bytes of a staged row, of each array: 2 KB a token in all
  constexpr int kK = kRow / kES, kPieces = kRow / 16;  // inner elements staged at a time
  constexpr int U = 8;
  __shared__ __align__(16) char hs[16 * kRow * kArr];
  __shared__ short ids[kMaxPairs], list[VR_MOE_LAYER_MAX_TOKENS];
  __shared__ uint32_t bits[32];
  __shared__ float part[8][16][17];
  int e;
  const int count = find_expert(a, blockIdx.y, ids, bits, list, &e);
  const int cb = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, q = lane >> 4;
  const int c0 = (cb * CG + wave % CG) * 16, pt = wave / CG, epr = a.E / a.R;
  if (count) {
    const char* w = a.down.p[e / epr] + ((uint64_t)(e % epr) * a.H + min(c0 + i, a.H - 1)) * a.I * kES;
    for (int t0 = 0; t0 < count; t0 += 16) {
      const int rows = min(count - t0, 16);
      v4f z[kArr];
#pragma unroll
      for (int h = 0; h < kArr; ++h) z[h] = v4f{0, 0, 0, 0};
      for (int k0 = 0; k0 < a.I; k0 += kK) {
        const int len = min(a.I - k0, kK), steps = (len + kStep - 1) / kStep;
        const int per = (steps + kPart - 1) / kPart, s1 = min(steps, (pt + 1) * per);
        v4u wv[U];
        auto fetch = [&](int s) {  // steps [s, s + U) of the weights; past the end: the last, unused or zero-filled
          const int k = k0 + s * kStep + q * kC;
          if (k0 + (s + U) * kStep <= a.I) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              wv[u] = load_whole<DT>(w + (uint64_t)(k + u * kStep) * kES);
          } else {
#pragma unroll
            for (int u = 0; u < U; ++u) wv[u] = load_piece<DT>(w + (uint64_t)(k + u * kStep) * kES, a.I - k - u * kStep);
          }
        };
        int s = pt * per;
        if (s < s1) fetch(s);
        __syncthreads();  // the staged rows of the step before have been read
        for (int id = tid; id < rows * kArr * kPieces; id += 512) {
          const int p = id % kPieces, h = id / kPieces % kArr, t = id / (kPieces * kArr);
          if (p * kC < len) {
            const v4u v = load_piece<DT>(h_row(a, list[t0 + t], kES) + h * a.h_part + (uint64_t)(k0 + p * kC) * kES, len - p * kC);
            *reinterpret_cast<v4u*>(hs + (t * kArr + h) * kRow + ((p ^ (t & 7)) << 4)) = v;
          }
        }
        __syncthreads();
        const int t = min(i, rows - 1);
        while (s < s1) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const int p = (s + u) * 4 + q;
#pragma unroll
            for (int h = 0; h < kArr; ++h) {
              v4u hv = {0, 0, 0, 0};
              if (p * kC < len) hv = *reinterpret_cast<const v4u*>(hs + (t * kArr + h) * kRow + ((p ^ (t & 7)) << 4));
              z[h] = mfma_piece<DT>(wv[u], hv, z[h]);
            }
          }
          s += U;
          if (s < s1) fetch(s);
        }
      }
      const v4f sum = kArr == 2 ? z[0] + z[kArr - 1] : z[0];
      if (kPart == 1) {
        if (i < rows) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c0 + q * 4 + j < a.H)
              a.y[(uint64_t)list[t0 + i] * a.H + c0 + q * 4 + j] = sum[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) part[wave][q * 4 + j][i] = sum[j];
        __syncthreads();
        for (int v = tid; v < CG * 256; v += 512) {
          const int c = v & 15, t = v >> 4 & 15, g = v >> 8, col = (cb * CG + g) * 16 + c;
          if (t < rows && col < a.H) {
            float y = 0.0f;
#pragma unroll
            for (int p = 0; p < kPart; ++p) y += part[p * CG + g][c][t];
            a.y[(uint64_t)list[t0 + t] * a.H + col] = y;
          }
        }
      }
    }
  }
}

// One token: out of 8 columns, its experts' products and their sum in one
// launch. 16 waves, each four rows of one expert's w_down at a time over the
// vector units: a matrix instruction would have 15 of its 16 token columns
// empty, and the rows' pieces are all in flight at once. Top-8 of 2048 x 1024
// bf16 experts: 8.9 us (5.1 at a large copy's 6.55 TB/s), against 16.2 us for
// k_moe_down and k_moe_sum.
template <int DT>
__global__ __launch_bounds__(1024) void k_moe_down_one(const MoeArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kArr = DT == VR_DT_BF16 ? 2 : 1, U = 2, kCols = 8;
  __shared__ float y[64][kCols];  // topk is 64 at most
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c0 = blockIdx.x * kCols, epr = a.E / a.R;
  for (int k = wave / 2; k < a.K; k += 8) {
    const int e = a.topk[k], col = c0 + wave % 2 * 4;
    if (e < 0) continue;
    const char* h = h_row(a, k, kES);
    const char* w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = a.down.p[e / epr] + ((uint64_t)(e % epr) * a.H + min(col + i, a.H - 1)) * a.I * kES;
    float s[4] = {0, 0, 0, 0};
    for (int i0 = 0; i0 < a.I; i0 += U * 64 * kC) {
      v4u wv[U][4], hv[U][kArr];
      const int at = i0 + lane * kC;
      if (i0 + U * 64 * kC <= a.I) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint64_t b = (uint64_t)(at + u * 64 * kC) * kES;
#pragma unroll
          for (int i = 0; i < 4; ++i) wv[u][i] = load_whole<DT>(w[i] + b);
#pragma unroll
          for (int v = 0; v < kArr; ++v) hv[u][v] = load_whole<DT>(h + v * a.h_part + b);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint64_t b = (uint64_t)(at + u * 64 * kC) * kES;
          const int n = a.I - at - u * 64 * kC;
#pragma unroll
          for (int i = 0; i < 4; ++i) wv[u][i] = load_piece<DT>(w[i] + b, n);
#pragma unroll
          for (int v = 0; v < kArr; ++v) hv[u][v] = load_piece<DT>(h + v * a.h_part + b, n);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          float f = piece_f32<DT>(hv[u][0], j);
          if (kArr == 2) f += piece_f32<DT>(hv[u][kArr - 1], j);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = fmaf(piece_f32<DT>(wv[u][i], j), f, s[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = wave_sum(s[i]);
    if (lane < 4) y[k][wave % 2 * 4 + lane] = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
  }
  __syncthreads();
  const int col = c0 + tid;
  if (tid >= kCols || col >= a.H) return;
  float acc = 0.0f;
  for (int k = 0; k < a.K; ++k)
    if (a.topk[k] >= 0) acc += a.weights[k] * y[k][tid];
  if (a.residual.p[0]) acc += Elem<DT>::load(a.residual.p[0], col);
  Elem<DT>::store(a.out.p[0], col, acc);
}

// out: each token's entries in k order.
template <int DT>
__global__ __launch_bounds__(256) void k_moe_sum(const MoeArgs a) {
  const int n = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  const int s = n / a.T;
  float acc = 0.0f;
#pragma unroll 8
  for (int k = 0; k < a.K; ++k) {
    const int p = n * a.K + k;
    if (a.topk[p] >= 0) acc += a.weights[p] * a.y[(uint64_t)p * a.H + c];
  }
  const uint64_t at = (uint64_t)(n % a.T) * a.H + c;
  if (a.residual.p[s]) acc += Elem<DT>::load(a.residual.p[s], at);
  Elem<DT>::store(a.out.p[s], at, acc);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
// Whether the logits have a launch of their own, spread over the chip: it and
// the choice then take 5.8 and 5.3 us (32 tokens, 256 experts of 2048 hidden
// elements), where a workgroup that does both takes 24 us, and 8 us for 64
// experts.
bool logits_apart(const vrMoeShape& s) { return (uint64_t)s.num_experts * s.hidden > 1u << 18; }

struct MoeLayout {
  int ldh;
  size_t logits, h, h_part, y, total;
};
MoeLayout layout(int R, const vrMoeShape& s) {
  MoeLayout l;
  const size_t N = (size_t)R * s.tokens, es = s.dtype == VR_DT_F32 ? 4 : 2;
  l.ldh = static_cast<int>((s.inner + 16 / es - 1) / (16 / es) * (16 / es));
  l.logits = 0;
  l.h = logits_apart(s) ? align256(N * s.num_experts * sizeof(double)) : 0;
  l.h_part = align256(N * s.topk * l.ldh * es);
  l.y = l.h + (s.dtype == VR_DT_F32 ? 1 : 2) * l.h_part;
  l.total = l.y + align256(N * s.topk * s.hidden * sizeof(float));
  return l;
}

template <int DT>
void launch_dt(const MoeArgs& a, hipStream_t st) {
  const int slots = std::min(a.N * a.K, a.E);
  const int threads = a.logits ? 64 : 1024;
  if (a.logits) hipLaunchKernelGGL((k_moe_logits<DT>), dim3((a.E + 15) / 16, a.N), dim3(256), 0, st, a);
  if (a.E <= 64) hipLaunchKernelGGL((k_moe_route<DT, 1>), dim3(a.N), dim3(threads), 0, st, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_moe_route<DT, 4>), dim3(a.N), dim3(threads), 0, st, a);
  else hipLaunchKernelGGL((k_moe_route<DT, 16>), dim3(a.N), dim3(threads), 0, st, a);
  // columns, then experts, in a direction each: their product may pass the 2^32 threads that a direction holds
  const dim3 up((a.I + 15) / 16, slots);
  with_act(a.act, [&](auto act) {
    if (a.act & VR_ACT_GATED) hipLaunchKernelGGL((k_moe_up<DT, act(), true>), up, dim3(512), 0, st, a);
    else hipLaunchKernelGGL((k_moe_up<DT, act(), false>), up, dim3(512), 0, st, a);
  });
  if (a.N == 1) {
    hipLaunchKernelGGL((k_moe_down_one<DT>), dim3((a.H + 7) / 8), dim3(1024), 0, st, a);
    return;
  }
  // as many columns to a workgroup as leave the chip four of them per compute unit
  const auto grid = [&](int cg) { return dim3((a.H + cg * 16 - 1) / (cg * 16), slots); };
  const auto groups = [&](int cg) { return grid(cg).x * slots; };
  if (groups(8) >= 1024) hipLaunchKernelGGL((k_moe_down<DT, 8>), grid(8), dim3(512), 0, st, a);
  else if (groups(4) >= 512) hipLaunchKernelGGL((k_moe_down<DT, 4>), grid(4), dim3(512), 0, st, a);
  else hipLaunchKernelGGL((k_moe_down<DT, 2>), grid(2), dim3(512), 0, st, a);
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
  a.logits = logits_apart(s) ? reinterpret_cast<double*>(ws + l.logits) : nullptr;
  a.h = ws + l.h;
  a.h_part = l.h_part;
  a.ldh = l.ldh;
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
