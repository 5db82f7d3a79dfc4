// Gradient of the MoE combine (vr_combine_backward). The combine mixes
//   out[s][t] = sum over k of weights[s][t][k] * y[d][p]
// with p = send_pos[s][t][k] the entry's row at rank d = expert / (E/R), so
//   dy[d][p] = weights[s][t][k] * dout[s][t]     (a put to the row's rank)
//   dweights[s][t][k] = dout[s][t] . y[d][p]     (a get from it)
//
// Bound by memory: for each entry one row is read and one written; a token's
// own row is read once for 8 (wide rows: 2) entries. A workgroup's entries are read
// together and their rows' addresses kept in the LDS, so that a lane holds no
// more than the rows' pieces and many waves fit; a group of 2^LOG lanes takes a
// token, its entries' loads in flight together. 8 ranks x 4096
// tokens of 512 bytes, top-8 of 256 experts: 57 us, 5.1 TB/s of rows in random
// places (each lane finding its rows by itself: 106 us, 3 waves to a SIMD; 4 or 8
// entries at a time, workgroups of 64 to 256 threads: within 2 us).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {


struct GradArgs {
  WinTab dout, y, dy;
  const int32_t *topk, *pos;  // [R][T][K]
  const float* weights;
  float* dweights;            // or null
  uint32_t* err;
  uint64_t row_bytes, cap;
  int R, T, K, per, E;        // per: experts of a rank
};

// An address read from the LDS, as one of global memory: the compiler makes
// flat loads and stores of it otherwise, which wait for the LDS too.
__device__ inline char* global(const char* p) {
  return (char*)reinterpret_cast<__attribute__((address_space(1))) char*>(reinterpret_cast<uintptr_t>(p));
}
// 16 bytes past the caches, which rows in random places only crowd (the case
// below: 64 us without, 62 with such stores, 57 with such loads too); any
// element alignment.
typedef v4u any_v4u __attribute__((aligned(2)));
__device__ inline v4u load_once(const char* p) { return __builtin_nontemporal_load(reinterpret_cast<const any_v4u*>(p)); }
template <int DT>
__device__ inline void store_once(char* p, const float* f) {
  v4u v;
  store_n<DT, Elem<DT>::kChunk>(&v, 0, f);
  __builtin_nontemporal_store(v, reinterpret_cast<any_v4u*>(p));
}

// Entries of a workgroup's tokens, in dynamic LDS: [kTok][K] each.
struct Entries {
  const char** from;  // the row of y; where there is none, the token's own row of dout (a valid address)
  char** to;          // the row of dy (without DY: of y), or null
  float* w;
  __device__ Entries(char* lds, int n) {
    from = reinterpret_cast<const char**>(lds);
    to = reinterpret_cast<char**>(lds + n * sizeof(char*));
    w = reinterpret_cast<float*>(lds + 2 * n * sizeof(char*));
  }
  static size_t bytes(int n) { return n * (2 * sizeof(char*) + sizeof(float)); }
};

// WHOLE: rows of whole pieces. kBatch entries at a time, kCh pieces of each to a lane.
template <int DT, int LOG, bool DY, bool DW, bool WHOLE, int kBatch, int kCh>
__global__ __launch_bounds__(256) void k_combine_back(const GradArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kL = 1 << LOG, kTok = 256 / kL;
  extern __shared__ __align__(16) char lds[];
  const int s = blockIdx.x % a.R, t0 = blockIdx.x / a.R * kTok, tokens = min(kTok, a.T - t0), K = a.K;
  const Entries en(lds, kTok * K);
  const char* dout = a.dout.p[s] + (uint64_t)t0 * a.row_bytes;
  const uint64_t e0 = ((uint64_t)s * a.T + t0) * K;
  for (int i = threadIdx.x; i < tokens * K; i += 256) {
    const int e = a.topk[e0 + i], p = a.pos[e0 + i];
    en.w[i] = a.weights[e0 + i];
    const char* from = nullptr;
    char* to = nullptr;
    if (e != -1 && (e < 0 || e >= a.E)) {
      atomic_or_u32(a.err, VR_ASYNC_BAD_EXPERT);
    } else if (e >= 0 && p != -1) {
      if (p < 0 || (uint64_t)p >= a.cap) {
        atomic_or_u32(a.err, VR_ASYNC_CAPACITY);
      } else {
        const int d = e / a.per;
        if (DW) from = a.y.p[d] + (uint64_t)p * a.row_bytes;
        to = (DY ? a.dy.p[d] : a.y.p[d]) + (uint64_t)p * a.row_bytes;
      }
    }
    if (DW && !from) {
      a.dweights[e0 + i] = 0.0f;
      from = dout + (uint64_t)(i / K) * a.row_bytes;
    }
    en.from[i] = from;
    en.to[i] = to;
  }
  __syncthreads();
  const int l = threadIdx.x & (kL - 1), t = threadIdx.x / kL;
  if (t >= tokens) return;
  const int H = static_cast<int>(a.row_bytes / Elem<DT>::kSize);
  const char* d = dout + (uint64_t)t * a.row_bytes;
  for (int k0 = 0; k0 < K; k0 += kBatch) {
    const int n = min(kBatch, K - k0), first = t * K + k0;
    float dot[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) dot[q] = 0.0f;
    for (int col0 = l * kC; col0 < H; col0 += kCh * kL * kC) {
      uint64_t off[kCh];
      int again[kCh];
      v4u dv[kCh], yv[kCh][kBatch];
      const bool tiny = !WHOLE && H < kC;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        // the last piece of a row that is no multiple of one starts early: its first `again` elements are another lane's too
        const int col = col0 + c * kL * kC, at = max(0, min(col, H - kC));
        again[c] = col - at;
        off[c] = (uint64_t)at * Elem<DT>::kSize;
        dv[c] = tiny ? load_piece<DT>(d, H) : load_whole<DT>(d + off[c]);
      }
      if (DW) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if (q >= n) break;
          const char* from = global(en.from[first + q]);
#pragma unroll
          for (int c = 0; c < kCh; ++c) yv[c][q] = tiny ? load_piece<DT>(from, H) : load_once(from + off[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if (kCh > 1 && again[c] >= kC) break;  // past the end, with all further ones
        float f[kC];
#pragma unroll
        for (int j = 0; j < kC; ++j) f[j] = piece_f32<DT>(dv[c], j);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if (q >= n) break;
          if (DW) {
#pragma unroll
            for (int j = 0; j < kC; ++j)
              if (WHOLE || j >= again[c]) dot[q] = fmaf(f[j], piece_f32<DT>(yv[c][q], j), dot[q]);
          }
          if (DY && en.to[first + q]) {
            char* to = global(en.to[first + q]);
            const float w = en.w[first + q];
            float g[kC];
#pragma unroll
            for (int j = 0; j < kC; ++j) g[j] = w * f[j];
            if (!tiny) {
              store_once<DT>(to + off[c], g);
            } else {
#pragma unroll
              for (int j = 0; j < kC - 1; ++j)
                if (j < H) Elem<DT>::store(to, j, g[j]);
            }
          }
        }
      }
    }
    if (DW) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const float v = lane_reduce<LOG>(dot[q], [](float x, float y) { return x + y; });
        // an entry without a row has its zero already
        if (l == q && q < n && en.to[first + q]) a.dweights[e0 + first + q] = v;
      }
    }
  }
}

template <int DT, int LOG, bool WHOLE, int kB, int kCh>
vrResult_t start(const GradArgs& a, hipStream_t st) {
  constexpr int kTok = 256 >> LOG;
  const dim3 grid(a.R * ((a.T + kTok - 1) / kTok));
  const size_t lds = Entries::bytes(kTok * a.K);  // at most 40 KiB
  if (!a.dweights) hipLaunchKernelGGL((k_combine_back<DT, LOG, true, false, WHOLE, kB, kCh>), grid, dim3(256), lds, st, a);
  else if (!a.dy.p[0]) hipLaunchKernelGGL((k_combine_back<DT, LOG, false, true, WHOLE, kB, kCh>), grid, dim3(256), lds, st, a);
  else hipLaunchKernelGGL((k_combine_back<DT, LOG, true, true, WHOLE, kB, kCh>), grid, dim3(256), lds, st, a);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}
template <int DT, int LOG>
vrResult_t start(const GradArgs& a, hipStream_t st) {
  // Rows of several pieces to a lane: two entries at a time, four pieces of each, so that loads and stores run along the
  // rows. 4 x 2048 tokens of 4 KiB, top-4: 60 us, eight entries and one piece 67, four and two 64.
  if constexpr (LOG == 6) {
    if (a.row_bytes > 16u << LOG)
      return a.row_bytes % 16 ? start<DT, LOG, false, 2, 4>(a, st) : start<DT, LOG, true, 2, 4>(a, st);
  }
  return a.row_bytes % 16 ? start<DT, LOG, false, 8, 1>(a, st) : start<DT, LOG, true, 8, 1>(a, st);
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
