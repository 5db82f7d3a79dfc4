// Shared by the layer kernels (route.hip, linear.hip, linear_q8.hip, moe_layer.hip,
// norm.hip, combine_grad.hip): element traits, activations, wave reductions and
// the row ranges of groups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "vr_device.hpp"
#include "vr_internal.hpp"

namespace vr {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// fp32 -> bf16 bits, round to nearest even (the hardware conversion; a NaN
// stays one).
__device__ inline uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }
__device__ inline uint32_t bf16_pack(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, v2bf{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
}

template <int DT> struct Elem;
template <> struct Elem<VR_DT_F32> {
  typedef float T;
  static constexpr int kSize = 4;
  static constexpr int kChunk = 4;  // elements of 16 bytes
  __device__ static float load(const void* p, uint64_t i) { return load4f_global(static_cast<const char*>(p) + 4 * i); }
  __device__ static void store(void* p, uint64_t i, float f) { static_cast<float*>(p)[i] = f; }
  __device__ static float round(float f) { return f; }
};
template <> struct Elem<VR_DT_BF16> {
  typedef uint16_t T;
  static constexpr int kSize = 2;
  static constexpr int kChunk = 8;
  __device__ static float load(const void* p, uint64_t i) {
    return __uint_as_float(static_cast<uint32_t>(load2_global(static_cast<const char*>(p) + 2 * i)) << 16);
  }
  __device__ static void store(void* p, uint64_t i, float f) { static_cast<uint16_t*>(p)[i] = bf16_bits(f); }
  __device__ static float round(float f) { return __uint_as_float(static_cast<uint32_t>(bf16_bits(f)) << 16); }
};

// Operands in 8 bits (rows with a scale each), by the type of what their products make.
constexpr int kI8ToF32 = 16, kI8ToBf16 = 17;
template <int DT> constexpr bool kInt8 = DT == kI8ToF32 || DT == kI8ToBf16;
template <int DT> constexpr int kOutOf = DT == kI8ToF32 ? VR_DT_F32 : DT == kI8ToBf16 ? VR_DT_BF16 : DT;
struct Elem8 {
  typedef uint8_t T;
  static constexpr int kSize = 1;
  static constexpr int kChunk = 16;
};
template <> struct Elem<kI8ToF32> : Elem8 {};
template <> struct Elem<kI8ToBf16> : Elem8 {};
typedef int v4i __attribute__((ext_vector_type(4)));
// Sums of products.
template <int DT> using Acc = std::conditional_t<kInt8<DT>, v4i, v4f>;

// N consecutive elements (N * size at most 16 bytes); any element alignment:
// the global loads and stores of this chip take it.
template <int DT, int N> __device__ inline void load_n(const void* p, uint64_t i, float* f) {
  const char* q = static_cast<const char*>(p) + i * Elem<DT>::kSize;
  if constexpr (N == 1) {
    f[0] = Elem<DT>::load(p, i);
  } else {
    typename Elem<DT>::T t[N];
    __builtin_memcpy(t, __builtin_assume_aligned(q, Elem<DT>::kSize), sizeof(t));
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (DT == VR_DT_F32) f[j] = t[j];
      else f[j] = __uint_as_float(static_cast<uint32_t>(t[j]) << 16);
    }
  }
}
template <int DT, int N> __device__ inline void store_n(void* p, uint64_t i, const float* f) {
  char* q = static_cast<char*>(p) + i * Elem<DT>::kSize;
  if constexpr (DT == VR_DT_F32) {
    __builtin_memcpy(__builtin_assume_aligned(q, 4), f, 4 * N);
  } else if constexpr (N == 1) {
    Elem<DT>::store(p, i, f[0]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) w[j] = bf16_pack(f[2 * j], f[2 * j + 1]);
    __builtin_memcpy(__builtin_assume_aligned(q, 2), w, 2 * N);
  }
}

// ---- activations ------------------------------------------------------------------
// act(z) and its derivative in binary32: relu max(z, 0) (a NaN stays one);
// gelu z cdf(z), cdf(z) = (1 + erf(z / sqrt 2)) / 2; silu z / (1 + exp(-z)).
// At -inf gelu and silu are -inf * 0, a NaN. fp32 tensors use the library's
// functions and an IEEE division. bf16 tensors use the hardware's exp2 and
// reciprocal (one step each) and the polynomial of upper_tail, below the
// outputs' rounding (2^-8 of the value) over the whole range: a 256 x 256
// tile's epilogue runs while nothing else is on its compute unit.
__device__ inline float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
template <int DT>
__device__ inline float sigmoid(float z) {
  if constexpr (DT == VR_DT_F32) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + fast_exp(-z));
}
// 1 - cdf(x) for x >= 0, as 2 to a polynomial in x: log2 of the tail is smooth
// where the tail itself falls over 38 decades. Coefficients: a least squares fit
// at Chebyshev points of [0, 13.2], reweighted until the error was at most 2^-12
// of the value and 4e-7 / max(1, x). Evaluated in binary32 it is off by 2.6e-4 of
// the value and by 4.2e-7 at most; past 13 the tail is below the smallest normal
// number and becomes 0. The leading term is negative, so it falls to 0 at
// infinity; a NaN stays one.
__device__ inline float upper_tail(float x) {
  float p = fmaf(x, -3.472188925e-10f, 1.874049538e-8f);
  p = fmaf(x, p, -3.703213736e-7f);
  p = fmaf(x, p, 2.263529268e-6f);
  p = fmaf(x, p, 3.237149940e-5f);
  p = fmaf(x, p, -7.960115327e-4f);
  p = fmaf(x, p, 8.136725053e-3f);
  p = fmaf(x, p, -5.340901017e-2f);
  p = fmaf(x, p, -4.588466585e-1f);
  p = fmaf(x, p, -1.151156425f);
  return __builtin_amdgcn_exp2f(fmaf(x, p, -9.999988675e-1f));
}
// cdf(z); *e = exp(-z^2 / 2)
template <int DT>
__device__ inline float normal_cdf(float z, float* e) {
  if constexpr (DT == VR_DT_F32) {
    // erfc multiplies its argument's relative error by z^2: the argument's two
    // roundings (of 1 / sqrt 2 and of the product) are put back to first order,
    // d erfc(t) = -2 / sqrt(pi) exp(-t^2) dt with exp(-t^2) = *e. At z = -11.6
    // they took 1e-5 of the value.
    *e = expf(-0.5f * z * z);
    const float t = z * -0.70710678f;
    const float off = fmaf(z, -0.70710678f, -t) + z * -1.2101617e-8f;
    return 0.5f * erfcf(t) - (fabsf(z) < 16.0f ? off * *e * 0.56418958f : 0.0f);
  } else {
    *e = fast_exp(-0.5f * z * z);
    const float q = upper_tail(fabsf(z));
    return z > 0.0f ? 1.0f - q : q;
  }
}
template <int DT, int ACT>
__device__ inline float act_value(float z) {
  if constexpr (ACT == VR_ACT_RELU) {
    return z > 0.0f || z != z ? z : 0.0f;
  } else if constexpr (ACT == VR_ACT_GELU) {
    float e;
    return z * normal_cdf<DT>(z, &e);
  } else if constexpr (ACT == VR_ACT_SILU) {
    if constexpr (DT == VR_DT_F32) return z / (1.0f + expf(-z));
    else return z * sigmoid<DT>(z);
  } else {
    return z;
  }
}
template <int DT>
__device__ inline void act_both(float z, uint32_t act, float* y, float* dy) {
  switch (act & 0xFu) {
    case VR_ACT_RELU:
      *y = z > 0.0f || z != z ? z : 0.0f;
      *dy = z > 0.0f ? 1.0f : 0.0f;
      return;
    case VR_ACT_GELU: {
      float e;
      const float cdf = normal_cdf<DT>(z, &e);
      *y = z * cdf;
      *dy = cdf + z * e * 0.3989422804014327f;  // 1 / sqrt(2 pi)
      return;
    }
    case VR_ACT_SILU: {
      const float s = sigmoid<DT>(z);
      *y = z * s;
      *dy = s * (1.0f + z * (1.0f - s));
      return;
    }
    default:
      *y = z;
      *dy = 1.0f;
  }
}
// f(std::integral_constant<int, ACT>) for the activation in `act`.
template <class F>
inline void with_act(uint32_t act, F f) {
  switch (act & 0xFu) {
    case VR_ACT_RELU: return f(std::integral_constant<int, VR_ACT_RELU>());
    case VR_ACT_GELU: return f(std::integral_constant<int, VR_ACT_GELU>());
    case VR_ACT_SILU: return f(std::integral_constant<int, VR_ACT_SILU>());
    default: return f(std::integral_constant<int, VR_ACT_NONE>());
  }
}

// ---- wave reductions ------------------------------------------------------------------
// Lane l's partner in step S of a reduction, over vector instructions alone
// (a shuffle is a trip through the LDS, and the router waits for each): lanes
// 1 and 2 apart, then mirrored in 8 and in 16
// lanes (by then 4 and 8 lanes hold equal values), then rows 16 and 32 apart.
// The two values of a step are the same in both partners, so every lane gets
// the same result, bit for bit.
template <int S>
__device__ inline void dpp_pair(uint32_t v, uint32_t* a, uint32_t* b) {
  if constexpr (S < 4) {
    constexpr int kCtrl[4] = {0xB1, 0x4E, 0x141, 0x140};  // quad_perm 1,0,3,2 and 2,3,0,1; row_half_mirror; row_mirror
    *a = v;
    *b = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), kCtrl[S], 0xF, 0xF, false));
  } else {
    v2u r;
    if constexpr (S == 4) r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane16_swap(v, v, false, false));
    else r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane32_swap(v, v, false, false));
    *a = r[0];
    *b = r[1];
  }
}
template <int S, class T>
__device__ inline void lane_pair(T v, T* a, T* b) {
  if constexpr (sizeof(T) == 4) {
    uint32_t x, y;
    dpp_pair<S>(__builtin_bit_cast(uint32_t, v), &x, &y);
    *a = __builtin_bit_cast(T, x);
    *b = __builtin_bit_cast(T, y);
  } else {
    const v2u w = __builtin_bit_cast(v2u, v);
    v2u x, y;
    uint32_t x0, x1, y0, y1;
    dpp_pair<S>(w[0], &x0, &y0);
    dpp_pair<S>(w[1], &x1, &y1);
    x = v2u{x0, x1};
    y = v2u{y0, y1};
    *a = __builtin_bit_cast(T, x);
    *b = __builtin_bit_cast(T, y);
  }
}
// Steps [0, STEPS): 4 reduce rows of 16 lanes, 6 the wave; all lanes of a row
// (the wave) get the result.
template <int STEPS, int S = 0, class T, class F>
__device__ inline T lane_reduce(T v, F f) {
  if constexpr (S < STEPS) {
    T a, b;
    lane_pair<S>(v, &a, &b);
    return lane_reduce<STEPS, S + 1>(f(a, b), f);
  } else {
    return v;
  }
}
__device__ inline float wave_max(float v) {
  return lane_reduce<6>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float wave_sum(float v) {
  return lane_reduce<6>(v, [](float a, float b) { return a + b; });
}
__device__ inline double wave_max(double v) {
  return lane_reduce<6>(v, [](double a, double b) { return fmax(a, b); });
}
__device__ inline double wave_sum(double v) {
  return lane_reduce<6>(v, [](double a, double b) { return a + b; });
}

// ---- groups -------------------------------------------------------------------------
// A group's rows [first, first + count) of a rank, and its row tiles: the
// groups' tiles are counted in order from 0, each group's rows rounded up to
// whole tiles.
struct GroupTile {
  int g;      // -1: no such tile
  int first;  // first row of the group
  int count;  // its rows
  int tile0;  // its first tile
};

// The group that holds tile `want` (BY_GROUP: group `want` itself), tiles of
// bm rows. counts: the rank's [G] group_rows, or null (one group, all rows).
// Every lane of the wave calls it with the same arguments. A negative count is
// taken as 0, and rows past `rows` are left out; either sets
// VR_ASYNC_CAPACITY (the caller that asks for 0 looks at every count).
template <bool BY_GROUP>
__device__ inline GroupTile find_group(const int32_t* counts, int G, int rows, int bm, int want, uint32_t* err) {
  if (!counts) return {BY_GROUP || want < (rows + bm - 1) / bm ? 0 : -1, 0, rows, 0};
  const int lane = static_cast<int>(lane_id());
  int row0 = 0, tile0 = 0;
  bool bad = false;
  GroupTile t = {-1, 0, 0, 0};
  for (int g0 = 0; g0 < G; g0 += 64) {
    const int c = g0 + lane < G ? counts[g0 + lane] : 0;
    const int pos = max(c, 0);
    int64_t s = pos;  // sums of 64 counts pass 32 bits
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t o = __shfl_up(s, m);
      if (lane >= m) s += o;
    }
    const int64_t end = s + row0;
    const int lo = static_cast<int>(end - pos < rows ? end - pos : rows);
    const int hi = static_cast<int>(end < rows ? end : rows);
    bad |= c < 0 || end > rows;
    const int n = (hi - lo + bm - 1) / bm;
    int k = n;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(k, m);
      if (lane >= m) k += o;
    }
    const uint64_t here = BY_GROUP ? ballot(g0 + lane == want) : ballot(tile0 + k > want);
    if (here && t.g < 0) {
      const int src = __builtin_ctzll(here);
      t.g = g0 + src;
      t.first = __builtin_amdgcn_readlane(lo, src);
      t.count = __builtin_amdgcn_readlane(hi, src) - t.first;
      t.tile0 = tile0 + __builtin_amdgcn_readlane(k - n, src);
      if (want) break;
    }
    row0 = __builtin_amdgcn_readlane(hi, 63);
    tile0 += __builtin_amdgcn_readlane(k, 63);
  }
  if (ballot(bad) && lane == 0) atomic_or_u32(err, VR_ASYNC_CAPACITY);
  return t;
}

// ---- 16-byte pieces of a row -----------------------------------------------------------
// A whole piece; any element alignment.
template <int DT>
__device__ inline v4u load_whole(const char* p) {
  v4u v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, Elem<DT>::kSize), 16);
  return v;
}
// The piece's first n elements (n may be past either end of the piece), the
// others 0. Any element alignment.
template <int DT>
__device__ inline v4u load_piece(const char* p, int n) {
  v4u v = {0, 0, 0, 0};
  if (n >= Elem<DT>::kChunk) {
    v = load_whole<DT>(p);
  } else if (kInt8<DT>) {
    // the piece is inside its row: the values' end is followed by 4 bytes at least, and a row is a multiple of 128
    if (n > 0) {
      v = load_whole<DT>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] &= n >= 4 * j + 4 ? ~0u : n > 4 * j ? (1u << (8 * (n - 4 * j))) - 1 : 0u;
    }
  } else if (n > 0) {
#pragma unroll
    for (int j = 0; j < Elem<DT>::kChunk - 1; ++j) {
      if constexpr (DT == VR_DT_F32) {
        if (j < n) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
      } else {
        if (j < n) v[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
      }
    }
  }
  return v;
}

// Element j of a piece.
template <int DT>
__device__ inline float piece_f32(v4u v, int j) {
  if constexpr (DT == VR_DT_F32) return __uint_as_float(v[j]);
  else return (j & 1) ? bf16hi(v[j / 2]) : bf16lo(v[j / 2]);
}

// ---- matrix instructions -----------------------------------------------------------------
// acc[i][j] += sum_k a[i][k] b[j][k] over one 16-byte piece per lane: lane l
// holds elements k = (l / 16) * piece ... of row i = l % 16 of a and j = l % 16
// of b; of acc it holds i = (l / 16) * 4 + 0..3, j = l % 16. bf16: 32 k per
// call, fp32: 16, 8 bits: 64.
template <int DT>
__device__ inline Acc<DT> mfma_piece(v4u a, v4u b, Acc<DT> acc) {
  if constexpr (kInt8<DT>) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), acc, 0, 0, 0);
  } else if constexpr (DT == VR_DT_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[s]), __uint_as_float(b[s]), acc, 0, 0, 0);
    return acc;
  }
}


// acc[i][j] += w[i] . x[j] over contraction elements [k, k1), of which K exist:
// the lane's row of each of NW 16-row blocks of weights and NX of tokens, all
// read straight into registers, U steps of loads in flight. k is a multiple of
// the step. For products bound by the weights' bytes: nothing is shared
// through the LDS, so the loads never wait for a barrier.
template <int DT, int NW, int NX, int U>
__device__ inline void stream_products(const char* const* w, const char* const* x, int k, int k1, int K,
                                       Acc<DT> (*acc)[NX]) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kStep = 4 * kC;
  const int q = (lane_id() >> 4) * kC;
  v4u wv[U][NW], xv[U][NX];
  auto use = [&](int u) {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int j = 0; j < NX; ++j) acc[i][j] = mfma_piece<DT>(wv[u][i], xv[u][j], acc[i][j]);
  };
  for (; k + U * kStep <= min(k1, K); k += U * kStep) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t at = (uint64_t)(k + u * kStep + q) * kES;
#pragma unroll
      for (int i = 0; i < NW; ++i) wv[u][i] = load_whole<DT>(w[i] + at);
#pragma unroll
      for (int j = 0; j < NX; ++j) xv[u][j] = load_whole<DT>(x[j] + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) use(u);
  }
  for (; k < k1; k += kStep) {
    const uint64_t at = (uint64_t)(k + q) * kES;
#pragma unroll
    for (int i = 0; i < NW; ++i) wv[0][i] = load_piece<DT>(w[i] + at, K - k - q);
#pragma unroll
    for (int j = 0; j < NX; ++j) xv[0][j] = load_piece<DT>(x[j] + at, K - k - q);
    use(0);
  }
}

}  // namespace vr
