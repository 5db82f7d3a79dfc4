// Rows of windows: the root-mean-square norm with the residual's addition and
// its gradients (vr_norm, vr_norm_backward), and rows in 8 bits
// (vr_quantize, vr_dequantize).
//
//   norm      h = round(x + residual); y = h / r * gain, r = sqrt(mean h^2 + eps)
//   gradient  n = h / r, g = dout * gain: dh = dsum + (g - n mean(g n)) / r;
//             dgain = sum over rows of dout n
//   8 bits    m = max |x|: scale = m / 127, value = rint(x * (127 / m)); 127 scales are a number
//
// All are bound by memory: a row is read once, held in registers between its
// reductions and its outputs, and everything that is made of it is written in
// the same pass. Rates below are bytes read and written once over a kernel's
// time; a large copy reaches 6.9 TB/s on this card.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "vr_layers.hpp"

namespace vr {
namespace {

typedef v4u v4u_any __attribute__((aligned(2)));  // at any element's alignment
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kLeastBits = 0x04000000u;  // 2^-119: 1/127 of less would be subnormal
constexpr float kMostScale = 0x1.020406p121f;  // 127 times the next is infinite, and the largest number's 1/127 rounds to that

struct RowArgs {
  WinTab x, residual, gain, sum, out, q8;
  const int32_t* counts;  // [R][G] or null
  uint32_t* err;
  int G, rows, cols;
  float eps;
  uint64_t row8;  // bytes of a q8 row
};

// Rows of rank r that belong to a group: all without counts. Every lane of a
// wave calls it.
__device__ inline int used_rows(const int32_t* counts, int r, int G, int rows, uint32_t* err) {
  if (!counts) return rows;
  const int lane = static_cast<int>(lane_id());
  int64_t n = 0;
  bool bad = false;
  for (int g = lane; g < G; g += 64) {
    const int c = counts[(size_t)r * G + g];
    n += max(c, 0);
    bad |= c < 0;
  }
  n = lane_reduce<6>(n, [](int64_t a, int64_t b) { return a + b; });
  bad |= n > rows;
  if (ballot(bad) && lane == 0) atomic_or_u32(err, VR_ASYNC_CAPACITY);
  return static_cast<int>(n < rows ? n : rows);
}

// A reduction over the TPR threads of a row: waves by lane exchange, their
// results through `red` (TPR / 64 words that nobody else reads until the
// workgroup's next barrier but one). Every thread gets the same result.
template <int TPR, class T, class F>
__device__ inline T row_reduce(T v, T* red, F f) {
  v = lane_reduce<6>(v, f);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = f(v, red[w]);
  }
  return v;
}
struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
__device__ inline uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// How a row of largest magnitude m (as bits: a NaN's are above infinity's)
// becomes one of 8 bits.
struct To8 {
  float mul, scale;
  bool zero;  // all values 0
};
__device__ inline To8 to_8(uint32_t m) {
  if (m >= kInfBits) return {0.0f, __uint_as_float(0x7FC00000u), true};
  if (m < kLeastBits) return {0.0f, 0.0f, true};
  return {127.0f / __uint_as_float(m), fminf(__uint_as_float(m) / 127.0f, kMostScale), false};
}
// Four values as bytes: added to 1.5 * 2^23 a product is rounded to a whole
// number, to nearest even and once, whose low byte is the sum's.
__device__ inline uint32_t bytes4(const float* f, const To8& q) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(fmaf(f[j], q.mul, 12582912.0f));
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
  return q.zero ? 0u : lo | hi;
}

// The N = 4 or 8 values of columns [col, col + N) of a q8 row; the last n of
// the row's values. ALIGN: of col, in bytes (rows start on words).
template <int N, int ALIGN>
__device__ inline void store_bytes(char* row, int col, int n, const float* f, const To8& q) {
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = bytes4(f + 4 * i, q);
  if (n >= N) {
    __builtin_memcpy(__builtin_assume_aligned(row + col, ALIGN), w, N);
  } else {
#pragma unroll
    for (int j = 0; j < N - 1; ++j)
      if (j < n) row[col + j] = static_cast<char>(w[j / 4] >> (8 * (j % 4)));
  }
}
// The zeros and the scale behind the values: up to 3 bytes, then 32-bit words. t of
// TPR >= 64 threads.
__device__ inline void store_scale(char* row, int cols, uint64_t row8, int t, const To8& q) {
  const int first = (cols + 3) & ~3, words = static_cast<int>(row8 - first) / 4;  // at most 32
  if (t < words) {
    reinterpret_cast<uint32_t*>(row + first)[t] = t == words - 1 ? __float_as_uint(q.scale) : 0u;
  } else if (t - 32 >= 0 && t - 32 < first - cols) {
    row[cols + t - 32] = 0;
  }
}

// A thread's piece p of a row of TPR threads side by side, 16 bytes to each. A
// row that is no multiple of a piece ends in one that starts early: its first
// `again` elements are another thread's too. All of a piece's (kChunk or more):
// it is past the end.
struct Piece {
  int at, again;
};
template <int DT, int TPR>
__device__ inline Piece piece(int p, int t, int cols) {
  constexpr int kC = Elem<DT>::kChunk;
  const int col = (p * TPR + t) * kC, at = min(col, cols - kC);
  return {at, col - at};
}
// A thread's P pieces of a row of at least one piece.
template <int DT, int TPR, int P>
__device__ inline void load_row(const char* row, int cols, int t, v4u* v) {
#pragma unroll
  for (int p = 0; p < P; ++p) v[p] = load_whole<DT>(row + (size_t)piece<DT, TPR>(p, t, cols).at * Elem<DT>::kSize);
}
// How a kernel takes its rows: of any length; of whole pieces; of whole pieces
// and past the caches, where all that a call reads and writes is more than the
// last of them holds (256 MiB). There that took 109 to 99 us off the gradients of
// 8 x 2048 rows of 4096 bf16 and 90 to 79 off 8 x 4096 rows of 2048 to 8 bits; rows
// that a cache holds it slows (4 x 8192 rows of 512 to 8 bits: 13 to 16 us).
enum Mode { kAny, kWhole, kStream };
constexpr int64_t kCacheBytes = 256ll << 20;
template <int DT, int TPR, int P, int MODE>
__device__ inline void load_once(const char* row, int cols, int t, v4u* v) {
  if constexpr (MODE == kStream) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      v[p] = __builtin_nontemporal_load(reinterpret_cast<const v4u_any*>(row + (size_t)piece<DT, TPR>(p, t, cols).at * Elem<DT>::kSize));
  } else {
    load_row<DT, TPR, P>(row, cols, t, v);
  }
}
template <int DT, int MODE>
__device__ inline void store_once(char* row, int col, const float* f) {
  if constexpr (MODE == kStream) {
    v4u v;
    store_n<DT, Elem<DT>::kChunk>(&v, 0, f);
    __builtin_nontemporal_store(v, reinterpret_cast<v4u_any*>(row + (size_t)col * Elem<DT>::kSize));
  } else {
    store_n<DT, Elem<DT>::kChunk>(row, col, f);
  }
}
template <int DT>
__device__ inline void widen(v4u v, float* f) {
#pragma unroll
  for (int j = 0; j < Elem<DT>::kChunk; ++j) f[j] = piece_f32<DT>(v, j);
}
// f(value, p, j) for the values of h that are this thread's alone. WHOLE: rows of whole pieces.
template <int DT, int TPR, int P, bool WHOLE, class F>
__device__ inline void each(int t, int cols, F f) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int again = piece<DT, TPR>(p, t, cols).again;
    if (WHOLE) {
      if (again == 0) {
#pragma unroll
        for (int j = 0; j < Elem<DT>::kChunk; ++j) f(p, j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < Elem<DT>::kChunk; ++j)
        if (j >= again) f(p, j);
    }
  }
}
// f(p, first column) for the pieces that are stored.
template <int DT, int TPR, int P, class F>
__device__ inline void each_piece(int t, int cols, F f) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const Piece q = piece<DT, TPR>(p, t, cols);
    if (q.again < Elem<DT>::kChunk) f(p, q.at);
  }
}
// Of the kernels that take rows of any length: the piece at column col, elements past the end not stored.
template <int DT>
__device__ inline void store_piece(char* row, int col, int cols, const float* f) {
  constexpr int kC = Elem<DT>::kChunk;
  if (cols - col >= kC) {
    store_n<DT, kC>(row, col, f);
  } else {
#pragma unroll
    for (int j = 0; j < kC - 1; ++j)
      if (j < cols - col) Elem<DT>::store(row, col + j, f[j]);
  }
}

// The square of a row's root, and 1 / root.
__device__ inline float root_square(float ss, int cols, float eps) { return ss / static_cast<float>(cols) + eps; }
__device__ inline float inverse_root(float ss, int cols, float eps) { return 1.0f / sqrtf(root_square(ss, cols, eps)); }
// What a row whose squares, or the root's square, pass binary32 is multiplied by
// before they are taken: a power of two that brings its largest magnitude (bits m, finite) to
// [1, 2). *bad: m is no number, and the root is infinite or NaN.
__device__ inline float down(uint32_t m, bool* bad) {
  *bad = m >= kInfBits;
  return ldexpf(1.0f, 127 - static_cast<int>(m >> 23));
}
// A gradient's row is taken again where the root's square is no binary32 number, or
// the mean of g n is so large that its product with an n (2^10 at most, the root of
// the most columns) could take the largest g past binary32, by half a step of 2^104: h
// is then brought below 2 and g below 2^65, where they are not, by powers of two. Sums
// of 2^20 products of those stay inside binary32.
constexpr float kMostMean = 0x1p93f;
__device__ inline bool again_scaled(float square, float mean) { return !(square < INFINITY && fabsf(mean) < kMostMean); }
struct Scales {
  float h, g, back;  // back = h / g, what brings the scaled row's gradient back
  bool bad;          // a value of h is no number, and the root is infinite or NaN
};
__device__ inline Scales scales_of(uint32_t mh, uint32_t mg) {  // largest magnitudes, as bits
  const int eh = max(static_cast<int>(mh >> 23) - 127, 0), eg = mg < kInfBits ? max(static_cast<int>(mg >> 23) - 191, 0) : 0;
  return {ldexpf(1.0f, -eh), ldexpf(1.0f, -eg), ldexpf(1.0f, eg - eh), mh >= kInfBits};
}

// Threads of a workgroup whose rows take TPR.
constexpr int threads_of(int tpr) { return tpr == 64 ? 256 : tpr; }

// A row to TPR threads (one wave: four rows to a workgroup), P pieces to a
// thread. NORM: the norm; else x itself, to 8 bits. A wave reduces its row
// without a barrier and takes up to 4 pieces of it; longer rows take as many
// threads as that needs. 8 x 4096 rows of 2048 bf16 with residual, sum and rows in
// 8 bits: 78 us, 6.0 TB/s; 4 x 8192 rows of 512 to 8 bits by group counts: 11 us; one
// row of 4096: 2.9 us, a launch. fp32: 8 x 2048 rows of 4096 with residual, sum and
// out 153 us, 7.0 TB/s. Four bf16 pieces to each of 1024 threads are too many: 33
// registers of them, the gain's in the main, lie in scratch, and 4096 rows of 12288
// take 270 us, 1.5 TB/s (to 8 bits, without gain or residual, 36).
template <int DT, int TPR, int P, bool NORM, int MODE>
__global__ __launch_bounds__(threads_of(TPR)) void k_rows(const RowArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kRows = threads_of(TPR) / TPR, kW = TPR / 64;
  __shared__ float red_sum[2][kW];
  __shared__ uint32_t red_max[2][kW];
  const int r = blockIdx.y, t = threadIdx.x % TPR, cols = a.cols;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  v4u gv[P];
  if (NORM && a.gain.p[r]) load_row<DT, TPR, P>(a.gain.p[r], cols, t, gv);
  v4u xn[P], rn[P];
  const auto fetch = [&](int row) {
    const uint64_t at = (uint64_t)row * cols * kES;
    load_once<DT, TPR, P, MODE>(a.x.p[r] + at, cols, t, xn);
    if (NORM && a.residual.p[r]) load_once<DT, TPR, P, MODE>(a.residual.p[r] + at, cols, t, rn);
  };
  int flip = 0, row = blockIdx.x * kRows + slot;
  if (row < a.rows) fetch(row);  // reads on before it is known whether a group holds it
  const int used = used_rows(a.counts, r, a.G, a.rows, a.err);
  for (; row < used; row += gridDim.x * kRows, flip ^= 1) {
    const uint64_t at = (uint64_t)row * cols * kES;
    v4u xv[P], rv[P];
#pragma unroll
    for (int p = 0; p < P; ++p) xv[p] = xn[p], rv[p] = rn[p];
    if (row + (int)gridDim.x * kRows < used) fetch(row + gridDim.x * kRows);
    float h[P][kC];
#pragma unroll
    for (int p = 0; p < P; ++p) widen<DT>(xv[p], h[p]);
    if constexpr (NORM) {
      if (a.residual.p[r]) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float f[kC];
          widen<DT>(rv[p], f);
#pragma unroll
          for (int j = 0; j < kC; ++j) h[p][j] = Elem<DT>::round(h[p][j] + f[j]);
        }
      }
      float ss = 0.0f;
      each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) { ss = fmaf(h[p][j], h[p][j], ss); });
      ss = row_reduce<TPR>(ss, red_sum[flip], Add());
      // only here: sum may lie where residual does, and where two threads share columns both have read them now
      if (a.sum.p[r]) each_piece<DT, TPR, P>(t, cols, [&](int p, int col) { store_once<DT, MODE>(a.sum.p[r] + at, col, h[p]); });
      float inv = inverse_root(ss, cols, a.eps);
      if (!(root_square(ss, cols, a.eps) < INFINITY)) {  // the same in all of the row's threads
        uint32_t m = 0;
        each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) { m = max(m, magnitude(h[p][j])); });
        m = row_reduce<TPR>(m, red_max[flip], Max());
        if (TPR > 64) __syncthreads();  // both words are written again
        bool bad;
        const float f = down(m, &bad);
        if (!bad) {
          ss = 0.0f;
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < kC; ++j) h[p][j] *= f;
          each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) { ss = fmaf(h[p][j], h[p][j], ss); });
          ss = row_reduce<TPR>(ss, red_sum[flip], Add());
          inv = inverse_root(ss, cols, a.eps * f * f);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float f[kC];
        widen<DT>(gv[p], f);
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          h[p][j] *= inv;
          if (a.gain.p[r]) h[p][j] *= f[j];
        }
      }
      if (a.out.p[r]) each_piece<DT, TPR, P>(t, cols, [&](int p, int col) { store_n<DT, kC>(a.out.p[r] + at, col, h[p]); });
    }
    if (!NORM || a.q8.p[r]) {
      uint32_t m = 0;
      each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) { m = max(m, magnitude(h[p][j])); });
      m = row_reduce<TPR>(m, red_max[flip], Max());
      const To8 q = to_8(m);
      if (m >= kInfBits && t == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
      char* to = a.q8.p[r] + (uint64_t)row * a.row8;
      each_piece<DT, TPR, P>(t, cols, [&](int p, int col) { store_bytes<kC, MODE == kAny ? 1 : 4>(to, col, kC, h[p], q); });
      store_scale(to, cols, a.row8, t, q);
    }
  }
}

// Rows too long for registers (and those of less than a piece): a workgroup
// reads its row again for each step.
constexpr int kLongThreads = 1024;
template <int DT, bool NORM>
__global__ __launch_bounds__(kLongThreads) void k_rows_long(const RowArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, T = kLongThreads;
  __shared__ float red_sum[T / 64];
  __shared__ uint32_t red_max[T / 64];
  const int r = blockIdx.y, t = threadIdx.x;
  const int used = used_rows(a.counts, r, a.G, a.rows, a.err);
  for (int row = blockIdx.x; row < used; row += gridDim.x) {
    const uint64_t at = (uint64_t)row * a.cols * kES;
    // h of the piece from column col; after the first step from sum, where that is written (it may be residual's own slice)
    const auto get = [&](int col, bool first, float* h) {
      const char* from = NORM && !first && a.sum.p[r] ? a.sum.p[r] : a.x.p[r];
      widen<DT>(load_piece<DT>(from + at + (uint64_t)col * kES, a.cols - col), h);
      if (!NORM || !a.residual.p[r] || from != a.x.p[r]) return;
      float f[kC];
      widen<DT>(load_piece<DT>(a.residual.p[r] + at + (uint64_t)col * kES, a.cols - col), f);
#pragma unroll
      for (int j = 0; j < kC; ++j) h[j] = Elem<DT>::round(h[j] + f[j]);
    };
    float inv = 1.0f, by = 1.0f;
    if constexpr (NORM) {
      float ss = 0.0f;
      for (int col = t * kC; col < a.cols; col += T * kC) {
        float h[kC];
        get(col, true, h);
        if (a.sum.p[r]) store_piece<DT>(a.sum.p[r] + at, col, a.cols, h);
#pragma unroll
        for (int j = 0; j < kC; ++j) ss = fmaf(h[j], h[j], ss);
      }
      ss = row_reduce<T>(ss, red_sum, Add());
      inv = inverse_root(ss, a.cols, a.eps);
      __syncthreads();
      if (!(root_square(ss, a.cols, a.eps) < INFINITY)) {
        uint32_t m = 0;
        for (int col = t * kC; col < a.cols; col += T * kC) {
          float h[kC];
          get(col, false, h);
#pragma unroll
          for (int j = 0; j < kC; ++j) m = max(m, magnitude(h[j]));
        }
        m = row_reduce<T>(m, red_max, Max());
        __syncthreads();
        bool bad;
        const float f = down(m, &bad);
        if (!bad) {
          by = f;
          ss = 0.0f;
          for (int col = t * kC; col < a.cols; col += T * kC) {
            float h[kC];
            get(col, false, h);
#pragma unroll
            for (int j = 0; j < kC; ++j) ss = fmaf(h[j] * by, h[j] * by, ss);
          }
          ss = row_reduce<T>(ss, red_sum, Add());
          __syncthreads();
          inv = inverse_root(ss, a.cols, a.eps * by * by);
        }
      }
    }
    const auto value = [&](int col, float* y) {
      get(col, false, y);
      if constexpr (NORM) {
        float f[kC];
        if (a.gain.p[r]) widen<DT>(load_piece<DT>(a.gain.p[r] + (uint64_t)col * kES, a.cols - col), f);
#pragma unroll
        for (int j = 0; j < kC; ++j) y[j] = y[j] * by * inv * (a.gain.p[r] ? f[j] : 1.0f);
      }
    };
    const bool quant = !NORM || a.q8.p[r];
    To8 q = {};
    if (quant) {
      uint32_t m = 0;
      for (int col = t * kC; col < a.cols; col += T * kC) {
        float y[kC];
        value(col, y);
#pragma unroll
        for (int j = 0; j < kC; ++j)
          if (col + j < a.cols) m = max(m, magnitude(y[j]));
      }
      m = row_reduce<T>(m, red_max, Max());
      q = to_8(m);
      if (m >= kInfBits && t == 0) atomic_or_u32(a.err, VR_ASYNC_BAD_VALUE);
    }
    char* to = quant ? a.q8.p[r] + (uint64_t)row * a.row8 : nullptr;
    for (int col = t * kC; col < a.cols; col += T * kC) {
      float y[kC];
      value(col, y);
      if (NORM && a.out.p[r]) store_piece<DT>(a.out.p[r] + at, col, a.cols, y);
      if (quant) store_bytes<kC, 4>(to, col, a.cols - col, y, q);
    }
    if (quant) store_scale(to, a.cols, a.row8, t, q);
    __syncthreads();  // red_max is read until here
  }
}

// A launch holds fewer than 2^32 threads in a direction: workgroups take further rows in turn.
uint32_t row_grid(int64_t blocks) { return static_cast<uint32_t>(std::min<int64_t>(blocks, 1 << 21)); }

template <int DT, int TPR, int P, bool NORM>
void start_rows(const RowArgs& a, int R, hipStream_t st) {
  constexpr int kRows = threads_of(TPR) / TPR;
  // Rows of a piece to a lane are little work for a wave: where there are many, 2048 workgroups take several each, the next
  // row on its way (4 x 8192 rows of 512 to 8 bits, which also count their groups' rows first: 13 to 11 us). Longer rows
  // lose by it (8 x 4096 rows of 2048: 79 to 84 us).
  const uint32_t blocks = row_grid((a.rows + kRows - 1) / kRows);
  const dim3 grid(TPR == 64 && P == 1 ? std::min(blocks, 2048u / R) : blocks, R);
  const int64_t n = (int64_t)R * a.rows * a.cols;
  int64_t bytes = n * Elem<DT>::kSize * (1 + (a.residual.p[0] != nullptr) + (a.sum.p[0] != nullptr) + (a.out.p[0] != nullptr));
  if (a.q8.p[0]) bytes += n;
  if (a.cols % Elem<DT>::kChunk) hipLaunchKernelGGL((k_rows<DT, TPR, P, NORM, kAny>), grid, dim3(threads_of(TPR)), 0, st, a);
  else if (bytes > kCacheBytes) hipLaunchKernelGGL((k_rows<DT, TPR, P, NORM, kStream>), grid, dim3(threads_of(TPR)), 0, st, a);
  else hipLaunchKernelGGL((k_rows<DT, TPR, P, NORM, kWhole>), grid, dim3(threads_of(TPR)), 0, st, a);
}
template <int DT, bool NORM>
vrResult_t start(const RowArgs& a, int R, hipStream_t st) {
  const int pieces = (a.cols + Elem<DT>::kChunk - 1) / Elem<DT>::kChunk;
  if (a.cols < Elem<DT>::kChunk || pieces > 4096)
    hipLaunchKernelGGL((k_rows_long<DT, NORM>), dim3(row_grid(a.rows), R), dim3(kLongThreads), 0, st, a);
  else if (pieces <= 64) start_rows<DT, 64, 1, NORM>(a, R, st);
  else if (pieces <= 128) start_rows<DT, 64, 2, NORM>(a, R, st);
  else if (pieces <= 256) start_rows<DT, 64, 4, NORM>(a, R, st);
  else if (pieces <= 512) start_rows<DT, 256, 2, NORM>(a, R, st);
  else if (pieces <= 1024) start_rows<DT, 256, 4, NORM>(a, R, st);
  else start_rows<DT, 1024, 4, NORM>(a, R, st);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

// ---- from 8 bits ---------------------------------------------------------------------------
// 8 values to a thread, LPR threads side by side, further ones in turn. Bound by
// memory: 8 x 4096 rows of 2048 to bf16: 30 us, 6.8 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void k_from_8(const RowArgs a, int lpr_log) {
  const int r = blockIdx.y, lpr = 1 << lpr_log, t = threadIdx.x & (lpr - 1), rows = 256 >> lpr_log;
  const int used = used_rows(a.counts, r, a.G, a.rows, a.err);
  for (int row = blockIdx.x * rows + (threadIdx.x >> lpr_log); row < used; row += gridDim.x * rows) {
    const char* from = a.q8.p[r] + (uint64_t)row * a.row8;
    char* to = a.out.p[r] + (uint64_t)row * a.cols * Elem<DT>::kSize;
    const float scale = *reinterpret_cast<const float*>(from + a.row8 - 4);
    for (int col = t * 8; col < a.cols; col += lpr * 8) {
      v2u w;  // inside the row: at least 4 bytes follow the values, and a row is a multiple of 128
      __builtin_memcpy(&w, __builtin_assume_aligned(from + col, 4), 8);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)))) * scale;
      if (a.cols - col >= 8) {
        store_n<DT, 8>(to, col, f);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < a.cols - col) Elem<DT>::store(to, col + j, f[j]);
      }
    }
  }
}

// ---- gradients -------------------------------------------------------------------------------
struct BackArgs {
  WinTab dout, h, gain, dsum, dh, dgain;
  float* partial;  // [R][slots][cols] sums of dout n over a workgroup's rows, or null
  float* roots;    // [R][rows][2], long rows: the factor for h and 1 / root of the product
  int rows, cols, slots;
  float eps;
};

// The least waves to a SIMD that a gradient's registers have to leave room for: 64 registers let two workgroups of 16 waves
// onto a compute unit, which the compiler misses by five (2000 rows of 4096 fp32: 25.4 us, else 27.4); the other modes
// would spill.
template <int DT, int TPR, int P, int MODE>
constexpr int kBackWaves = DT == VR_DT_F32 && TPR == 1024 && P == 1 && MODE == kWhole ? 8 : 1;

// A row to TPR threads as above. Workgroup x takes rows x, x + slots, ... (of
// one wave: four at a time) and keeps its columns' sums for dgain in registers:
// the sums of a whole rank would be atomics, whose order changes results, and one
// row of sums per row another pass over the data. Three rows are read for one that
// is written: 8 x 2048 rows of 4096 bf16 with dsum and dgain 98 us, 5.5 TB/s (other
// threads to a row and 512 to 2048 slots: 98 to 104); fp32 5.0 to 5.6 TB/s.
template <int DT, int TPR, int P, int MODE>
__global__ __launch_bounds__(threads_of(TPR), (kBackWaves<DT, TPR, P, MODE>)) void k_norm_back(const BackArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, kRows = threads_of(TPR) / TPR, kW = TPR / 64;
  __shared__ float red[2][2][kW];
  __shared__ uint32_t red_max[2][kW];
  const int r = blockIdx.y, t = threadIdx.x % TPR, cols = a.cols;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const bool gained = a.gain.p[r] != nullptr, more = a.dsum.p[r] != nullptr;
  float acc[P][kC];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < kC; ++j) acc[p][j] = 0.0f;
  v4u gv[P];
  if (gained) load_row<DT, TPR, P>(a.gain.p[r], cols, t, gv);
  v4u hn[P], dn[P], sn[P];
  const auto fetch = [&](int row) {
    const uint64_t at = (uint64_t)row * cols * kES;
    load_once<DT, TPR, P, MODE>(a.h.p[r] + at, cols, t, hn);
    load_once<DT, TPR, P, MODE>(a.dout.p[r] + at, cols, t, dn);
    if (more) load_once<DT, TPR, P, MODE>(a.dsum.p[r] + at, cols, t, sn);
  };
  int flip = 0, row = blockIdx.x * kRows + slot;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += gridDim.x * kRows, flip ^= 1) {
    const uint64_t at = (uint64_t)row * cols * kES;
    v4u hv[P], dv[P], sv[P];
#pragma unroll
    for (int p = 0; p < P; ++p) hv[p] = hn[p], dv[p] = dn[p], sv[p] = sn[p];
    if (row + (int)gridDim.x * kRows < a.rows) fetch(row + gridDim.x * kRows);
    if constexpr (MODE == kAny && TPR > 64) {
      // dh may lie where dsum does: where two threads share columns both have read them before the workgroup meets in sums()
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (more) asm volatile("" : "+v"(sv[p]));
    }
    float by = 1.0f, gby = 1.0f, back = 1.0f, ss = 0.0f, sg = 0.0f;
    const auto weighted = [&](int p, int j) {
      const float d = piece_f32<DT>(dv[p], j);
      return gained ? d * piece_f32<DT>(gv[p], j) : d;
    };
    const auto sums = [&] {
      ss = sg = 0.0f;
      each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) {
        const float h = piece_f32<DT>(hv[p], j) * by;
        ss = fmaf(h, h, ss);
        sg = fmaf(weighted(p, j) * gby, h, sg);
      });
      ss = wave_sum(ss);
      sg = wave_sum(sg);
      if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) {
          red[flip][0][threadIdx.x >> 6] = ss;
          red[flip][1][threadIdx.x >> 6] = sg;
        }
        __syncthreads();
        ss = red[flip][0][0];
        sg = red[flip][1][0];
#pragma unroll
        for (int w = 1; w < kW; ++w) {
          ss += red[flip][0][w];
          sg += red[flip][1][w];
        }
      }
    };
    const auto mean_gn = [&](float inv) { return sg * inv / static_cast<float>(cols); };
    sums();
    float inv = inverse_root(ss, cols, a.eps), mean = mean_gn(inv);
    if (again_scaled(root_square(ss, cols, a.eps), mean)) {
      // here and below, as if read anew: the compiler keeps widened values across this seldom way otherwise, and of bf16 spills one
      if constexpr (TPR == 1024 && P == 2) {
#pragma unroll
        for (int p = 0; p < P; ++p) asm volatile("" : "+v"(dv[p]));
      }
      uint32_t mh = 0, mg = 0;
      each<DT, TPR, P, MODE != kAny>(t, cols, [&](int p, int j) {
        mh = max(mh, magnitude(piece_f32<DT>(hv[p], j)));
        mg = max(mg, magnitude(weighted(p, j)));
      });
      mh = row_reduce<TPR>(mh, red_max[0], Max());
      mg = row_reduce<TPR>(mg, red_max[1], Max());
      if (TPR > 64) __syncthreads();  // red is written again, and red_max by the next such row
      const Scales f = scales_of(mh, mg);
      if (!f.bad) {
        by = f.h;
        gby = f.g;
        back = f.back;
        sums();
        inv = inverse_root(ss, cols, a.eps * by * by);
        mean = mean_gn(inv);
      }
      if constexpr (TPR == 1024 && P == 2) {
#pragma unroll
        for (int p = 0; p < P; ++p) asm volatile("" : "+v"(dv[p]));
      }
    }
    each_piece<DT, TPR, P>(t, cols, [&](int p, int col) {
      float v[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const float n = piece_f32<DT>(hv[p], j) * by * inv, d = piece_f32<DT>(dv[p], j);
        acc[p][j] = fmaf(d, n, acc[p][j]);
        v[j] = (weighted(p, j) * gby - n * mean) * inv * back;
        if (more) v[j] += piece_f32<DT>(sv[p], j);
      }
      if (a.dh.p[r]) store_once<DT, MODE>(a.dh.p[r] + at, col, v);
    });
  }
  if (!a.partial) return;
  float* out = a.partial + ((uint64_t)r * a.slots + blockIdx.x) * cols;
  if constexpr (kRows > 1) {
    __shared__ float part[kRows][P * 64 * kC];  // two threads that share a column hold the same sum
    each_piece<DT, TPR, P>(t, cols, [&](int p, int col) {
#pragma unroll
      for (int j = 0; j < kC; ++j) part[slot][col + j] = acc[p][j];
    });
    __syncthreads();
    for (int i = threadIdx.x; i < cols; i += 256) {
      float s = part[0][i];
#pragma unroll
      for (int w = 1; w < kRows; ++w) s += part[w][i];
      out[i] = s;
    }
  } else {
    each_piece<DT, TPR, P>(t, cols, [&](int p, int col) {
#pragma unroll
      for (int j = 0; j < kC; j += 4) store_n<VR_DT_F32, 4>(out, col + j, acc[p] + j);
    });
  }
}

// Rows too long for registers (and those of less than a piece): dh, and the
// roots for the sums of dgain. h and dout are read twice here and once more for
// dgain: 2048 rows of 32768 bf16 with dsum 287 us, 1.9 TB/s of what is needed once.
template <int DT>
__global__ __launch_bounds__(kLongThreads) void k_norm_back_long(const BackArgs a) {
  constexpr int kC = Elem<DT>::kChunk, kES = Elem<DT>::kSize, T = kLongThreads;
  __shared__ float red[2][T / 64];
  __shared__ uint32_t red_max[2][T / 64];
  const int r = blockIdx.y, t = threadIdx.x;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint64_t at = (uint64_t)row * a.cols * kES;
    const auto get = [&](const char* base, uint64_t from, int col, float* f) {
      widen<DT>(load_piece<DT>(base + from + (uint64_t)col * kES, a.cols - col), f);
    };
    // g of the piece: dout * gain
    const auto weighted = [&](int col, float* g) {
      get(a.dout.p[r], at, col, g);
      if (!a.gain.p[r]) return;
      float f[kC];
      get(a.gain.p[r], 0, col, f);
#pragma unroll
      for (int j = 0; j < kC; ++j) g[j] *= f[j];
    };
    float by = 1.0f, gby = 1.0f, back = 1.0f, ss, sg;
    const auto sums = [&] {
      ss = sg = 0.0f;
      for (int col = t * kC; col < a.cols; col += T * kC) {
        float h[kC], g[kC];
        get(a.h.p[r], at, col, h);
        weighted(col, g);
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          ss = fmaf(h[j] * by, h[j] * by, ss);
          sg = fmaf(g[j] * gby, h[j] * by, sg);
        }
      }
      ss = row_reduce<T>(ss, red[0], Add());
      sg = row_reduce<T>(sg, red[1], Add());
      __syncthreads();
    };
    const auto mean_gn = [&](float inv) { return sg * inv / static_cast<float>(a.cols); };
    sums();
    float inv = inverse_root(ss, a.cols, a.eps), mean = mean_gn(inv);
    if (again_scaled(root_square(ss, a.cols, a.eps), mean)) {
      uint32_t mh = 0, mg = 0;
      for (int col = t * kC; col < a.cols; col += T * kC) {
        float h[kC], g[kC];
        get(a.h.p[r], at, col, h);
        weighted(col, g);
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          mh = max(mh, magnitude(h[j]));
          mg = max(mg, magnitude(g[j]));
        }
      }
      mh = row_reduce<T>(mh, red_max[0], Max());
      mg = row_reduce<T>(mg, red_max[1], Max());
      __syncthreads();
      const Scales f = scales_of(mh, mg);
      if (!f.bad) {
        by = f.h;
        gby = f.g;
        back = f.back;
        sums();
        inv = inverse_root(ss, a.cols, a.eps * by * by);
        mean = mean_gn(inv);
      }
    }
    if (t == 0 && a.roots) {
      a.roots[((uint64_t)r * a.rows + row) * 2] = by;
      a.roots[((uint64_t)r * a.rows + row) * 2 + 1] = inv;
    }
    if (!a.dh.p[r]) continue;
    for (int col = t * kC; col < a.cols; col += T * kC) {
      float h[kC], g[kC], s[kC];
      get(a.h.p[r], at, col, h);
      weighted(col, g);
      if (a.dsum.p[r]) get(a.dsum.p[r], at, col, s);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const float n = h[j] * by * inv, v = (g[j] * gby - n * mean) * inv * back;
        g[j] = a.dsum.p[r] ? v + s[j] : v;
      }
      store_piece<DT>(a.dh.p[r] + at, col, a.cols, g);
    }
  }
}
// ... and these sums: 256 columns to a workgroup, every slots-th row.
template <int DT>
__global__ __launch_bounds__(256) void k_dgain_long(const BackArgs a) {
  const int r = blockIdx.z, col = blockIdx.y * 256 + threadIdx.x;
  if (col >= a.cols) return;
  float s = 0.0f;
#pragma unroll 4
  for (int row = blockIdx.x; row < a.rows; row += a.slots) {
    const float* q = a.roots + ((uint64_t)r * a.rows + row) * 2;
    const uint64_t at = (uint64_t)row * a.cols + col;
    s = fmaf(Elem<DT>::load(a.dout.p[r], at), Elem<DT>::load(a.h.p[r], at) * q[0] * q[1], s);
  }
  a.partial[((uint64_t)r * a.slots + blockIdx.x) * a.cols + col] = s;
}

// dgain of 32 columns: 32 half waves take every 32nd slot each, and their sums
// are added in order. 17 MB of sums, which the last cache still holds: 5 us.
template <int DT>
__global__ __launch_bounds__(1024) void k_dgain(const BackArgs a) {
  const int r = blockIdx.y, lane = threadIdx.x & 31, part = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const float* p = a.partial + (uint64_t)r * a.slots * a.cols + min(col, a.cols - 1);
  float s = 0.0f;
#pragma unroll 8
  for (int i = part; i < a.slots; i += 32) s += p[(uint64_t)i * a.cols];
  __shared__ float sum[32][32];
  sum[part][lane] = s;
  __syncthreads();
  if (part || col >= a.cols) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += sum[w][lane];
  Elem<DT>::store(a.dgain.p[r], col, s);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct BackLayout {
  int tpr, pieces;  // threads to a row, pieces to a thread; 0: long rows
  int slots;
  size_t roots, total;
};
BackLayout back_layout(int R, const vrNormShape& s) {
  BackLayout l = {};
  const int n = (s.cols + (s.dtype == VR_DT_F32 ? 4 : 8) - 1) / (s.dtype == VR_DT_F32 ? 4 : 8);
  if (s.cols < (s.dtype == VR_DT_F32 ? 4 : 8)) l.tpr = 0;
  else if (n <= 64) l.tpr = 64, l.pieces = 1;
  else if (n <= 128) l.tpr = 64, l.pieces = 2;
  // A wave with 4 pieces a lane meets at no barrier, but has a quarter of the waves: 8 ranks' rows of 2048 bf16 32.2 and
  // 32.6 us at 8192 rows in all, 44 and 44 at 12288, 58 and 54 at 16384, 107 and 95 at 32768 (rows of 2047: 135 and 103; one
  // rank's 30000: 84 and 85).
  else if (n <= 256 && (int64_t)R * s.rows >= 16384) l.tpr = 64, l.pieces = 4;
  else if (n <= 256) l.tpr = 256, l.pieces = 1;
  else if (n <= 512) l.tpr = 256, l.pieces = 2;
  else if (n <= 1024) l.tpr = 1024, l.pieces = 1;
  else if (n <= 2048) l.tpr = 1024, l.pieces = 2;
  const int at_once = l.tpr == 64 ? 4 : 1, most = std::max(1, (l.tpr == 1024 ? 512 : 1024) / R);
  l.slots = std::max(1, std::min(most, (s.rows + at_once - 1) / at_once));
  l.roots = align256((size_t)R * l.slots * s.cols * sizeof(float));
  l.total = l.roots + (l.tpr ? 0 : align256((size_t)R * s.rows * 2 * sizeof(float)));
  return l;
}

template <int DT, int TPR, int P>
void start_back(const BackArgs& a, int R, hipStream_t st) {
  const dim3 grid(a.slots, R);
  const int64_t bytes = (int64_t)R * a.rows * a.cols * Elem<DT>::kSize * (2 + (a.dsum.p[0] != nullptr) + (a.dh.p[0] != nullptr));
  if (a.cols % Elem<DT>::kChunk) hipLaunchKernelGGL((k_norm_back<DT, TPR, P, kAny>), grid, dim3(threads_of(TPR)), 0, st, a);
  else if (bytes > kCacheBytes) hipLaunchKernelGGL((k_norm_back<DT, TPR, P, kStream>), grid, dim3(threads_of(TPR)), 0, st, a);
  else hipLaunchKernelGGL((k_norm_back<DT, TPR, P, kWhole>), grid, dim3(threads_of(TPR)), 0, st, a);
}
template <int DT>
vrResult_t norm_backward(const BackArgs& a, const BackLayout& l, int R, hipStream_t st) {
  if (a.rows && l.tpr) {
    if (l.tpr == 64 && l.pieces == 1) start_back<DT, 64, 1>(a, R, st);
    else if (l.tpr == 64 && l.pieces == 2) start_back<DT, 64, 2>(a, R, st);
    else if (l.tpr == 64) start_back<DT, 64, 4>(a, R, st);
    else if (l.tpr == 256 && l.pieces == 1) start_back<DT, 256, 1>(a, R, st);
    else if (l.tpr == 256) start_back<DT, 256, 2>(a, R, st);
    else if (l.pieces == 1) start_back<DT, 1024, 1>(a, R, st);
    else start_back<DT, 1024, 2>(a, R, st);
  } else if (a.rows) {
    hipLaunchKernelGGL((k_norm_back_long<DT>), dim3(row_grid(a.rows), R), dim3(kLongThreads), 0, st, a);
    if (a.partial) hipLaunchKernelGGL((k_dgain_long<DT>), dim3(l.slots, (a.cols + 255) / 256, R), dim3(256), 0, st, a);
  }
  if (a.partial) {
    BackArgs d = a;
    if (!a.rows) d.slots = 0;  // no sums were written: zeros
    hipLaunchKernelGGL((k_dgain<DT>), dim3((a.cols + 31) / 32, R), dim3(1024), 0, st, d);
  }
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

}  // namespace

vrResult_t launch_norm(vrComm* c, const vrNormShape& s, const vrSlice& x, const vrSlice& residual, const vrSlice& gain,
                       const vrSlice& sum, const vrSlice& out, const vrSlice& q8, hipStream_t st) {
  RowArgs a = {};
  a.x = slice_tab(x);
  a.residual = slice_tab(residual);
  a.gain = slice_tab(gain);
  a.sum = slice_tab(sum);
  a.out = slice_tab(out);
  a.q8 = slice_tab(q8);
  a.err = c->err;
  a.rows = s.rows;
  a.cols = s.cols;
  a.eps = s.eps;
  a.row8 = q8_row_bytes(s.cols);
  return s.dtype == VR_DT_F32 ? start<VR_DT_F32, true>(a, c->nranks, st) : start<VR_DT_BF16, true>(a, c->nranks, st);
}

vrResult_t launch_quantize(vrComm* c, const vrSlice& x, int dtype, int rows, int cols, int groups,
                           const int32_t* group_rows, const vrSlice& q8, hipStream_t st) {
  RowArgs a = {};
  a.x = slice_tab(x);
  a.q8 = slice_tab(q8);
  a.counts = group_rows;
  a.err = c->err;
  a.G = groups;
  a.rows = rows;
  a.cols = cols;
  a.row8 = q8_row_bytes(cols);
  return dtype == VR_DT_F32 ? start<VR_DT_F32, false>(a, c->nranks, st) : start<VR_DT_BF16, false>(a, c->nranks, st);
}

vrResult_t launch_dequantize(vrComm* c, const vrSlice& q8, int dtype, int rows, int cols, int groups,
                             const int32_t* group_rows, const vrSlice& x, hipStream_t st) {
  RowArgs a = {};
  a.q8 = slice_tab(q8);
  a.out = slice_tab(x);
  a.counts = group_rows;
  a.err = c->err;
  a.G = groups;
  a.rows = rows;
  a.cols = cols;
  a.row8 = q8_row_bytes(cols);
  int log = 3;
  while (log < 8 && (8 << log) < cols) ++log;
  const int at_once = 256 >> log;
  // With counts to add up first, 4096 workgroups take several rows each (4 x 8192 rows of 512: 10.6 to 9.7 us, 2 x 8000 of
  // 2048: 17.8 to 15.6); without, short-lived ones are faster (8 x 4096 rows of 2048: 30 and 32 us).
  const uint32_t blocks = row_grid((rows + at_once - 1) / at_once);
  const dim3 grid(group_rows ? std::min(blocks, 4096u / c->nranks) : blocks, c->nranks);
  if (dtype == VR_DT_F32) hipLaunchKernelGGL((k_from_8<VR_DT_F32>), grid, dim3(256), 0, st, a, log);
  else hipLaunchKernelGGL((k_from_8<VR_DT_BF16>), grid, dim3(256), 0, st, a, log);
  return hipGetLastError() == hipSuccess ? VR_OK : VR_ERR_HIP;
}

size_t norm_backward_workspace_bytes(int R, const vrNormShape& s) { return back_layout(R, s).total; }

vrResult_t launch_norm_backward(vrComm* c, const vrNormShape& s, const vrSlice& dout, const vrSlice& h,
                                const vrSlice& gain, const vrSlice& dsum, const vrSlice& dh, const vrSlice& dgain,
                                char* ws, hipStream_t st) {
  const BackLayout l = back_layout(c->nranks, s);
  BackArgs a = {};
  a.dout = slice_tab(dout);
  a.h = slice_tab(h);
  a.gain = slice_tab(gain);
  a.dsum = slice_tab(dsum);
  a.dh = slice_tab(dh);
  a.dgain = slice_tab(dgain);
  a.partial = dgain.window ? reinterpret_cast<float*>(ws) : nullptr;
  a.roots = !l.tpr && dgain.window ? reinterpret_cast<float*>(ws + l.roots) : nullptr;
  a.rows = s.rows;
  a.cols = s.cols;
  a.slots = l.slots;
  a.eps = s.eps;
  return s.dtype == VR_DT_F32 ? norm_backward<VR_DT_F32>(a, l, c->nranks, st)
                              : norm_backward<VR_DT_BF16>(a, l, c->nranks, st);
}

}  // namespace vr
