// Matrix products of rows in 8 bits over windows, dense or by expert
// (vr_linear_q8): out = act(z) (gated: act(z_g) * z_u) + residual with
//   z[m][n] = (sum over k of x[m][k] w[n][k]) * scale of x's row m * scale of
//             w's row n + bias[n]
// The sums are 32-bit integers, exact; they become binary32 once, at the end. The
// tiles and the kernels for few rows are those of vr_linear, with matrix
// instructions of twice the rate and half the bytes of bf16; large calls take
// k_gemm_run. 8192 x 4096 x 4096 with gelu, bias and residual, three sets of inputs
// in turn: 151 us, 1.82 POP/s (bf16 in the same run: 257 us); 8 x 32768 rows (15/16
// used) by 32 experts, 512 -> 512 gated: 247 us, 1.05 POP/s.
#include <hip/hip_runtime.h>

#include "vr_gemm.hpp"

namespace vr {
namespace {

template <int DT>
vrResult_t linear_q8(vrComm* c, const vrLinearShape& s, const vrSlice& x, const vrSlice& w, const vrSlice& bias,
                     const vrSlice& residual, const int32_t* group_rows, const vrSlice& out, hipStream_t st) {
  const bool gated = (s.act & VR_ACT_GATED) != 0;
  GemmArgs a = {};
  a.a = slice_tab(x);
  a.b = slice_tab(w);
  a.bias = slice_tab(bias);
  a.residual = slice_tab(residual);
  a.out = slice_tab(out);
  a.counts = group_rows;
  a.err = c->err;
  a.R = c->nranks;
  a.G = s.groups;
  a.rows = s.rows;
  a.N = gated ? 2 * s.out : s.out;
  a.K = s.in;
  a.O = s.out;
  a.lda = a.ldb = q8_row_bytes(s.in);
  a.b_group = (uint64_t)a.N * a.ldb;
  vrResult_t e = VR_OK;
  with_act(s.act, [&](auto act) {
    e = gated ? launch_gemm<DT, kFwd, act(), true>(a, st) : launch_gemm<DT, kFwd, act(), false>(a, st);
  });
  return e;
}

}  // namespace

vrResult_t launch_linear_q8(vrComm* c, const vrLinearShape& s, const vrSlice& x, const vrSlice& w, const vrSlice& bias,
                            const vrSlice& residual, const int32_t* group_rows, const vrSlice& out, hipStream_t st) {
  return s.dtype == VR_DT_F32 ? linear_q8<kI8ToF32>(c, s, x, w, bias, residual, group_rows, out, st)
                              : linear_q8<kI8ToBf16>(c, s, x, w, bias, residual, group_rows, out, st);
}

}  // namespace vr
