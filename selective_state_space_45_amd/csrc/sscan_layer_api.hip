// C entry points of what stands around the recurrence in a layer: argument checks and
// launches.  The operations are defined in include/selscan.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "selscan.h"
#include "sscan_checks.h"
#include "sscan_layer.h"

namespace {

using namespace sscan;

size_t size_of(int dtype) { return dtype == SSCAN_BF16 ? 2 : 4; }
int64_t stride_or(int64_t stride, int64_t dense) { return stride == 0 ? dense : stride; }

// Outputs share bytes with nothing else of the call.
template <size_t NO, size_t NI>
int check_apart(const Buf (&outs)[NO], const Buf (&ins)[NI]) {
  for (const Buf& o : outs) {
    for (const Buf& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return fail(SSCAN_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (const Buf& q : outs)
      if (&q < &o && overlaps(o.p, o.n, q.p, q.n)) return fail(SSCAN_ERR_INVALID_ARG, "two outputs overlap");
  }
  return SSCAN_OK;
}

// The bytes of an input that outputs keep apart from.  A dense output with elements of `size` bytes
// may be `stream`, in which case an input that is the same tensor, element for element, is not counted:
// each element is read before it is written, by the same lane.  (Other outputs keep apart from it as
// they do from the output.)
Buf apart_from(const Tok& in, int64_t rows, int64_t dim, size_t es, const void* out, const void* stream, size_t size) {
  if (out && out == stream && in.p == out && (rows == 1 || in.stride == dim) && es == size) return {nullptr, 0};
  return extent(in, rows, dim, es);
}

// Sizes of an operator on rows.  Workgroups are counted in 31 bits, at least one a row.
int check_rows(int64_t rows, int64_t dim, int dtype) {
  if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return fail(SSCAN_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
  if (rows < 0 || dim < 0)
    return fail(SSCAN_ERR_INVALID_ARG, "negative size (rows %lld, dim %lld)", (long long)rows, (long long)dim);
  if (dim > SSCAN_RMS_MAX_DIM)
    return fail(SSCAN_ERR_INVALID_ARG, "dim %lld above SSCAN_RMS_MAX_DIM (%d)", (long long)dim, SSCAN_RMS_MAX_DIM);
  if (rows > INT32_MAX) return fail(SSCAN_ERR_INVALID_ARG, "rows %lld too large", (long long)rows);
  return SSCAN_OK;
}

int check_residual_dtype(int dtype, int residual_dtype) {
  if (residual_dtype != SSCAN_F32 && residual_dtype != dtype)
    return fail(SSCAN_ERR_UNSUPPORTED, "residual_dtype %d is neither SSCAN_F32 nor dtype", residual_dtype);
  return SSCAN_OK;
}

int check_eps(float eps) {
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(SSCAN_ERR_INVALID_ARG, "eps must be finite and at least 0");
  return SSCAN_OK;
}

int rms_fwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* x, int64_t x_stride,
            const void* residual, const float* weight, float eps, void* y, void* residual_out, int8_t* codes,
            int64_t codes_stride, float* scales, void* stream) {
  SSCAN_TRY(check_rows(rows, dim, dtype));
  SSCAN_TRY(check_residual_dtype(dtype, residual_dtype));
  SSCAN_TRY(check_eps(eps));
  if (rows == 0 || dim == 0) return ok();
  if (!x || (!y && !residual_out && !codes))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x and an output are required)");
  if ((codes != nullptr) != (scales != nullptr))
    return fail(SSCAN_ERR_INVALID_ARG, "codes must be given exactly when scales are");
  const size_t es = size_of(dtype), er = size_of(residual_dtype);
  const Tok tx{"x", x, stride_or(x_stride, dim)}, tr{"residual", residual, dim}, ty{"y", y, dim},
      tk{"residual_out", residual_out, dim}, tc{"codes", codes, stride_or(codes_stride, dim)};
  SSCAN_TRY(check_tok(tx, rows, dim, es));
  SSCAN_TRY(check_tok(tr, rows, dim, er));
  SSCAN_TRY(check_tok(ty, rows, dim, es));
  SSCAN_TRY(check_tok(tk, rows, dim, er));
  SSCAN_TRY(check_tok(tc, rows, dim, 1));
  SSCAN_TRY(check_f32("weight", weight));
  SSCAN_TRY(check_f32("scales", scales));
  const Buf outs[] = {extent(ty, rows, dim, es), extent(tk, rows, dim, er), extent(tc, rows, dim, 1),
                      {scales, static_cast<size_t>(rows) * 4}};
  const auto apart = [&](const Tok& t, size_t e) { return apart_from(t, rows, dim, e, residual_out, residual, er); };
  const Buf ins[] = {apart(tx, es), apart(tr, er), {weight, static_cast<size_t>(dim) * 4}};
  SSCAN_TRY(check_apart(outs, ins));
  RmsFwdParams p{};
  p.x = x; p.sx = tx.stride; p.residual = residual; p.weight = weight; p.eps = eps;
  p.y = y; p.kept = residual_out; p.codes = codes; p.sc = tc.stride; p.scales = scales;
  p.rows = rows; p.dim = static_cast<int>(dim);
  const hipError_t e = launch_rms_fwd(p, dtype == SSCAN_BF16, residual_dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "norm launch");
}

int rms_bwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* s, int64_t s_stride,
            const float* weight, float eps, const void* dy, const void* dresidual_out, void* dx, int64_t dx_stride,
            void* dresidual, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  SSCAN_TRY(check_rows(rows, dim, dtype));
  SSCAN_TRY(check_residual_dtype(dtype, residual_dtype));
  SSCAN_TRY(check_eps(eps));
  if (dim == 0 || (rows == 0 && !dweight)) return ok();
  if (!dx && !dresidual && !dweight)
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (one of dx, dresidual and dweight is required)");
  if (rows > 0 && (!s || !dy)) return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (s and dy are required)");
  const size_t es = size_of(dtype), er = size_of(residual_dtype);
  const Tok ts{"s", s, stride_or(s_stride, dim)}, tdy{"dy", dy, dim}, tdk{"dresidual_out", dresidual_out, dim},
      tdx{"dx", dx, stride_or(dx_stride, dim)}, tdr{"dresidual", dresidual, dim};
  SSCAN_TRY(check_tok(ts, rows, dim, er));
  SSCAN_TRY(check_tok(tdy, rows, dim, es));
  SSCAN_TRY(check_tok(tdk, rows, dim, er));
  SSCAN_TRY(check_tok(tdx, rows, dim, es));
  SSCAN_TRY(check_tok(tdr, rows, dim, er));
  SSCAN_TRY(check_f32("weight", weight));
  SSCAN_TRY(check_f32("dweight", dweight));
  const size_t need = dweight ? rms_bwd_workspace_bytes(rows, dim) : 0;
  SSCAN_TRY(check_buffer("workspace", workspace, workspace_bytes, need, 256));
  const size_t par = static_cast<size_t>(dim) * 4;
  const Buf outs[] = {extent(tdx, rows, dim, es), extent(tdr, rows, dim, er), {dweight, par}, {workspace, need}};
  const auto apart = [&](const Tok& t, size_t e) { return apart_from(t, rows, dim, e, dresidual, dresidual_out, er); };
  const Buf ins[] = {apart(ts, er), apart(tdy, es), apart(tdk, er), {weight, par}};
  SSCAN_TRY(check_apart(outs, ins));
  RmsBwdParams p{};
  p.s = s; p.ss = ts.stride; p.weight = weight; p.eps = eps; p.dy = dy; p.dkept = dresidual_out;
  p.dx = dx; p.sdx = tdx.stride; p.dresidual = dresidual; p.dweight = dweight;
  p.partial = static_cast<float*>(workspace); p.rows = rows; p.dim = static_cast<int>(dim);
  const hipError_t e = launch_rms_bwd(p, dtype == SSCAN_BF16, residual_dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "norm backward launch");
}

int i8_quant(int64_t rows, int64_t dim, int dtype, const void* x, int64_t x_stride, int8_t* codes, int64_t codes_stride,
             float* scales, void* stream) {
  SSCAN_TRY(check_rows(rows, dim, dtype));
  if (rows == 0) return ok();
  if (!scales || (dim > 0 && (!x || !codes)))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x, codes and scales are required)");
  const size_t es = size_of(dtype);
  const Tok tx{"x", x, stride_or(x_stride, dim)}, tc{"codes", codes, stride_or(codes_stride, dim)};
  SSCAN_TRY(check_tok(tx, rows, dim, es));
  SSCAN_TRY(check_tok(tc, rows, dim, 1));
  SSCAN_TRY(check_f32("scales", scales));
  const Buf outs[] = {extent(tc, rows, dim, 1), {scales, static_cast<size_t>(rows) * 4}};
  const Buf ins[] = {extent(tx, rows, dim, es)};
  SSCAN_TRY(check_apart(outs, ins));
  RmsFwdParams p{};
  p.x = x; p.sx = tx.stride; p.codes = codes; p.sc = tc.stride; p.scales = scales;
  p.rows = rows; p.dim = static_cast<int>(dim);
  const hipError_t e = launch_i8_quant(p, dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "8-bit rows launch");
}

int check_mnk(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0)
    return fail(SSCAN_ERR_INVALID_ARG, "negative size (m %lld, n %lld, k %lld)", (long long)m, (long long)n, (long long)k);
  if (k > SSCAN_I8_MAX_K)
    return fail(SSCAN_ERR_INVALID_ARG, "k %lld above SSCAN_I8_MAX_K (%d)", (long long)k, SSCAN_I8_MAX_K);
  if (m > INT32_MAX || n > INT32_MAX) return fail(SSCAN_ERR_INVALID_ARG, "m or n too large");
  // output tiles of 16 x 16 are counted in 32 bits
  if (!fits(m, n, 1) || ((m + 15) / 16) * ((n + 15) / 16) > INT32_MAX) return fail(SSCAN_ERR_INVALID_ARG, "m*n too large");
  return SSCAN_OK;
}

int i8_matmul(int64_t m, int64_t n, int64_t k, const int8_t* a, int64_t a_stride, const float* a_scales,
              const int8_t* b, int64_t b_stride, const float* b_scales, const float* bias, int dtype, void* out,
              int64_t out_stride, void* stream) {
  if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return fail(SSCAN_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
  SSCAN_TRY(check_mnk(m, n, k));
  if (m == 0 || n == 0) return ok();
  if (!a_scales || !b_scales || !out || (k > 0 && (!a || !b)))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (a, a_scales, b, b_scales and out are required)");
  const size_t es = size_of(dtype);
  const Tok ta{"a", a, stride_or(a_stride, k)}, tb{"b", b, stride_or(b_stride, k)}, to{"out", out, stride_or(out_stride, n)};
  SSCAN_TRY(check_tok(ta, m, k, 1));
  SSCAN_TRY(check_tok(tb, n, k, 1));
  SSCAN_TRY(check_tok(to, m, n, es));
  SSCAN_TRY(check_f32("a_scales", a_scales));
  SSCAN_TRY(check_f32("b_scales", b_scales));
  SSCAN_TRY(check_f32("bias", bias));
  const size_t cols = static_cast<size_t>(n) * 4;
  const Buf outs[] = {extent(to, m, n, es)};
  const Buf ins[] = {extent(ta, m, k, 1), extent(tb, n, k, 1), {a_scales, static_cast<size_t>(m) * 4}, {b_scales, cols},
                     {bias, cols}};
  SSCAN_TRY(check_apart(outs, ins));
  MatmulParams p{};
  p.a = a; p.b = b; p.sa = ta.stride; p.sb = tb.stride; p.as = a_scales; p.bs = b_scales; p.bias = bias;
  p.out = out; p.so = to.stride;
  p.m = static_cast<int>(m); p.n = static_cast<int>(n); p.k = static_cast<int>(k);
  const hipError_t e = launch_i8_matmul(p, dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "8-bit product launch");
}

int check_conv(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype) {
  SSCAN_TRY(check_sizes(batch, seqlen, dim, dtype));
  SSCAN_TRY(check_tiles(batch, seqlen, dim));
  if (dconv < 1 || dconv > SSCAN_MAX_DCONV)
    return fail(SSCAN_ERR_UNSUPPORTED, "dconv %lld outside [1, %d]", (long long)dconv, SSCAN_MAX_DCONV);
  return SSCAN_OK;
}

// Sequences and channels: one lane each of the kernels that write states.
int check_sequences(int64_t nseq, int64_t dim) {
  if (!fits(nseq, dim, SSCAN_MAX_DCONV)) return fail(SSCAN_ERR_INVALID_ARG, "num_seqs*dim too large");
  return check_lanes(nseq * dim);
}

int dwconv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu, const void* x,
               int64_t x_stride, const float* conv_w, const float* conv_b, const float* initial_state,
               const int32_t* offsets, int64_t num_seqs, void* y, float* last_state, void* stream) {
  SSCAN_TRY(check_conv(batch, seqlen, dim, dconv, dtype));
  SSCAN_TRY(check_offsets(batch, offsets, num_seqs));
  if (batch == 0 || dim == 0) return ok();
  const int64_t rows = batch * seqlen, nseq = offsets ? num_seqs : batch;
  SSCAN_TRY(check_sequences(nseq, dim));
  const size_t es = size_of(dtype);
  if (!conv_w || (rows > 0 && (!x || !y)))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x, conv_w and y are required)");
  const Tok tx{"x", x, stride_or(x_stride, dim)}, ty{"y", y, dim};
  SSCAN_TRY(check_tok(tx, rows, dim, es));
  SSCAN_TRY(check_tok(ty, rows, dim, es));
  SSCAN_TRY(check_f32("conv_w", conv_w));
  SSCAN_TRY(check_f32("conv_b", conv_b));
  SSCAN_TRY(check_f32("initial_state", initial_state));
  SSCAN_TRY(check_f32("last_state", last_state));
  const size_t par = static_cast<size_t>(dim) * 4, st = static_cast<size_t>(nseq) * (dconv - 1) * par;
  const Buf outs[] = {extent(ty, rows, dim, es), {last_state, st}};
  const Buf ins[] = {extent(tx, rows, dim, es), {conv_w, par * dconv}, {conv_b, par}, {initial_state, st},
                     {offsets, offsets ? static_cast<size_t>(num_seqs + 1) * 4 : 0}};
  SSCAN_TRY(check_apart(outs, ins));
  ConvParams p{};
  p.x = x; p.sx = tx.stride; p.w = conv_w; p.b = conv_b; p.h0 = initial_state; p.offsets = offsets;
  p.y = y; p.h_last = dconv > 1 ? last_state : nullptr;
  p.batch = batch; p.L = seqlen; p.dim = dim; p.num_seqs = nseq; p.silu = silu != 0;
  const hipError_t e = launch_dwconv_fwd(p, static_cast<int>(dconv), dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "convolution launch");
}

int dwconv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu, const void* x,
               int64_t x_stride, const float* conv_w, const float* conv_b, const float* initial_state,
               const int32_t* offsets, int64_t num_seqs, const void* dy, const float* dlast_state, void* dx,
               int64_t dx_stride, float* dconv_w, float* dconv_b, float* dinitial_state, void* workspace,
               size_t workspace_bytes, void* stream) {
  SSCAN_TRY(check_conv(batch, seqlen, dim, dconv, dtype));
  SSCAN_TRY(check_offsets(batch, offsets, num_seqs));
  if (dim == 0) return ok();
  const int64_t rows = batch * seqlen, nseq = offsets ? num_seqs : batch;
  SSCAN_TRY(check_sequences(nseq, dim));
  const size_t es = size_of(dtype);
  if (!conv_w || !dconv_w || (rows > 0 && (!x || !dy || !dx)))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x, conv_w, dy, dx and dconv_w are required)");
  const Tok tx{"x", x, stride_or(x_stride, dim)}, tdy{"dy", dy, dim}, tdx{"dx", dx, stride_or(dx_stride, dim)};
  SSCAN_TRY(check_tok(tx, rows, dim, es));
  SSCAN_TRY(check_tok(tdy, rows, dim, es));
  SSCAN_TRY(check_tok(tdx, rows, dim, es));
  SSCAN_TRY(check_f32("conv_w", conv_w));
  SSCAN_TRY(check_f32("conv_b", conv_b));
  SSCAN_TRY(check_f32("initial_state", initial_state));
  SSCAN_TRY(check_f32("dlast_state", dlast_state));
  SSCAN_TRY(check_f32("dconv_w", dconv_w));
  SSCAN_TRY(check_f32("dconv_b", dconv_b));
  SSCAN_TRY(check_f32("dinitial_state", dinitial_state));
  const size_t need = dwconv_bwd_workspace_bytes(batch, seqlen, dim, static_cast<int>(dconv));
  SSCAN_TRY(check_buffer("workspace", workspace, workspace_bytes, need, 256));
  const size_t par = static_cast<size_t>(dim) * 4, st = static_cast<size_t>(nseq) * (dconv - 1) * par;
  const Buf outs[] = {extent(tdx, rows, dim, es), {dconv_w, par * dconv}, {dconv_b, par}, {dinitial_state, st},
                      {workspace, need}};
  const Buf ins[] = {extent(tx, rows, dim, es), extent(tdy, rows, dim, es), {conv_w, par * dconv}, {conv_b, par},
                     {initial_state, st}, {dlast_state, st}, {offsets, offsets ? static_cast<size_t>(num_seqs + 1) * 4 : 0}};
  SSCAN_TRY(check_apart(outs, ins));
  ConvParams p{};
  p.x = x; p.sx = tx.stride; p.w = conv_w; p.b = conv_b; p.h0 = initial_state; p.offsets = offsets;
  p.dy = dy; p.dlast = dconv > 1 ? dlast_state : nullptr; p.dx = dx; p.sdx = tdx.stride;
  p.dw = dconv_w; p.db = dconv_b; p.dh0 = dconv > 1 ? dinitial_state : nullptr; p.partial = static_cast<float*>(workspace);
  p.batch = batch; p.L = seqlen; p.dim = dim; p.num_seqs = nseq; p.silu = silu != 0;
  const hipError_t e = launch_dwconv_bwd(p, static_cast<int>(dconv), dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "convolution backward launch");
}

int dwconv_step(int64_t batch, int64_t dim, int64_t dconv, int dtype, int silu, float* state, int64_t num_slots,
                const int32_t* slots, const int32_t* slots_out, const void* x, int64_t x_stride, const float* conv_w,
                const float* conv_b, void* y, void* stream) {
  SSCAN_TRY(check_conv(batch, 1, dim, dconv, dtype));
  if (num_slots < 0 || !fits(num_slots, dim, SSCAN_MAX_DCONV))
    return fail(SSCAN_ERR_INVALID_ARG, "num_slots %lld negative or too large", (long long)num_slots);
  if (!slots && batch > num_slots)
    return fail(SSCAN_ERR_INVALID_ARG, "batch %lld above num_slots %lld without slots", (long long)batch,
                (long long)num_slots);
  if (batch == 0 || dim == 0) return ok();
  if ((num_slots > 0 && dconv > 1 && !state) || !x || !conv_w || !y)
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (state, x, conv_w and y are required)");
  const size_t es = size_of(dtype);
  const Tok tx{"x", x, stride_or(x_stride, dim)}, ty{"y", y, dim};
  SSCAN_TRY(check_tok(tx, batch, dim, es));
  SSCAN_TRY(check_tok(ty, batch, dim, es));
  SSCAN_TRY(check_f32("state", state));
  SSCAN_TRY(check_f32("slots", slots));
  SSCAN_TRY(check_f32("slots_out", slots_out));
  SSCAN_TRY(check_f32("conv_w", conv_w));
  SSCAN_TRY(check_f32("conv_b", conv_b));
  const size_t par = static_cast<size_t>(dim) * 4, idx = static_cast<size_t>(batch) * 4;
  const Buf outs[] = {extent(ty, batch, dim, es), {state, static_cast<size_t>(num_slots) * (dconv - 1) * par}};
  const Buf ins[] = {extent(tx, batch, dim, es), {conv_w, par * dconv}, {conv_b, par}, {slots, idx}, {slots_out, idx}};
  SSCAN_TRY(check_apart(outs, ins));
  ConvStepParams p{};
  p.state = state; p.num_slots = num_slots; p.slots = slots; p.slots_out = slots_out;
  p.x = x; p.sx = tx.stride; p.w = conv_w; p.b = conv_b; p.y = y; p.batch = batch; p.dim = dim; p.silu = silu != 0;
  const hipError_t e = launch_dwconv_step(p, static_cast<int>(dconv), dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "convolution step launch");
}

}  // namespace

extern "C" {

sscan_status sscan_rms_fwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* x, int64_t x_stride,
                           const void* residual, const float* weight, float eps, void* y, void* residual_out,
                           int8_t* codes, int64_t codes_stride, float* scales, void* stream) {
  return static_cast<sscan_status>(rms_fwd(rows, dim, dtype, residual_dtype, x, x_stride, residual, weight, eps, y,
                                           residual_out, codes, codes_stride, scales, stream));
}

size_t sscan_rms_bwd_workspace_size(int64_t rows, int64_t dim) {
  if (rows < 0 || rows > INT32_MAX || dim < 0 || dim > SSCAN_RMS_MAX_DIM) return 0;
  return rms_bwd_workspace_bytes(rows, dim);
}

sscan_status sscan_rms_bwd(int64_t rows, int64_t dim, int dtype, int residual_dtype, const void* s, int64_t s_stride,
                           const float* weight, float eps, const void* dy, const void* dresidual_out, void* dx,
                           int64_t dx_stride, void* dresidual, float* dweight, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return static_cast<sscan_status>(rms_bwd(rows, dim, dtype, residual_dtype, s, s_stride, weight, eps, dy,
                                           dresidual_out, dx, dx_stride, dresidual, dweight, workspace,
                                           workspace_bytes, stream));
}

sscan_status sscan_i8_quant(int64_t rows, int64_t dim, int dtype, const void* x, int64_t x_stride, int8_t* codes,
                            int64_t codes_stride, float* scales, void* stream) {
  return static_cast<sscan_status>(i8_quant(rows, dim, dtype, x, x_stride, codes, codes_stride, scales, stream));
}

sscan_status sscan_i8_matmul(int64_t m, int64_t n, int64_t k, const int8_t* a, int64_t a_stride,
                             const float* a_scales, const int8_t* b, int64_t b_stride, const float* b_scales,
                             const float* bias, int dtype, void* out, int64_t out_stride, void* stream) {
  return static_cast<sscan_status>(i8_matmul(m, n, k, a, a_stride, a_scales, b, b_stride, b_scales, bias, dtype, out,
                                             out_stride, stream));
}

sscan_status sscan_dwconv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu,
                              const void* x, int64_t x_stride, const float* conv_w, const float* conv_b,
                              const float* initial_state, const int32_t* offsets, int64_t num_seqs, void* y,
                              float* last_state, void* stream) {
  return static_cast<sscan_status>(dwconv_fwd(batch, seqlen, dim, dconv, dtype, silu, x, x_stride, conv_w, conv_b,
                                              initial_state, offsets, num_seqs, y, last_state, stream));
}

size_t sscan_dwconv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv) {
  if (!valid_sizes(batch, seqlen, dim) || dconv < 1 || dconv > SSCAN_MAX_DCONV) return 0;
  return dwconv_bwd_workspace_bytes(batch, seqlen, dim, static_cast<int>(dconv));
}

sscan_status sscan_dwconv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t dconv, int dtype, int silu,
                              const void* x, int64_t x_stride, const float* conv_w, const float* conv_b,
                              const float* initial_state, const int32_t* offsets, int64_t num_seqs, const void* dy,
                              const float* dlast_state, void* dx, int64_t dx_stride, float* dconv_w, float* dconv_b,
                              float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
  return static_cast<sscan_status>(dwconv_bwd(batch, seqlen, dim, dconv, dtype, silu, x, x_stride, conv_w, conv_b,
                                              initial_state, offsets, num_seqs, dy, dlast_state, dx, dx_stride,
                                              dconv_w, dconv_b, dinitial_state, workspace, workspace_bytes, stream));
}

sscan_status sscan_dwconv_step(int64_t batch, int64_t dim, int64_t dconv, int dtype, int silu, float* state,
                               int64_t num_slots, const int32_t* slots, const int32_t* slots_out, const void* x,
                               int64_t x_stride, const float* conv_w, const float* conv_b, void* y, void* stream) {
  return static_cast<sscan_status>(dwconv_step(batch, dim, dconv, dtype, silu, state, num_slots, slots, slots_out, x,
                                               x_stride, conv_w, conv_b, y, stream));
}

}  // extern "C"
