// C entry points of the gated linear recurrence and the 8-bit activations: argument
// checks and launches.  The operations are defined in include/selscan.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "selscan.h"
#include "sscan_glr.h"
#include "sscan_host.h"

namespace {

using sscan::Buf;
using sscan::aligned;
using sscan::fail;
using sscan::hip_fail;
using sscan::ok;
using sscan::overlaps;

static_assert(sscan::kGlrBlock == SSCAN_GLR_BLOCK && sscan::kActGroup == SSCAN_ACT8_GROUP, "header constants");

// Largest batch * seqlen * stride: byte offsets stay far inside 63 bits.
constexpr int64_t kMaxElems = int64_t(1) << 48;

bool fits(int64_t a, int64_t b, int64_t c) {
  if (a <= 0 || b <= 0 || c <= 0) return true;
  return a <= kMaxElems && b <= kMaxElems / a && c <= kMaxElems / (a * b);
}

bool valid_sizes(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch >= 0 && seqlen >= 0 && dim >= 0 && seqlen <= SSCAN_MAX_SEQLEN && fits(batch, seqlen, dim) &&
         fits(batch, 1, dim);
}

int check_sizes(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
  if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return fail(SSCAN_ERR_UNSUPPORTED, "unknown dtype %d", dtype);
  if (batch < 0 || seqlen < 0 || dim < 0)
    return fail(SSCAN_ERR_INVALID_ARG, "negative size (batch %lld, seqlen %lld, dim %lld)", (long long)batch,
                (long long)seqlen, (long long)dim);
  if (seqlen > SSCAN_MAX_SEQLEN)
    return fail(SSCAN_ERR_INVALID_ARG, "seqlen %lld above SSCAN_MAX_SEQLEN (%lld)", (long long)seqlen,
                (long long)SSCAN_MAX_SEQLEN);
  if (!valid_sizes(batch, seqlen, dim)) return fail(SSCAN_ERR_INVALID_ARG, "batch*seqlen*dim too large");
  return SSCAN_OK;
}

// The recurrence's kernels count their tiles (64 tokens, at least 64 channels) in 31 bits,
// and its step its workgroups, which are fewer; grid_of gives launches of any such number.
// A channel's byte offset in a row is held in 32.
int check_tiles(int64_t batch, int64_t seqlen, int64_t dim) {
  if (dim > (1 << 28)) return fail(SSCAN_ERR_INVALID_ARG, "dim too large");
  const int64_t blocks = (seqlen + SSCAN_GLR_BLOCK - 1) / SSCAN_GLR_BLOCK, sets = (dim + 63) / 64;
  if (batch > 0 && blocks > 0 && sets > 0 && (blocks > INT32_MAX / sets || batch > INT32_MAX / (blocks * sets)))
    return fail(SSCAN_ERR_INVALID_ARG, "batch*seqlen*dim too large");
  return SSCAN_OK;
}

// One lane each for `n` items, 256 a workgroup, whose number is held in 31 bits.
int check_lanes(int64_t n) {
  return n / 256 < INT32_MAX ? int(SSCAN_OK) : fail(SSCAN_ERR_INVALID_ARG, "batch*seqlen*dim too large");
}

// A token tensor: rows of dim elements, `stride` elements apart.
struct Tok {
  const char* name;
  const void* p;
  int64_t stride;
};

// Whether two token tensors of `rows` rows share bytes.  Rows of equal stride may be
// interleaved (columns of one larger matrix): then they are apart when their columns are.
bool tok_overlap(const Tok& a, const Tok& b, int64_t rows, int64_t dim, size_t es) {
  if (!a.p || !b.p || rows == 0 || dim == 0) return false;
  const size_t width = static_cast<size_t>(dim) * es;
  const size_t na = static_cast<size_t>(rows - 1) * a.stride * es + width;
  const size_t nb = static_cast<size_t>(rows - 1) * b.stride * es + width;
  if (!overlaps(a.p, na, b.p, nb)) return false;
  if (a.stride != b.stride) return true;
  const size_t pitch = static_cast<size_t>(a.stride) * es;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t gap = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;
  return !(gap >= width && gap + width <= pitch);
}

Buf extent(const Tok& t, int64_t rows, int64_t dim, size_t es) {
  if (!t.p || rows == 0 || dim == 0) return {nullptr, 0};
  return {t.p, (static_cast<size_t>(rows - 1) * t.stride + dim) * es};
}

int check_tok(const Tok& t, int64_t rows, int64_t dim, size_t es) {
  if (!t.p) return SSCAN_OK;
  if (!aligned(t.p, es)) return fail(SSCAN_ERR_INVALID_ARG, "%s not aligned to its element size", t.name);
  if (t.stride < dim)
    return fail(SSCAN_ERR_INVALID_ARG, "token stride of %s (%lld) below dim (%lld)", t.name, (long long)t.stride,
                (long long)dim);
  if (!fits(rows, t.stride, 1)) return fail(SSCAN_ERR_INVALID_ARG, "token stride of %s too large", t.name);
  return SSCAN_OK;
}

int check_f32(const char* name, const void* p) {
  return p && !aligned(p, 4) ? fail(SSCAN_ERR_INVALID_ARG, "%s not 4-byte aligned", name) : SSCAN_OK;
}

int check_scale(float c) {
  if (!(c > 0.f) || std::isinf(c)) return fail(SSCAN_ERR_INVALID_ARG, "decay_scale must be positive and finite");
  return SSCAN_OK;
}

int check_offsets(int64_t batch, const int32_t* offsets, int64_t num_seqs) {
  if (!offsets) return SSCAN_OK;
  if (!aligned(offsets, 4)) return fail(SSCAN_ERR_INVALID_ARG, "offsets not 4-byte aligned");
  if (batch != 1) return fail(SSCAN_ERR_INVALID_ARG, "offsets need batch 1 (got %lld)", (long long)batch);
  if (num_seqs < 1 || num_seqs > SSCAN_MAX_SEQLEN)
    return fail(SSCAN_ERR_INVALID_ARG, "num_seqs %lld outside [1, %lld]", (long long)num_seqs,
                (long long)SSCAN_MAX_SEQLEN);
  return SSCAN_OK;
}

// A required scratch or saved buffer.
int check_buffer(const char* name, const void* p, size_t have, size_t need, size_t align) {
  if (need == 0) return SSCAN_OK;
  if (!p) return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (%s)", name);
  if (!aligned(p, align)) return fail(SSCAN_ERR_INVALID_ARG, "%s not %zu-byte aligned", name, align);
  if (have < need) return fail(SSCAN_ERR_INVALID_ARG, "%s too small (%zu < %zu bytes)", name, have, need);
  return SSCAN_OK;
}

// First failure of a list of checks (each is SSCAN_OK when it holds).
#define SSCAN_TRY(call)          \
  do {                           \
    const int rc_ = (call);      \
    if (rc_) return rc_;         \
  } while (0)

int64_t stride_of(const int64_t* strides, int k, int64_t dim) { return strides ? strides[k] : dim; }

int glr_fwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r, const void* i,
            const void* z, const int64_t* strides, const float* lam, const float* r_bias, const float* i_bias,
            float decay_scale, const float* initial_state, const int32_t* offsets, int64_t num_seqs, void* y,
            float* last_state, float* checkpoints, size_t checkpoint_bytes, void* saved, size_t saved_bytes,
            void* workspace, size_t workspace_bytes, void* stream) {
  SSCAN_TRY(check_sizes(batch, seqlen, dim, dtype));
  SSCAN_TRY(check_tiles(batch, seqlen, dim));
  SSCAN_TRY(check_offsets(batch, offsets, num_seqs));
  SSCAN_TRY(check_scale(decay_scale));
  if (batch == 0 || dim == 0) return ok();
  const int64_t rows = batch * seqlen;
  const int64_t nseq = offsets ? num_seqs : batch;
  if (!fits(nseq, dim, 1)) return fail(SSCAN_ERR_INVALID_ARG, "num_seqs*dim too large");
  const size_t es = dtype == SSCAN_BF16 ? 2 : 4;
  if (!lam || (rows > 0 && (!x || !r || !i || !y)))
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x, r, i, lam and y are required)");
  const Tok in[] = {{"x", x, stride_of(strides, 0, dim)}, {"r", r, stride_of(strides, 1, dim)},
                    {"i", i, stride_of(strides, 2, dim)}, {"z", z, stride_of(strides, 3, dim)}};
  const Tok out{"y", y, dim};
  for (const Tok& t : in) SSCAN_TRY(check_tok(t, rows, dim, es));
  SSCAN_TRY(check_tok(out, rows, dim, es));
  SSCAN_TRY(check_f32("lam", lam));
  SSCAN_TRY(check_f32("r_bias", r_bias));
  SSCAN_TRY(check_f32("i_bias", i_bias));
  SSCAN_TRY(check_f32("initial_state", initial_state));
  SSCAN_TRY(check_f32("last_state", last_state));
  const size_t need_ck = checkpoints ? sscan_glr_checkpoint_bytes(batch, seqlen, dim) : 0;
  const size_t need_sv = saved ? sscan_glr_saved_bytes(batch, seqlen, dim, z != nullptr) : 0;
  const size_t need_ws = sscan_glr_fwd_workspace_size(batch, seqlen, dim);
  SSCAN_TRY(check_buffer("checkpoints", checkpoints, checkpoint_bytes, need_ck, 4));
  SSCAN_TRY(check_buffer("saved", saved, saved_bytes, need_sv, 256));
  SSCAN_TRY(check_buffer("workspace", workspace, workspace_bytes, need_ws, 256));
  // outputs and scratch share bytes with nothing else of the call; the last state may
  // be the initial one, which every channel reads before it writes
  const size_t st = static_cast<size_t>(nseq) * dim * 4, par = static_cast<size_t>(dim) * 4;
  const Buf outs[] = {extent(out, rows, dim, es), {last_state, st}, {checkpoints, need_ck}, {saved, need_sv},
                      {workspace, need_ws}};
  const Buf ins[] = {extent(in[0], rows, dim, es), extent(in[1], rows, dim, es), extent(in[2], rows, dim, es),
                     extent(in[3], rows, dim, es), {lam, par}, {r_bias, par}, {i_bias, par},
                     {offsets, offsets ? static_cast<size_t>(num_seqs + 1) * 4 : 0}, {initial_state, st}};
  for (const Buf& o : outs) {
    for (const Buf& n : ins)
      if (overlaps(o.p, o.n, n.p, n.n) && !(o.p == last_state && n.p == initial_state && o.p == n.p))
        return fail(SSCAN_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (const Buf& q : outs)
      if (&q < &o && overlaps(o.p, o.n, q.p, q.n)) return fail(SSCAN_ERR_INVALID_ARG, "two outputs overlap");
  }
  sscan::GlrFwdParams p{};
  p.x = x; p.r = r; p.i = i; p.z = z;
  p.sx = in[0].stride; p.sr = in[1].stride; p.si = in[2].stride; p.sz = in[3].stride;
  p.lam = lam; p.r_bias = r_bias; p.i_bias = i_bias; p.decay_scale = decay_scale;
  p.h0 = initial_state; p.offsets = offsets; p.y = y; p.h_last = last_state; p.ckpt = checkpoints;
  p.codes = static_cast<int8_t*>(saved);
  p.saved_stride = sscan::act8_total(batch, seqlen, dim);
  p.exps_at = sscan::act8_exps_at(batch, seqlen, dim);
  p.workspace = workspace;
  p.batch = batch; p.L = seqlen; p.dim = dim; p.num_seqs = num_seqs;
  const hipError_t e = sscan::launch_glr_fwd(p, dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gated recurrence launch");
}

int glr_bwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r, const void* i,
            const void* z, const int64_t* strides, const void* saved, size_t saved_bytes, const float* lam,
            const float* r_bias, const float* i_bias, float decay_scale, const float* initial_state,
            const int32_t* offsets, int64_t num_seqs, const float* checkpoints, size_t checkpoint_bytes,
            const void* dy, const float* dlast_state, void* dx, void* dr, void* di, void* dz,
            const int64_t* grad_strides, float* dlam, float* dr_bias, float* di_bias, float* dinitial_state,
            void* workspace, size_t workspace_bytes, void* stream) {
  SSCAN_TRY(check_sizes(batch, seqlen, dim, dtype));
  SSCAN_TRY(check_tiles(batch, seqlen, dim));
  SSCAN_TRY(check_offsets(batch, offsets, num_seqs));
  SSCAN_TRY(check_scale(decay_scale));
  if (dim == 0) return ok();
  const int64_t rows = batch * seqlen;
  const int64_t nseq = offsets ? num_seqs : batch;
  if (!fits(nseq, dim, 1)) return fail(SSCAN_ERR_INVALID_ARG, "num_seqs*dim too large");
  const size_t es = dtype == SSCAN_BF16 ? 2 : 4;
  if (saved && (x || r || i || z))
    return fail(SSCAN_ERR_INVALID_ARG, "x, r, i and z must be null when the activations come from saved");
  if (!lam || !dlam || (rows > 0 && (!dy || !dx || !dr || !di || (!saved && (!x || !r || !i)))))
    return fail(SSCAN_ERR_INVALID_ARG,
                "null required pointer (lam, dy, dx, dr, di, dlam, and x, r, i or saved are required)");
  if (!saved && rows > 0 && (z != nullptr) != (dz != nullptr))
    return fail(SSCAN_ERR_INVALID_ARG, "dz must be given exactly when z is");
  const Tok in[] = {{"x", x, stride_of(strides, 0, dim)}, {"r", r, stride_of(strides, 1, dim)},
                    {"i", i, stride_of(strides, 2, dim)}, {"z", z, stride_of(strides, 3, dim)}, {"dy", dy, dim}};
  const Tok out[] = {{"dx", dx, stride_of(grad_strides, 0, dim)}, {"dr", dr, stride_of(grad_strides, 1, dim)},
                     {"di", di, stride_of(grad_strides, 2, dim)}, {"dz", dz, stride_of(grad_strides, 3, dim)}};
  for (const Tok& t : in) SSCAN_TRY(check_tok(t, rows, dim, es));
  for (const Tok& t : out) SSCAN_TRY(check_tok(t, rows, dim, es));
  SSCAN_TRY(check_f32("lam", lam));
  SSCAN_TRY(check_f32("r_bias", r_bias));
  SSCAN_TRY(check_f32("i_bias", i_bias));
  SSCAN_TRY(check_f32("initial_state", initial_state));
  SSCAN_TRY(check_f32("dlast_state", dlast_state));
  SSCAN_TRY(check_f32("dlam", dlam));
  SSCAN_TRY(check_f32("dr_bias", dr_bias));
  SSCAN_TRY(check_f32("di_bias", di_bias));
  SSCAN_TRY(check_f32("dinitial_state", dinitial_state));
  const size_t need_ck = sscan_glr_checkpoint_bytes(batch, seqlen, dim);
  const size_t need_sv = saved ? sscan_glr_saved_bytes(batch, seqlen, dim, dz != nullptr) : 0;
  const size_t need_ws = sscan_glr_bwd_workspace_size(batch, seqlen, dim);
  SSCAN_TRY(check_buffer("checkpoints", checkpoints, checkpoint_bytes, need_ck, 4));
  SSCAN_TRY(check_buffer("saved", saved, saved_bytes, need_sv, 256));
  SSCAN_TRY(check_buffer("workspace", workspace, workspace_bytes, need_ws, 256));
  const size_t st = static_cast<size_t>(nseq) * dim * 4, par = static_cast<size_t>(dim) * 4;
  const Buf ins[] = {extent(in[0], rows, dim, es), extent(in[1], rows, dim, es), extent(in[2], rows, dim, es),
                     extent(in[3], rows, dim, es), extent(in[4], rows, dim, es), {saved, need_sv}, {lam, par},
                     {r_bias, par}, {i_bias, par}, {offsets, offsets ? static_cast<size_t>(num_seqs + 1) * 4 : 0},
                     {initial_state, st}, {dlast_state, st}, {checkpoints, need_ck}};
  const Buf flat[] = {{dlam, par}, {dr_bias, par}, {di_bias, par}, {dinitial_state, st}, {workspace, need_ws}};
  for (const Tok& o : out) {
    const Buf e = extent(o, rows, dim, es);
    for (const Buf& n : ins)
      if (overlaps(e.p, e.n, n.p, n.n)) return fail(SSCAN_ERR_INVALID_ARG, "%s overlaps an input", o.name);
    for (const Buf& q : flat)
      if (overlaps(e.p, e.n, q.p, q.n)) return fail(SSCAN_ERR_INVALID_ARG, "two outputs overlap");
    for (const Tok& q : out)
      if (&q < &o && tok_overlap(o, q, rows, dim, es))
        return fail(SSCAN_ERR_INVALID_ARG, "%s overlaps %s", o.name, q.name);
  }
  for (const Buf& o : flat) {
    for (const Buf& n : ins)
      if (overlaps(o.p, o.n, n.p, n.n))
        return fail(SSCAN_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (const Buf& q : flat)
      if (&q < &o && overlaps(o.p, o.n, q.p, q.n)) return fail(SSCAN_ERR_INVALID_ARG, "two outputs overlap");
  }
  sscan::GlrBwdParams p{};
  p.x = x; p.r = r; p.i = i; p.z = z;
  p.sx = in[0].stride; p.sr = in[1].stride; p.si = in[2].stride; p.sz = in[3].stride;
  p.codes = static_cast<const int8_t*>(saved);
  p.saved_stride = sscan::act8_total(batch, seqlen, dim);
  p.exps_at = sscan::act8_exps_at(batch, seqlen, dim);
  p.lam = lam; p.r_bias = r_bias; p.i_bias = i_bias; p.decay_scale = decay_scale;
  p.h0 = initial_state; p.offsets = offsets; p.ckpt = checkpoints; p.dy = dy; p.dlast = dlast_state;
  p.dx = dx; p.dr = dr; p.di = di; p.dz = dz;
  p.gx = out[0].stride; p.gr = out[1].stride; p.gi = out[2].stride; p.gz = out[3].stride;
  p.dlam = dlam; p.dr_bias = dr_bias; p.di_bias = di_bias; p.dh0 = dinitial_state;
  p.workspace = workspace;
  p.batch = batch; p.L = seqlen; p.dim = dim; p.num_seqs = num_seqs;
  const hipError_t e = sscan::launch_glr_bwd(p, dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gated recurrence backward launch");
}

int glr_step(int64_t batch, int64_t dim, int dtype, float* state, int64_t num_slots, const int32_t* slots,
             const int32_t* slots_out, const void* x, const void* r, const void* i, const void* z,
             const int64_t* strides, const float* lam, const float* r_bias, const float* i_bias, float decay_scale,
             void* y, void* stream) {
  SSCAN_TRY(check_sizes(batch, 1, dim, dtype));
  SSCAN_TRY(check_tiles(batch, 1, dim));
  if (num_slots < 0 || !fits(num_slots, dim, 1))
    return fail(SSCAN_ERR_INVALID_ARG, "num_slots %lld negative or too large", (long long)num_slots);
  if (!slots && batch > num_slots)
    return fail(SSCAN_ERR_INVALID_ARG, "batch %lld above num_slots %lld without slots", (long long)batch,
                (long long)num_slots);
  SSCAN_TRY(check_scale(decay_scale));
  if (batch == 0 || dim == 0) return ok();
  if ((num_slots > 0 && !state) || !x || !r || !i || !lam || !y)
    return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (state, x, r, i, lam and y are required)");
  const size_t es = dtype == SSCAN_BF16 ? 2 : 4;
  const Tok in[] = {{"x", x, stride_of(strides, 0, dim)}, {"r", r, stride_of(strides, 1, dim)},
                    {"i", i, stride_of(strides, 2, dim)}, {"z", z, stride_of(strides, 3, dim)}};
  const Tok out{"y", y, dim};
  for (const Tok& t : in) SSCAN_TRY(check_tok(t, batch, dim, es));
  SSCAN_TRY(check_tok(out, batch, dim, es));
  SSCAN_TRY(check_f32("state", state));
  SSCAN_TRY(check_f32("slots", slots));
  SSCAN_TRY(check_f32("slots_out", slots_out));
  SSCAN_TRY(check_f32("lam", lam));
  SSCAN_TRY(check_f32("r_bias", r_bias));
  SSCAN_TRY(check_f32("i_bias", i_bias));
  const size_t par = static_cast<size_t>(dim) * 4, idx = static_cast<size_t>(batch) * 4;
  const Buf outs[] = {extent(out, batch, dim, es), {state, static_cast<size_t>(num_slots) * dim * 4}};
  const Buf ins[] = {extent(in[0], batch, dim, es), extent(in[1], batch, dim, es), extent(in[2], batch, dim, es),
                     extent(in[3], batch, dim, es), {lam, par}, {r_bias, par}, {i_bias, par}, {slots, idx},
                     {slots_out, idx}};
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return fail(SSCAN_ERR_INVALID_ARG, "y overlaps the state");
  for (const Buf& o : outs)
    for (const Buf& n : ins)
      if (overlaps(o.p, o.n, n.p, n.n)) return fail(SSCAN_ERR_INVALID_ARG, "y or the state overlaps an input");
  sscan::GlrStepParams p{};
  p.state = state; p.num_slots = num_slots; p.slots = slots; p.slots_out = slots_out;
  p.x = x; p.r = r; p.i = i; p.z = z;
  p.sx = in[0].stride; p.sr = in[1].stride; p.si = in[2].stride; p.sz = in[3].stride;
  p.lam = lam; p.r_bias = r_bias; p.i_bias = i_bias; p.decay_scale = decay_scale;
  p.y = y; p.batch = batch; p.dim = dim;
  const hipError_t e = sscan::launch_glr_step(p, dtype == SSCAN_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gated recurrence step launch");
}

int act8_check(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const Tok& x, const void* packed,
               size_t packed_bytes) {
  SSCAN_TRY(check_sizes(batch, seqlen, dim, dtype));
  const int64_t rows = batch * seqlen;
  if (rows == 0 || dim == 0) return SSCAN_OK;
  SSCAN_TRY(check_lanes(batch * ((seqlen + SSCAN_ACT8_GROUP - 1) / SSCAN_ACT8_GROUP) * dim));
  const size_t es = dtype == SSCAN_BF16 ? 2 : 4;
  if (!x.p) return fail(SSCAN_ERR_INVALID_ARG, "null required pointer (x)");
  SSCAN_TRY(check_tok(x, rows, dim, es));
  const size_t need = sscan_act8_bytes(batch, seqlen, dim);
  SSCAN_TRY(check_buffer("packed", packed, packed_bytes, need, 256));
  const Buf e = extent(x, rows, dim, es);
  if (overlaps(e.p, e.n, packed, need)) return fail(SSCAN_ERR_INVALID_ARG, "packed overlaps x");
  return SSCAN_OK;
}

}  // namespace

extern "C" {

size_t sscan_act8_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  if (!valid_sizes(batch, seqlen, dim) || batch == 0 || seqlen == 0 || dim == 0) return 0;
  return sscan::act8_total(batch, seqlen, dim);
}

sscan_status sscan_act8_pack(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, int64_t x_stride,
                             void* packed, size_t packed_bytes, void* stream) {
  const int64_t stride = x_stride == 0 ? dim : x_stride;
  const int rc = act8_check(batch, seqlen, dim, dtype, {"x", x, stride}, packed, packed_bytes);
  if (rc) return static_cast<sscan_status>(rc);
  if (batch == 0 || seqlen == 0 || dim == 0) return static_cast<sscan_status>(ok());
  const hipError_t e = sscan::launch_act8_pack(x, stride, packed, batch, seqlen, dim, dtype == SSCAN_BF16,
                                               static_cast<hipStream_t>(stream));
  return static_cast<sscan_status>(e == hipSuccess ? ok() : hip_fail(e, "pack launch"));
}

sscan_status sscan_act8_unpack(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* packed,
                               size_t packed_bytes, void* x, void* stream) {
  const int rc = act8_check(batch, seqlen, dim, dtype, {"x", x, dim}, packed, packed_bytes);
  if (rc) return static_cast<sscan_status>(rc);
  if (batch == 0 || seqlen == 0 || dim == 0) return static_cast<sscan_status>(ok());
  const hipError_t e = sscan::launch_act8_unpack(packed, x, batch, seqlen, dim, dtype == SSCAN_BF16,
                                                 static_cast<hipStream_t>(stream));
  return static_cast<sscan_status>(e == hipSuccess ? ok() : hip_fail(e, "unpack launch"));
}

size_t sscan_glr_checkpoint_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  if (!valid_sizes(batch, seqlen, dim)) return 0;
  return static_cast<size_t>(batch) * ((seqlen + SSCAN_GLR_BLOCK - 1) / SSCAN_GLR_BLOCK) * dim * sizeof(float);
}

size_t sscan_glr_saved_bytes(int64_t batch, int64_t seqlen, int64_t dim, int gated) {
  return (gated ? 4 : 3) * sscan_act8_bytes(batch, seqlen, dim);
}

size_t sscan_glr_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim) {
  return valid_sizes(batch, seqlen, dim) ? sscan::glr_fwd_workspace_bytes(batch, seqlen, dim) : 0;
}

size_t sscan_glr_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim) {
  return valid_sizes(batch, seqlen, dim) ? sscan::glr_bwd_workspace_bytes(batch, seqlen, dim) : 0;
}

sscan_status sscan_glr_fwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r,
                           const void* i, const void* z, const int64_t* strides, const float* lam,
                           const float* r_bias, const float* i_bias, float decay_scale, const float* initial_state,
                           const int32_t* offsets, int64_t num_seqs, void* y, float* last_state, float* checkpoints,
                           size_t checkpoint_bytes, void* saved, size_t saved_bytes, void* workspace,
                           size_t workspace_bytes, void* stream) {
  return static_cast<sscan_status>(glr_fwd(batch, seqlen, dim, dtype, x, r, i, z, strides, lam, r_bias, i_bias,
                                           decay_scale, initial_state, offsets, num_seqs, y, last_state, checkpoints,
                                           checkpoint_bytes, saved, saved_bytes, workspace, workspace_bytes, stream));
}

sscan_status sscan_glr_bwd(int64_t batch, int64_t seqlen, int64_t dim, int dtype, const void* x, const void* r,
                           const void* i, const void* z, const int64_t* strides, const void* saved,
                           size_t saved_bytes, const float* lam, const float* r_bias, const float* i_bias,
                           float decay_scale, const float* initial_state, const int32_t* offsets, int64_t num_seqs,
                           const float* checkpoints, size_t checkpoint_bytes, const void* dy,
                           const float* dlast_state, void* dx, void* dr, void* di, void* dz,
                           const int64_t* grad_strides, float* dlam, float* dr_bias, float* di_bias,
                           float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
  return static_cast<sscan_status>(
      glr_bwd(batch, seqlen, dim, dtype, x, r, i, z, strides, saved, saved_bytes, lam, r_bias, i_bias, decay_scale,
              initial_state, offsets, num_seqs, checkpoints, checkpoint_bytes, dy, dlast_state, dx, dr, di, dz,
              grad_strides, dlam, dr_bias, di_bias, dinitial_state, workspace, workspace_bytes, stream));
}

sscan_status sscan_glr_step(int64_t batch, int64_t dim, int dtype, float* state, int64_t num_slots,
                            const int32_t* slots, const int32_t* slots_out, const void* x, const void* r,
                            const void* i, const void* z, const int64_t* strides, const float* lam,
                            const float* r_bias, const float* i_bias, float decay_scale, void* y, void* stream) {
  return static_cast<sscan_status>(glr_step(batch, dim, dtype, state, num_slots, slots, slots_out, x, r, i, z, strides,
                                            lam, r_bias, i_bias, decay_scale, y, stream));
}

}  // extern "C"
