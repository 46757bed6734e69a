// Argument checks of token tensors, packed requests and buffers, shared by the entry points
// that take them.
#pragma once

#include "selscan.h"
#include "sscan_host.h"

namespace sscan {

// Largest batch * seqlen * stride: byte offsets stay far inside 63 bits.
constexpr int64_t kMaxElems = int64_t(1) << 48;

inline bool fits(int64_t a, int64_t b, int64_t c) {
  if (a <= 0 || b <= 0 || c <= 0) return true;
  return a <= kMaxElems && b <= kMaxElems / a && c <= kMaxElems / (a * b);
}

inline bool valid_sizes(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch >= 0 && seqlen >= 0 && dim >= 0 && seqlen <= SSCAN_MAX_SEQLEN && fits(batch, seqlen, dim) &&
         fits(batch, 1, dim);
}

inline int check_sizes(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
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
inline int check_tiles(int64_t batch, int64_t seqlen, int64_t dim) {
  if (dim > (1 << 28)) return fail(SSCAN_ERR_INVALID_ARG, "dim too large");
  const int64_t blocks = (seqlen + SSCAN_GLR_BLOCK - 1) / SSCAN_GLR_BLOCK, sets = (dim + 63) / 64;
  if (batch > 0 && blocks > 0 && sets > 0 && (blocks > INT32_MAX / sets || batch > INT32_MAX / (blocks * sets)))
    return fail(SSCAN_ERR_INVALID_ARG, "batch*seqlen*dim too large");
  return SSCAN_OK;
}

// One lane each for `n` items, 256 a workgroup, whose number is held in 31 bits.
inline int check_lanes(int64_t n) {
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
inline bool tok_overlap(const Tok& a, const Tok& b, int64_t rows, int64_t dim, size_t es) {
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

inline Buf extent(const Tok& t, int64_t rows, int64_t dim, size_t es) {
  if (!t.p || rows == 0 || dim == 0) return {nullptr, 0};
  return {t.p, (static_cast<size_t>(rows - 1) * t.stride + dim) * es};
}

inline int check_tok(const Tok& t, int64_t rows, int64_t dim, size_t es) {
  if (!t.p) return SSCAN_OK;
  if (!aligned(t.p, es)) return fail(SSCAN_ERR_INVALID_ARG, "%s not aligned to its element size", t.name);
  if (t.stride < dim)
    return fail(SSCAN_ERR_INVALID_ARG, "token stride of %s (%lld) below dim (%lld)", t.name, (long long)t.stride,
                (long long)dim);
  if (!fits(rows, t.stride, 1)) return fail(SSCAN_ERR_INVALID_ARG, "token stride of %s too large", t.name);
  return SSCAN_OK;
}

inline int check_f32(const char* name, const void* p) {
  return p && !aligned(p, 4) ? fail(SSCAN_ERR_INVALID_ARG, "%s not 4-byte aligned", name) : SSCAN_OK;
}

inline int check_offsets(int64_t batch, const int32_t* offsets, int64_t num_seqs) {
  if (!offsets) return SSCAN_OK;
  if (!aligned(offsets, 4)) return fail(SSCAN_ERR_INVALID_ARG, "offsets not 4-byte aligned");
  if (batch != 1) return fail(SSCAN_ERR_INVALID_ARG, "offsets need batch 1 (got %lld)", (long long)batch);
  if (num_seqs < 1 || num_seqs > SSCAN_MAX_SEQLEN)
    return fail(SSCAN_ERR_INVALID_ARG, "num_seqs %lld outside [1, %lld]", (long long)num_seqs,
                (long long)SSCAN_MAX_SEQLEN);
  return SSCAN_OK;
}

// A required scratch or saved buffer.
inline int check_buffer(const char* name, const void* p, size_t have, size_t need, size_t align) {
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

}  // namespace sscan
