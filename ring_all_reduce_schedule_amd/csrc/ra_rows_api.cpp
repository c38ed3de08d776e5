// ra_rows_api.cpp -- C entry points of the row operators declared in include/ra.h
// (norm, cross entropy, log probabilities, embedding) and of the gradients' norm and
// clipping: argument checks, then one call to the launchers in ra_norm.hip,
// ra_xent.hip, ra_logprob.hip, ra_embed.hip and ra_grads.hip.  Nothing here waits,
// allocates device memory or throws.
#include "ra.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <memory>
#include <new>

#include "ra_internal.h"

namespace {

using ra::fail;
using ra::fail_hip;

// ---------------------------------------------------------------- checks

int check_ranks(int p) {
  if (p < 1) return fail(RA_ERR_INVALID_ARG, "p = %d, need p >= 1", p);
  if (p > RA_MAX_RANKS) return fail(RA_ERR_UNSUPPORTED, "p = %d exceeds RA_MAX_RANKS = %d", p, RA_MAX_RANKS);
  return RA_OK;
}

// The types these operators compute on.
int check_real(const char* what, int dtype) {
  if (dtype == RA_FLOAT32 || dtype == RA_BFLOAT16 || dtype == RA_FLOAT16) return RA_OK;
  if (dtype < RA_INT32 || dtype > RA_FLOAT8_E4M3) return fail(RA_ERR_INVALID_ARG, "unknown %s %d", what, dtype);
  return fail(RA_ERR_UNSUPPORTED, "%s %d: these operators take float32, bfloat16 and float16", what, dtype);
}

// A second type, that has to be the first one or float32.
int check_second(const char* what, int dtype, int first) {
  int rc = check_real(what, dtype);
  if (rc == RA_OK && dtype != first && dtype != RA_FLOAT32)
    rc = fail(RA_ERR_UNSUPPORTED, "%s %d: need the buffers' type or float32", what, dtype);
  return rc;
}

int check_index(const char* what, int dtype) {
  if (dtype == RA_INT32 || dtype == RA_INT64) return RA_OK;
  return fail(RA_ERR_INVALID_ARG, "%s %d: need RA_INT32 or RA_INT64", what, dtype);
}

int check_rows(int64_t tokens, int64_t hidden, int64_t most, const char* name) {
  if (tokens < 0) return fail(RA_ERR_INVALID_ARG, "tokens = %lld, need tokens >= 0", (long long)tokens);
  if (hidden < 1) return fail(RA_ERR_INVALID_ARG, "%s = %lld, need %s >= 1", name, (long long)hidden, name);
  if (hidden > most)
    return fail(RA_ERR_UNSUPPORTED, "%s = %lld exceeds %lld", name, (long long)hidden, (long long)most);
  if (tokens > (INT64_MAX >> 4) / hidden)
    return fail(RA_ERR_INVALID_ARG, "tokens = %lld overflow the address space", (long long)tokens);
  return RA_OK;
}

int check_count(const char* what, int n, int lo, int hi) {
  if (n >= lo && n <= hi) return RA_OK;
  return fail(RA_ERR_INVALID_ARG, "%s = %d, need %d..%d", what, n, lo, hi);
}

// The bytes [lo, hi) of an array.
struct Span {
  uint64_t lo, hi;
  const char* what;
  int index;
  bool write;
};

bool before(const Span& a, const Span& b) { return a.lo < b.lo; }
// Lists mostly come in the order of their addresses, for which a look will do.
void sort_spans(Span* list, int64_t n) {
  if (!std::is_sorted(list, list + n, before)) std::sort(list, list + n, before);
}

int overlap(const Span& a, const Span& b) {
  return fail(RA_ERR_ALIAS, "%s (%d) and %s (%d) overlap", a.what, a.index, b.what, b.index);
}

// Whether no byte is written by one array and in another, of a sorted list.
int check_spans(const Span* list, int64_t n) {
  const Span *read = nullptr, *written = nullptr;   // the ones so far that end last
  for (int64_t i = 0; i < n; ++i) {
    const Span& x = list[i];
    const Span* with = written && x.lo < written->hi         ? written
                       : x.write && read && x.lo < read->hi ? read
                                                             : nullptr;
    if (with) return overlap(*with, x);
    const Span*& last = x.write ? written : read;
    if (!last || x.hi > last->hi) last = &x;
  }
  return RA_OK;
}

// The arrays of one call: each is present, starts on a boundary of its elements,
// and shares no byte with another one where either is written.  al() says whether
// all of them also start on the boundary that the aligned kernels take.
class Arrays {
 public:
  // optional: NULL is fine.  fit: bytes that aligned kernels want the start to be a multiple of.
  int add(const char* what, int index, const void* ptr, int64_t bytes, int elem, bool write, bool optional = false,
          int fit = 16) {
    if (!ptr) {
      if (optional || bytes == 0) return RA_OK;
      return index < 0 ? fail(RA_ERR_INVALID_ARG, "%s is NULL", what)
                       : fail(RA_ERR_INVALID_ARG, "%s[%d] is NULL", what, index);
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(ptr);
    if (at % elem != 0)
      return fail(RA_ERR_MISALIGNED, "%s%s = %p is not on a boundary of its %d-byte elements", what,
                  index < 0 ? "" : "[]", ptr, elem);
    if (at % fit != 0) aligned_ = false;
    if (bytes > 0) {
      if (n_ == kMost) return fail(RA_ERR_UNSUPPORTED, "more than %d arrays in a call", kMost);
      list_[n_++] = {at, at + (uint64_t)bytes, what, index, write};
    }
    return RA_OK;
  }
  // ptr may be exactly an array that was added before as read: both are then one, written.
  int add_or_same(const char* what, int index, const void* ptr, int64_t bytes, int elem) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(ptr);
    for (int i = 0; ptr && i < n_; ++i) {
      if (list_[i].lo == at && list_[i].hi == at + (uint64_t)bytes && !list_[i].write) {
        list_[i].write = true;
        return RA_OK;
      }
    }
    return add(what, index, ptr, bytes, elem, true);
  }
  int overlaps() {
    sort_spans(list_, n_);
    return check_spans(list_, n_);
  }
  bool al() const { return aligned_; }

 private:
  // Three lists of the ranks' (a norm's buffers, outputs and scales) and single arrays.
  static constexpr int kMost = 3 * RA_MAX_RANKS + 16;
  Span list_[kMost];
  int n_ = 0;
  bool aligned_ = true;
};

int add_ranks(Arrays* to, const char* what, const void* const* ptrs, int n, int64_t bytes, int elem, bool write,
              ra::RankPtrs* P, int fit = 16) {
  if (n > 0 && !ptrs) return fail(RA_ERR_INVALID_ARG, "%s is NULL", what);
  for (int r = 0; r < n; ++r) {
    int rc = to->add(what, r, ptrs[r], bytes, elem, write, false, fit);
    if (rc != RA_OK) return rc;
    P->b[r] = const_cast<void*>(ptrs[r]);
  }
  return RA_OK;
}

void debug_rows(const char* call, int p, int64_t tokens, int64_t cols, int dtype, bool al, int64_t extra) {
  if (ra::debug_on())
    std::fprintf(stderr, "[ra] %s p=%d tokens=%lld columns=%lld dtype=%d aligned=%d splits=%lld\n", call, p,
                 (long long)tokens, (long long)cols, dtype, (int)al, (long long)extra);
}

// 0, 1, 2: odd rows, aligned rows, aligned rows of a call of `bytes` that streams.
int access_of(bool al, int64_t bytes) { return !al ? 0 : bytes > ra::kStreamingBytes ? 2 : 1; }

int launched(hipError_t e) { return e == hipSuccess ? RA_OK : fail_hip(e, "kernel launch"); }

int check_workspace(Arrays* to, void* workspace, int64_t have, int64_t need) {
  if (need == 0) return RA_OK;
  if (have < need)
    return fail(RA_ERR_INVALID_ARG, "workspace of %lld bytes, need %lld", (long long)have, (long long)need);
  return to->add("workspace", -1, workspace, need, 16, true);
}

int64_t norm_bwd_bytes(int64_t tokens, int64_t hidden) {
  return (int64_t)ra::norm_bwd_blocks(tokens) * hidden * (int64_t)sizeof(float);
}

int64_t xent_bytes(int64_t tokens, int64_t vocab, int p, bool grad) {
  return ra::xent_words(tokens, ra::xent_splits(tokens, (int)vocab, p, grad)) * (int64_t)sizeof(float);
}

// The sizes that one call of the embedding's gradient takes.  The workspace call asks this
// too: beyond them its size would not be one, and pass 64 bits in the end.
int check_embed_bwd(int64_t tokens, int64_t vocab, int64_t hidden) {
  if (ra::embed_bwd_fits(tokens, (int)vocab, (int)hidden)) return RA_OK;
  return fail(RA_ERR_UNSUPPORTED, "tokens = %lld of %lld columns: too many for one call", (long long)tokens,
              (long long)hidden);
}

// Logits whose vocabulary is cut over the ranks.
int check_vocab(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype,
                const char* index, int index_dtype) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_index(index, index_dtype);
  if (rc == RA_OK) rc = check_rows(tokens, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK && (valid < 1 || valid > vocab))
    rc = fail(RA_ERR_INVALID_ARG, "valid = %lld, need 1..vocab = %lld", (long long)valid, (long long)vocab);
  if (rc == RA_OK && !logits) rc = fail(RA_ERR_INVALID_ARG, "logits is NULL");
  return rc;
}

int check_xent(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype, int target_dtype) {
  return check_vocab(logits, p, tokens, vocab, valid, dtype, "target_dtype", target_dtype);
}

// The logits and their gradients (or null), and the geometry of their rows.
int add_vocab(Arrays* to, ra::VocabArgs* a, void* const* logits, void* const* grads, int p, int64_t tokens,
              int64_t vocab, int64_t valid, int dtype) {
  const int e = ra::elem_bytes(dtype);
  a->p = p;
  a->tokens = tokens;
  a->cut = {(int32_t)(vocab / p), (int32_t)(vocab % p)};
  a->vocab = (int32_t)vocab;
  a->valid = (int32_t)valid;
  ra::vocab_geometry(a);
  int rc = RA_OK;
  for (int r = 0; r < p && rc == RA_OK; ++r) {
    const int64_t bytes = a->tokens * (a->cut.base + (r < a->cut.extra)) * e;
    rc = to->add("logits", r, logits[r], bytes, e, false);
    a->x.b[r] = logits[r];
  }
  for (int r = 0; grads && r < p && rc == RA_OK; ++r) {
    const int64_t bytes = a->tokens * (a->cut.base + (r < a->cut.extra)) * e;
    // in place: each piece's gradient over its own logits, and over no other's
    if (grads[r] == logits[r]) rc = to->add_or_same("grads", r, grads[r], bytes, e);
    else rc = to->add("grads", r, grads[r], bytes, e, true);
    a->dx.b[r] = grads[r];
  }
  return rc;
}

int add_xent(Arrays* to, ra::XentArgs* a, void* const* logits, void* const* grads, int p, int64_t tokens,
             int64_t vocab, int64_t valid, int dtype, const void* targets, int target_dtype, const float* dloss,
             float grad_scale) {
  a->target = targets;
  a->target64 = target_dtype == RA_INT64;
  a->dloss = dloss;
  a->grad_scale = grad_scale;
  int rc = add_vocab(to, a, logits, grads, p, tokens, vocab, valid, dtype);
  const int te = ra::elem_bytes(target_dtype);
  if (rc == RA_OK) rc = to->add("targets", -1, targets, a->tokens * te, te, false, false, 1);
  if (rc == RA_OK) rc = to->add("dloss", -1, dloss, a->tokens * 4, 4, false, true, 1);
  return rc;
}

int check_positive(const char* what, float x) {
  if (x > 0.0f && std::isfinite(x)) return RA_OK;
  return fail(RA_ERR_INVALID_ARG, "%s must be finite and > 0", what);
}

int check_top(int64_t valid, int top) {
  if (top < 0) return fail(RA_ERR_INVALID_ARG, "top = %d, need top >= 0", top);
  if (top > ra::kTopMost) return fail(RA_ERR_UNSUPPORTED, "top = %d exceeds %d", top, ra::kTopMost);
  if (top > valid) return fail(RA_ERR_INVALID_ARG, "top = %d of %lld valid columns", top, (long long)valid);
  return RA_OK;
}

int64_t logprob_bytes(int64_t tokens, int64_t vocab, int p, int top) {
  return ra::logp_bytes(tokens, ra::logp_splits(tokens, (int)vocab, p), top);
}

// A norm has to be positive; infinity is one that nothing reaches.
int check_clip(float max_norm, float scale) {
  if (!(max_norm > 0.0f)) return fail(RA_ERR_INVALID_ARG, "max_norm must be > 0");
  return check_positive("scale", scale);
}

// Tensors of one call, and elements of them all: workgroups and their parts are counted in 32 bits.
constexpr int64_t kListMost = 1 << 20, kListElements = 1ll << 40;

int check_elements(int64_t n) {
  if (n < 0) return fail(RA_ERR_INVALID_ARG, "n = %lld, need n >= 0", (long long)n);
  if (n > kListElements) return fail(RA_ERR_UNSUPPORTED, "n = %lld, at most 2^40 elements", (long long)n);
  return RA_OK;
}

int check_list_length(int64_t n) {
  if (n < 0) return fail(RA_ERR_INVALID_ARG, "n = %lld, need n >= 0", (long long)n);
  if (n > kListMost)
    return fail(RA_ERR_UNSUPPORTED, "n = %lld tensors, at most %lld in a call", (long long)n, (long long)kListMost);
  return RA_OK;
}

// A list of tensors of any sizes, read, and (outs) what is written for each: the tensor itself or
// another array.  Neither may share memory with another one that is written.
int check_list(ra::TensorListArgs& a, float* norm, void* workspace, int64_t have) {
  int rc = RA_OK;
  if (a.n > 0 && (!a.in || !a.counts || !a.types)) return fail(RA_ERR_INVALID_ARG, "tensors, counts or dtypes is NULL");
  const int64_t need = ra::grad_norm_bytes(a.n);
  if (have < need)
    return fail(RA_ERR_INVALID_ARG, "workspace of %lld bytes, need %lld", (long long)have, (long long)need);
  // host memory, for the call alone: the tensors, the outputs, and the two lists in one
  std::unique_ptr<Span[]> room(new (std::nothrow) Span[4 * a.n + 1]);
  if (!room) return fail(RA_ERR_UNSUPPORTED, "no host memory for %lld tensors", (long long)a.n);
  Span *read = room.get(), *written = read + a.n, *all = written + a.n;
  int64_t reads = 0, writes = 0, elements = 0, bytes = 0;
  auto make = [](Span* to, const char* what, int64_t i, const void* ptr, int64_t bytes, int elem, bool write) {
    if (!ptr) return fail(RA_ERR_INVALID_ARG, "%s[%lld] is NULL", what, (long long)i);
    const uintptr_t at = reinterpret_cast<uintptr_t>(ptr);
    if (at % elem != 0)
      return fail(RA_ERR_MISALIGNED, "%s[%lld] = %p is not on a boundary of its %d-byte elements", what, (long long)i,
                  ptr, elem);
    *to = {at, at + (uint64_t)bytes, what, (int)i, write};
    return (int)RA_OK;
  };
  Span own[2];      // these overlap nothing
  rc = make(&own[0], "norm", 0, norm, 4, 4, true);
  if (rc == RA_OK) rc = make(&own[1], "workspace", 0, workspace, need, 16, true);
  if (rc == RA_OK && own[0].lo < own[1].hi && own[1].lo < own[0].hi) rc = overlap(own[0], own[1]);
  for (int64_t i = 0; i < a.n && rc == RA_OK; ++i) {
    const int64_t count = a.counts[i];
    if (count < 0) return fail(RA_ERR_INVALID_ARG, "counts[%lld] = %lld", (long long)i, (long long)count);
    if (count > kListElements || (elements += count) > kListElements)
      return fail(RA_ERR_UNSUPPORTED, "more than 2^40 elements in a call");
    rc = check_real("dtype", a.types[i]);
    if (rc == RA_OK && a.out && a.out_types) rc = check_second("out_dtype", a.out_types[i], a.types[i]);
    if (rc != RA_OK || count == 0) continue;
    const int e = ra::elem_bytes(a.types[i]);
    const int to = a.out && a.out_types ? a.out_types[i] : a.types[i], eo = ra::elem_bytes(to);
    const bool same = a.out && a.out[i] == a.in[i] && to == a.types[i];
    rc = make(&read[reads++], "tensors", i, a.in[i], count * e, e, same);
    if (rc == RA_OK && a.out && !same) rc = make(&written[writes++], "outs", i, a.out[i], count * eo, eo, true);
    bytes += count * (e + (a.out ? eo : 0));
  }
  if (rc != RA_OK) return rc;
  a.stream = bytes > ra::kStreamingBytes;
  sort_spans(read, reads);
  sort_spans(written, writes);
  std::merge(read, read + reads, written, written + writes, all, before);
  for (int64_t i = 0; i < reads + writes; ++i)
    for (const Span& x : own)
      if (all[i].lo < x.hi && x.lo < all[i].hi) return overlap(all[i], x);
  return check_spans(all, reads + writes);
}

}  // namespace

extern "C" {

int ra_allreduce_rmsnorm(void* const* bufs, int p, int64_t tokens, int64_t hidden, int dtype,
                         const void* residual_in, void* residual_out, int residual_dtype, const void* weight,
                         float eps, void* const* outs, int n_out, int out_dtype, float* const* scales, int group,
                         float* rstd, hipStream_t stream) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_rows(tokens, hidden, ra::kNormMaxHidden, "hidden");
  const bool res = residual_in || residual_out;
  if (rc == RA_OK && res) rc = check_second("residual_dtype", residual_dtype, dtype);
  if (rc == RA_OK) rc = check_count("n_out", n_out, 1, p);
  if (rc != RA_OK) return rc;
  const bool f8 = out_dtype == RA_FLOAT8_E4M3;
  if (!f8 && out_dtype != dtype) {
    rc = check_real("out_dtype", out_dtype);
    return rc != RA_OK ? rc
                       : fail(RA_ERR_UNSUPPORTED, "out_dtype %d: need the buffers' type or RA_FLOAT8_E4M3", out_dtype);
  }
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return fail(RA_ERR_INVALID_ARG, "group = %d, need 0, 32, 64 or 128", group);
  if (group != 0 && !f8) return fail(RA_ERR_INVALID_ARG, "group needs an 8-bit output");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(RA_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (tokens == 0) return RA_OK;

  const int e = ra::elem_bytes(dtype), er = res ? ra::elem_bytes(residual_dtype) : 1, eo = f8 ? 1 : e;
  const int64_t n = tokens * hidden, groups = group ? (hidden + group - 1) / group : 1;
  Arrays all;
  ra::NormArgs a;
  std::memset(&a, 0, sizeof a);
  rc = add_ranks(&all, "bufs", bufs, p, n * e, e, false, &a.in);
  if (rc == RA_OK) rc = all.add("weight", -1, weight, hidden * e, e, false);
  if (rc == RA_OK) rc = all.add("residual_in", -1, residual_in, n * er, er, false, true);
  if (rc == RA_OK && residual_out)
    rc = residual_out == residual_in ? all.add_or_same("residual_out", -1, residual_out, n * er, er)
                                     : all.add("residual_out", -1, residual_out, n * er, er, true);
  if (rc == RA_OK) rc = all.add("rstd", -1, rstd, tokens * 4, 4, true, true, 1);
  if (rc != RA_OK) return rc;
  if (!outs) return fail(RA_ERR_INVALID_ARG, "outs is NULL");
  for (int r = 0; r < n_out; ++r) {
    // a rank's output may take the place of a rank's partial
    bool same = false;
    for (int q = 0; q < p; ++q) same = same || outs[r] == bufs[q];
    rc = same && !f8 ? all.add_or_same("outs", r, outs[r], n * eo, eo)
                     : all.add("outs", r, outs[r], n * eo, eo, true, false, f8 ? 8 : 16);
    if (rc != RA_OK) return rc;
    a.out.b[r] = outs[r];
  }
  if (f8) {
    rc = add_ranks(&all, "scales", reinterpret_cast<const void* const*>(scales), n_out, tokens * groups * 4, 4, true,
                   &a.scale, 1);
    if (rc != RA_OK) return rc;
  }
  rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.res = residual_in;
  a.res_out = residual_out;
  a.weight = weight;
  a.rstd = rstd;
  a.tokens = tokens;
  a.hidden = (int32_t)hidden;
  a.p = p;
  a.n_out = n_out;
  a.group = group;
  a.eps = eps;
  a.inv_h = 1.0f / (float)hidden;
  const bool al = all.al() && hidden % 8 == 0;
  debug_rows("allreduce_rmsnorm", p, tokens, hidden, dtype, al, 1);
  return launched(ra::launch_norm(
      a, dtype, residual_dtype, f8, access_of(al, n * (p * e + (residual_in ? er : 0) + (residual_out ? er : 0) + n_out * eo)),
      stream));
}

int ra_allreduce_rmsnorm_backward_workspace(int64_t tokens, int64_t hidden, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_rows(tokens, hidden, ra::kNormMaxHidden, "hidden");
  if (rc == RA_OK) *bytes = norm_bwd_bytes(tokens, hidden);
  return rc;
}

int ra_allreduce_rmsnorm_backward(void* const* dys, int p, int64_t tokens, int64_t hidden, int dtype, const void* h,
                                  int h_dtype, const float* rstd, const void* weight, const void* dh_in, void* dh,
                                  void* const* dxs, int n_dx, float* dweight, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_rows(tokens, hidden, ra::kNormMaxHidden, "hidden");
  if (rc == RA_OK) rc = check_second("h_dtype", h_dtype, dtype);
  if (rc == RA_OK) rc = check_count("n_dx", n_dx, 0, p);
  if (rc != RA_OK) return rc;
  if (tokens == 0 && !dweight) return RA_OK;

  const int e = ra::elem_bytes(dtype), eh = ra::elem_bytes(h_dtype);
  const int64_t n = tokens * hidden;
  Arrays all;
  ra::NormBwdArgs a;
  std::memset(&a, 0, sizeof a);
  if (tokens > 0) {
    rc = add_ranks(&all, "dys", dys, p, n * e, e, false, &a.in);
    if (rc == RA_OK) rc = all.add("h", -1, h, n * eh, eh, false);
    if (rc == RA_OK) rc = all.add("rstd", -1, rstd, tokens * 4, 4, false, false, 1);
    if (rc == RA_OK) rc = all.add("weight", -1, weight, hidden * e, e, false);
    if (rc == RA_OK) rc = all.add("dh_in", -1, dh_in, n * eh, eh, false, true);
    if (rc == RA_OK)
      rc = dh && dh == dh_in ? all.add_or_same("dh", -1, dh, n * eh, eh) : all.add("dh", -1, dh, n * eh, eh, true);
    if (rc == RA_OK && n_dx > 0 && !dxs) rc = fail(RA_ERR_INVALID_ARG, "dxs is NULL");
    for (int r = 0; r < n_dx && rc == RA_OK; ++r) {
      bool same = false;
      for (int q = 0; q < p; ++q) same = same || dxs[r] == dys[q];
      rc = same ? all.add_or_same("dxs", r, dxs[r], n * e, e) : all.add("dxs", r, dxs[r], n * e, e, true);
      a.dx.b[r] = dxs[r];
    }
  }
  if (rc == RA_OK) rc = all.add("dweight", -1, dweight, hidden * 4, 4, true, true, 1);
  if (rc == RA_OK && dweight)
    rc = check_workspace(&all, workspace, workspace_bytes, norm_bwd_bytes(tokens, hidden));
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.h = h;
  a.rstd = rstd;
  a.weight = weight;
  a.dh_in = dh_in;
  a.dh = dh;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  a.tokens = tokens;
  a.hidden = (int32_t)hidden;
  a.p = p;
  a.n_dx = n_dx;
  a.inv_h = 1.0f / (float)hidden;
  const bool al = all.al() && hidden % 8 == 0;
  debug_rows("allreduce_rmsnorm_backward", p, tokens, hidden, dtype, al, 1);
  return launched(ra::launch_norm_bwd(
      a, dtype, h_dtype, dweight, access_of(al, n * (p * e + (dh_in ? 3 : 2) * eh + n_dx * e)), stream));
}

int ra_cross_entropy_workspace(int64_t tokens, int64_t vocab, int p, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_rows(tokens, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK) *bytes = std::max(xent_bytes(tokens, vocab, p, false), xent_bytes(tokens, vocab, p, true));
  return rc;
}

int ra_cross_entropy(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype,
                     const void* targets, int target_dtype, float* loss, float* lse, void* const* grads,
                     const float* dloss, float grad_scale, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  int rc = check_xent(logits, p, tokens, vocab, valid, dtype, target_dtype);
  if (rc != RA_OK) return rc;
  if (tokens == 0) return RA_OK;   // before the next line: an empty array's address may be NULL
  if (!loss && !lse && !grads) return fail(RA_ERR_INVALID_ARG, "loss, lse and grads are all NULL");
  Arrays all;
  ra::XentArgs a;
  std::memset(&a, 0, sizeof a);
  rc = add_xent(&all, &a, logits, grads, p, tokens, vocab, valid, dtype, targets, target_dtype, dloss, grad_scale);
  if (rc == RA_OK) rc = all.add("loss", -1, loss, tokens * 4, 4, true, true, 1);
  if (rc == RA_OK) rc = all.add("lse", -1, lse, tokens * 4, 4, true, true, 1);
  if (rc == RA_OK) rc = check_workspace(&all, workspace, workspace_bytes, xent_bytes(tokens, vocab, p, grads != nullptr));
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.loss = loss;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.splits = ra::xent_splits(tokens, (int)vocab, p, grads != nullptr);
  const bool al = all.al() && a.cut.extra == 0 && a.cut.base % 8 == 0;
  debug_rows("cross_entropy", p, tokens, vocab, dtype, al, a.splits);
  return launched(ra::launch_xent(a, dtype, grads != nullptr, al, stream));
}

int ra_cross_entropy_backward(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype,
                              const void* targets, int target_dtype, const float* lse, void* const* grads,
                              const float* dloss, float grad_scale, hipStream_t stream) {
  int rc = check_xent(logits, p, tokens, vocab, valid, dtype, target_dtype);
  if (rc != RA_OK) return rc;
  if (!grads) return fail(RA_ERR_INVALID_ARG, "grads is NULL");
  if (tokens == 0) return RA_OK;
  Arrays all;
  ra::XentArgs a;
  std::memset(&a, 0, sizeof a);
  rc = add_xent(&all, &a, logits, grads, p, tokens, vocab, valid, dtype, targets, target_dtype, dloss, grad_scale);
  if (rc == RA_OK) rc = all.add("lse", -1, lse, tokens * 4, 4, false, false, 1);
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.lse_in = lse;
  // A row is cut so that a wave has about four chunks.
  a.splits = (int32_t)std::max<int64_t>(1, (int64_t)a.total / 16);
  const bool al = all.al() && a.cut.extra == 0 && a.cut.base % 8 == 0;
  debug_rows("cross_entropy_backward", p, tokens, vocab, dtype, al, a.splits);
  return launched(ra::launch_xent_bwd(a, dtype, al, stream));
}

int ra_embedding(const void* const* tables, int p, int64_t vocab, int64_t hidden, int dtype, const void* ids,
                 int id_dtype, int64_t tokens, float scale, void* const* outs, int n_out, hipStream_t stream) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_index("id_dtype", id_dtype);
  if (rc == RA_OK) rc = check_rows(tokens, hidden, ra::kEmbedMaxHidden, "hidden");
  if (rc == RA_OK) rc = check_rows(0, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK) rc = check_count("n_out", n_out, 1, p);
  if (rc != RA_OK) return rc;
  if (tokens == 0) return RA_OK;
  const int e = ra::elem_bytes(dtype), ei = ra::elem_bytes(id_dtype);
  Arrays all;
  ra::EmbedArgs a;
  std::memset(&a, 0, sizeof a);
  a.cut = {(int32_t)(vocab / p), (int32_t)(vocab % p)};
  if (!tables) return fail(RA_ERR_INVALID_ARG, "tables is NULL");
  for (int r = 0; r < p && rc == RA_OK; ++r) {
    rc = all.add("tables", r, tables[r], (int64_t)(a.cut.base + (r < a.cut.extra)) * hidden * e, e, false);
    a.table.b[r] = const_cast<void*>(tables[r]);
  }
  if (rc == RA_OK) rc = all.add("ids", -1, ids, tokens * ei, ei, false, false, 1);
  if (rc == RA_OK)
    rc = add_ranks(&all, "outs", const_cast<const void* const*>(outs), n_out, tokens * hidden * e, e, true, &a.out);
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.ids = ids;
  a.ids64 = id_dtype == RA_INT64;
  a.tokens = tokens;
  a.p = p;
  a.vocab = (int32_t)vocab;
  a.hidden = (int32_t)hidden;
  a.n_out = n_out;
  a.scale = scale;
  const bool al = all.al() && hidden % 8 == 0;
  debug_rows("embedding", p, tokens, hidden, dtype, al, 1);
  return launched(ra::launch_embed(a, dtype, access_of(al, tokens * hidden * e * n_out), stream));
}

int ra_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_rows(tokens, hidden, ra::kEmbedMaxHidden, "hidden");
  if (rc == RA_OK) rc = check_rows(0, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK) rc = check_embed_bwd(tokens, vocab, hidden);
  if (rc == RA_OK) *bytes = ra::embed_bwd_words(tokens, (int)hidden) * 4;
  return rc;
}

int ra_embedding_backward(const void* dy, int64_t tokens, int64_t hidden, int dtype, const void* ids, int id_dtype,
                          float scale, void* const* dtables, int p, int64_t vocab, int dtable_dtype, int accumulate,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_second("dtable_dtype", dtable_dtype, dtype);
  if (rc == RA_OK) rc = check_index("id_dtype", id_dtype);
  if (rc == RA_OK) rc = check_rows(tokens, hidden, ra::kEmbedMaxHidden, "hidden");
  if (rc == RA_OK) rc = check_rows(0, vocab, ra::kXentMaxVocab, "vocab");
  if (rc != RA_OK) return rc;
  rc = check_embed_bwd(tokens, vocab, hidden);
  if (rc != RA_OK) return rc;
  if (tokens == 0 && accumulate) return RA_OK;
  const int e = ra::elem_bytes(dtype), et = ra::elem_bytes(dtable_dtype), ei = ra::elem_bytes(id_dtype);
  const int64_t need = ra::embed_bwd_words(tokens, (int)hidden) * 4;
  Arrays all;
  ra::EmbedBwdArgs a;
  std::memset(&a, 0, sizeof a);
  a.cut = {(int32_t)(vocab / p), (int32_t)(vocab % p)};
  if (!dtables) return fail(RA_ERR_INVALID_ARG, "dtables is NULL");
  for (int r = 0; r < p && rc == RA_OK; ++r) {
    rc = all.add("dtables", r, dtables[r], (int64_t)(a.cut.base + (r < a.cut.extra)) * hidden * et, et, true);
    a.table.b[r] = dtables[r];
  }
  if (rc == RA_OK) rc = all.add("dy", -1, dy, tokens * hidden * e, e, false);
  if (rc == RA_OK) rc = all.add("ids", -1, ids, tokens * ei, ei, false, false, 1);
  if (rc == RA_OK) rc = check_workspace(&all, workspace, workspace_bytes, need);
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.dy = dy;
  a.ids = ids;
  a.ids64 = id_dtype == RA_INT64;
  a.work = static_cast<int32_t*>(workspace);
  a.tokens = tokens;
  a.p = p;
  a.vocab = (int32_t)vocab;
  a.hidden = (int32_t)hidden;
  a.accumulate = accumulate != 0;
  a.scale = scale;
  const bool al = all.al() && hidden % 8 == 0;
  debug_rows("embedding_backward", p, tokens, hidden, dtype, al, 1);
  return launched(ra::launch_embed_bwd(a, dtype, dtable_dtype, al, stream));
}

int ra_token_logprobs_workspace(int64_t tokens, int64_t vocab, int p, int top, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_rows(tokens, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK) rc = check_top(vocab, top);
  if (rc == RA_OK) *bytes = logprob_bytes(tokens, vocab, p, top);
  return rc;
}

int ra_token_logprobs(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype,
                      float scale, const void* ids, int id_dtype, float* logprob, float* entropy, float* lse, int top,
                      void* top_ids, float* top_logprobs, void* workspace, int64_t workspace_bytes,
                      hipStream_t stream) {
  int rc = check_vocab(logits, p, tokens, vocab, valid, dtype, "id_dtype", id_dtype);
  if (rc == RA_OK) rc = check_positive("scale", scale);
  if (rc == RA_OK) rc = check_top(valid, top);
  if (rc != RA_OK) return rc;
  if (tokens == 0) return RA_OK;   // before the next lines: an empty array's address may be NULL
  if (top > 0 && !top_ids && !top_logprobs) return fail(RA_ERR_INVALID_ARG, "top_ids and top_logprobs are both NULL");
  if (!logprob && !entropy && !lse && top == 0)
    return fail(RA_ERR_INVALID_ARG, "logprob, entropy and lse are all NULL, and top is 0");
  if (logprob && !ids) return fail(RA_ERR_INVALID_ARG, "logprob needs ids");
  Arrays all;
  ra::LogpArgs a;
  std::memset(&a, 0, sizeof a);
  rc = add_vocab(&all, &a, logits, nullptr, p, tokens, vocab, valid, dtype);
  const int ei = ra::elem_bytes(id_dtype);
  if (rc == RA_OK) rc = all.add("ids", -1, ids, tokens * ei, ei, false, true, 1);
  if (rc == RA_OK) rc = all.add("logprob", -1, logprob, tokens * 4, 4, true, true, 1);
  if (rc == RA_OK) rc = all.add("entropy", -1, entropy, tokens * 4, 4, true, true, 1);
  if (rc == RA_OK) rc = all.add("lse", -1, lse, tokens * 4, 4, true, true, 1);
  if (rc == RA_OK && top > 0) rc = all.add("top_ids", -1, top_ids, tokens * top * ei, ei, true, true, 1);
  if (rc == RA_OK && top > 0) rc = all.add("top_logprobs", -1, top_logprobs, tokens * top * 4, 4, true, true, 1);
  if (rc == RA_OK) rc = check_workspace(&all, workspace, workspace_bytes, logprob_bytes(tokens, vocab, p, top));
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.ids = ids;
  a.ids64 = id_dtype == RA_INT64;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top = top;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.part = static_cast<float*>(workspace);
  a.scale = scale;
  a.splits = ra::logp_splits(tokens, (int)vocab, p);
  const bool al = all.al() && a.cut.extra == 0 && a.cut.base % 8 == 0;
  debug_rows("token_logprobs", p, tokens, vocab, dtype, al, a.splits);
  return launched(ra::launch_logp(a, dtype, access_of(al, tokens * vocab * ra::elem_bytes(dtype)), stream));
}

int ra_token_logprobs_backward(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype,
                               float scale, const void* ids, int id_dtype, const float* lse, const float* entropy,
                               const float* dlogprob, const float* dentropy, void* const* grads,
                               hipStream_t stream) {
  int rc = check_vocab(logits, p, tokens, vocab, valid, dtype, "id_dtype", id_dtype);
  if (rc == RA_OK) rc = check_positive("scale", scale);
  if (rc == RA_OK && !grads) rc = fail(RA_ERR_INVALID_ARG, "grads is NULL");
  if (rc != RA_OK) return rc;
  if (tokens == 0) return RA_OK;
  if (!dlogprob && !dentropy) return fail(RA_ERR_INVALID_ARG, "dlogprob and dentropy are both NULL");
  if (dlogprob && !ids) return fail(RA_ERR_INVALID_ARG, "dlogprob needs ids");
  if (dentropy && !entropy) return fail(RA_ERR_INVALID_ARG, "dentropy needs entropy");
  Arrays all;
  ra::LogpArgs a;
  std::memset(&a, 0, sizeof a);
  rc = add_vocab(&all, &a, logits, grads, p, tokens, vocab, valid, dtype);
  const int ei = ra::elem_bytes(id_dtype);
  if (rc == RA_OK) rc = all.add("ids", -1, ids, tokens * ei, ei, false, true, 1);
  if (rc == RA_OK) rc = all.add("lse", -1, lse, tokens * 4, 4, false, false, 1);
  if (rc == RA_OK) rc = all.add("entropy", -1, entropy, tokens * 4, 4, false, true, 1);
  if (rc == RA_OK) rc = all.add("dlogprob", -1, dlogprob, tokens * 4, 4, false, true, 1);
  if (rc == RA_OK) rc = all.add("dentropy", -1, dentropy, tokens * 4, 4, false, true, 1);
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.ids = ids;
  a.ids64 = id_dtype == RA_INT64;
  a.lse_in = lse;
  a.entropy_in = entropy;
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  a.scale = scale;
  const bool al = all.al() && a.cut.extra == 0 && a.cut.base % 8 == 0;
  debug_rows("token_logprobs_backward", p, tokens, vocab, dtype, al, 1);
  return launched(ra::launch_logp_bwd(a, dtype, al, 2 * tokens * vocab * ra::elem_bytes(dtype) > ra::kStreamingBytes, stream));
}

int ra_grad_norm_workspace(int64_t n, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_list_length(n);
  if (rc == RA_OK) *bytes = ra::grad_norm_bytes(n);
  return rc;
}

int ra_grad_norm(const void* const* tensors, const int64_t* counts, const int* dtypes, int64_t n, float scale,
                 float* norm, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_list_length(n);
  if (rc == RA_OK) rc = check_positive("scale", scale);
  ra::TensorListArgs a = {tensors, nullptr, counts, dtypes, nullptr, n, n, false};
  if (rc == RA_OK) rc = check_list(a, norm, workspace, workspace_bytes);
  if (rc != RA_OK) return rc;
  debug_rows("grad_norm", 1, n, 0, n > 0 ? dtypes[0] : 0, false, 1);
  return launched(ra::launch_grad_norm(a, {nullptr, nullptr, norm, 0, INFINITY, scale}, workspace, stream));
}

int ra_grad_clip(void* const* tensors, const int64_t* counts, const int* dtypes, int64_t n, int64_t counted,
                 float max_norm, float scale, void* const* outs, const int* out_dtypes, float* norm, void* workspace,
                 int64_t workspace_bytes, hipStream_t stream) {
  int rc = check_list_length(n);
  if (rc == RA_OK && (counted < 0 || counted > n))
    rc = fail(RA_ERR_INVALID_ARG, "counted = %lld, need 0..n = %lld", (long long)counted, (long long)n);
  if (rc == RA_OK) rc = check_clip(max_norm, scale);
  ra::TensorListArgs a = {tensors, outs ? outs : tensors, counts, dtypes, outs ? out_dtypes : nullptr, n, counted, false};
  if (rc == RA_OK) rc = check_list(a, norm, workspace, workspace_bytes);
  if (rc != RA_OK) return rc;
  debug_rows("grad_clip", 1, n, 0, n > 0 ? dtypes[0] : 0, false, 1);
  return launched(ra::launch_grad_clip(a, {nullptr, nullptr, norm, 0, max_norm, scale}, workspace, stream));
}

int ra_allreduce_clip_workspace(int64_t n, int64_t* bytes) {
  if (!bytes) return fail(RA_ERR_INVALID_ARG, "bytes is NULL");
  int rc = check_elements(n);
  if (rc == RA_OK) *bytes = ra::fold_clip_bytes(n);
  return rc;
}

int ra_allreduce_clip(void* const* bufs, int p, int64_t n, int dtype, int op, float max_norm, float scale,
                      void* const* outs, int n_out, float* norm, void* workspace, int64_t workspace_bytes,
                      hipStream_t stream) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_elements(n);
  if (rc == RA_OK) rc = check_count("n_out", n_out, 1, p);
  if (rc == RA_OK) rc = check_clip(max_norm, scale);
  if (rc != RA_OK) return rc;
  if (op != RA_SUM && op != RA_AVG) {
    if (op != RA_MAX) return fail(RA_ERR_INVALID_ARG, "unknown op %d", op);
    return fail(RA_ERR_UNSUPPORTED, "op %d: need RA_SUM or RA_AVG", op);
  }
  const int e = ra::elem_bytes(dtype);
  Arrays all;
  ra::FoldArgs a;
  std::memset(&a, 0, sizeof a);
  if (n > 0) {
    rc = add_ranks(&all, "bufs", bufs, p, n * e, e, false, &a.in);
    if (rc == RA_OK && !outs) rc = fail(RA_ERR_INVALID_ARG, "outs is NULL");
    for (int r = 0; r < n_out && rc == RA_OK; ++r) {
      // a rank's output may take the place of a rank's buffer
      bool same = false;
      for (int q = 0; q < p; ++q) same = same || outs[r] == bufs[q];
      rc = same ? all.add_or_same("outs", r, outs[r], n * e, e) : all.add("outs", r, outs[r], n * e, e, true);
      a.out.b[r] = outs[r];
    }
  }
  if (rc == RA_OK) rc = all.add("norm", -1, norm, 4, 4, true);
  if (rc == RA_OK) rc = check_workspace(&all, workspace, workspace_bytes, ra::fold_clip_bytes(n));
  if (rc == RA_OK) rc = all.overlaps();
  if (rc != RA_OK) return rc;
  a.n = n;
  a.p = p;
  a.n_out = n_out;
  a.mean = op == RA_AVG;
  debug_rows("allreduce_clip", p, n, 1, dtype, false, 1);
  return launched(ra::launch_fold_clip(a, dtype, {nullptr, nullptr, norm, 0, max_norm, scale},
                                       n * e * (p + n_out) > ra::kStreamingBytes, workspace, stream));
}

}  // extern "C"
