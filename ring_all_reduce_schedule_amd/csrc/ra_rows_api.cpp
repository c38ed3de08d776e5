// ra_rows_api.cpp -- C entry points of the row operators declared in include/ra.h
// (norm, cross entropy, embedding): argument checks, then one call to the
// launchers in ra_norm.hip, ra_xent.hip and ra_embed.hip.  Nothing here waits,
// allocates or throws.
#include "ra.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

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
    std::sort(list_, list_ + n_, [](const One& a, const One& b) { return a.lo < b.lo; });
    const One *read = nullptr, *written = nullptr;   // the ones so far that end last
    for (int i = 0; i < n_; ++i) {
      const One& x = list_[i];
      const One* with = written && x.lo < written->hi         ? written
                        : x.write && read && x.lo < read->hi ? read
                                                              : nullptr;
      if (with)
        return fail(RA_ERR_ALIAS, "%s (%d) and %s (%d) overlap", with->what, with->index, x.what, x.index);
      const One*& last = x.write ? written : read;
      if (!last || x.hi > last->hi) last = &x;
    }
    return RA_OK;
  }
  bool al() const { return aligned_; }

 private:
  struct One {
    uint64_t lo, hi;
    const char* what;
    int index;
    bool write;
  };
  // Three lists of the ranks' (a norm's buffers, outputs and scales) and single arrays.
  static constexpr int kMost = 3 * RA_MAX_RANKS + 16;
  One list_[kMost];
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

// Logits and gradients of a cross entropy, and what both directions need of them.
int check_xent(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid, int dtype, int target_dtype) {
  int rc = check_ranks(p);
  if (rc == RA_OK) rc = check_real("dtype", dtype);
  if (rc == RA_OK) rc = check_index("target_dtype", target_dtype);
  if (rc == RA_OK) rc = check_rows(tokens, vocab, ra::kXentMaxVocab, "vocab");
  if (rc == RA_OK && (valid < 1 || valid > vocab))
    rc = fail(RA_ERR_INVALID_ARG, "valid = %lld, need 1..vocab = %lld", (long long)valid, (long long)vocab);
  if (rc == RA_OK && !logits) rc = fail(RA_ERR_INVALID_ARG, "logits is NULL");
  return rc;
}

int add_xent(Arrays* to, ra::XentArgs* a, void* const* logits, void* const* grads, int64_t vocab, int64_t valid,
             int dtype, const void* targets, int target_dtype, const float* dloss, float grad_scale) {
  const int e = ra::elem_bytes(dtype), p = a->p;
  a->cut = {(int32_t)(vocab / p), (int32_t)(vocab % p)};
  a->vocab = (int32_t)vocab;
  a->valid = (int32_t)valid;
  a->target = targets;
  a->target64 = target_dtype == RA_INT64;
  a->dloss = dloss;
  a->grad_scale = grad_scale;
  ra::xent_geometry(a);
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
  const int te = ra::elem_bytes(target_dtype);
  if (rc == RA_OK) rc = to->add("targets", -1, targets, a->tokens * te, te, false, false, 1);
  if (rc == RA_OK) rc = to->add("dloss", -1, dloss, a->tokens * 4, 4, false, true, 1);
  return rc;
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
  a.p = p;
  a.tokens = tokens;
  rc = add_xent(&all, &a, logits, grads, vocab, valid, dtype, targets, target_dtype, dloss, grad_scale);
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
  a.p = p;
  a.tokens = tokens;
  rc = add_xent(&all, &a, logits, grads, vocab, valid, dtype, targets, target_dtype, dloss, grad_scale);
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

}  // extern "C"
