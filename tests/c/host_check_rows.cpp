// host_check_rows.cpp -- the host side of the row operators (argument checks, the list
// of a call's arrays and its overlaps, workspace sizes) exercised without a GPU, built
// with AddressSanitizer on the library's host code.  No call here reaches a kernel:
// every one is refused, has no tokens, or needs no device.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "ra.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("FAIL %s: %d, expected %d (last error: %s)\n", what, got, want, ra_last_error());
    ++failures;
  }
}

// Addresses a MiB apart that nothing is at: calls only compare them.
static uintptr_t at(int i) { return uintptr_t(0x7f0000000000ull) + uintptr_t(i) * (1 << 20); }
static void* ptr(int i) { return reinterpret_cast<void*>(at(i)); }
static float* f32(int i) { return reinterpret_cast<float*>(at(i)); }
// Arrays whose pointer table ends with them, so that a read past it is found.
static std::vector<void*> table(int first, int n) {
  std::vector<void*> v(n);
  for (int i = 0; i < n; ++i) v[i] = ptr(first + i);
  return v;
}
static std::vector<float*> floats(int first, int n) {
  std::vector<float*> v(n);
  for (int i = 0; i < n; ++i) v[i] = f32(first + i);
  return v;
}

constexpr int64_t T = 64;            // tokens

// Every array that a call can have, at every p; `bad` (or -1) is laid over another one.
static void norm(int p, int hidden, int group, int bad, int other) {
  std::vector<void*> bufs = table(0, p), outs = table(64, p), scales = table(128, p);
  void* more[4] = {ptr(192), ptr(193), ptr(194), ptr(195)};     // residual in and out, weight, rstd
  auto place = [&](int i) -> void** {
    return i < p ? &bufs[i] : i < 2 * p ? &outs[i - p] : i < 3 * p ? &scales[i - 2 * p] : &more[i - 3 * p];
  };
  *place(bad) = *place(other);
  expect(ra_allreduce_rmsnorm(bufs.data(), p, T, hidden, RA_BFLOAT16, more[0], more[1], RA_FLOAT32, more[2], 1e-5f,
                              outs.data(), p, RA_FLOAT8_E4M3, reinterpret_cast<float* const*>(scales.data()), group, static_cast<float*>(more[3]),
                              nullptr), RA_ERR_ALIAS, "norm with arrays laid over each other");
}

static void norm_backward(int p, int bad, int other) {
  std::vector<void*> dys = table(0, p), dxs = table(64, p);
  void* more[7] = {ptr(128), ptr(129), ptr(130), ptr(131), ptr(132), ptr(133), ptr(134)};
  auto place = [&](int i) -> void** { return i < p ? &dys[i] : i < 2 * p ? &dxs[i - p] : &more[i - 2 * p]; };
  *place(bad) = *place(other);
  int64_t bytes = 0;
  expect(ra_allreduce_rmsnorm_backward_workspace(T, 1000, &bytes), RA_OK, "norm backward workspace");
  // h, rstd, weight, dh_in, dh, dweight, workspace
  expect(ra_allreduce_rmsnorm_backward(dys.data(), p, T, 1000, RA_BFLOAT16, more[0], RA_FLOAT32,
                                       static_cast<float*>(more[1]), more[2], more[3], more[4], dxs.data(), p,
                                       static_cast<float*>(more[5]), more[6], bytes, nullptr),
         RA_ERR_ALIAS, "norm backward with arrays laid over each other");
}

static void cross_entropy(int p, int bad, int other) {
  std::vector<void*> logits = table(0, p), grads = table(64, p);
  void* more[5] = {ptr(128), ptr(129), ptr(130), ptr(131), ptr(132)};   // targets, dloss, loss, lse, workspace
  auto place = [&](int i) -> void** { return i < p ? &logits[i] : i < 2 * p ? &grads[i - p] : &more[i - 2 * p]; };
  *place(bad) = *place(other);
  int64_t bytes = 0;
  expect(ra_cross_entropy_workspace(T, 65536, p, &bytes), RA_OK, "cross entropy workspace");
  expect(ra_cross_entropy(logits.data(), p, T, 65536, 65000, RA_FLOAT16, more[0], RA_INT64,
                          static_cast<float*>(more[2]), static_cast<float*>(more[3]), grads.data(),
                          static_cast<float*>(more[1]), 1.0f, more[4], bytes, nullptr),
         RA_ERR_ALIAS, "cross entropy with arrays laid over each other");
  if (bad == 2 * p + 3 && other >= p && other < 2 * p)       // lse is read there, the gradients written
    expect(ra_cross_entropy_backward(logits.data(), p, T, 65536, 65000, RA_FLOAT16, more[0], RA_INT64,
                                     static_cast<float*>(more[3]), grads.data(), static_cast<float*>(more[1]), 1.0f,
                                     nullptr), RA_ERR_ALIAS, "its backward");
}

static void embedding(int p, int bad, int other) {
  std::vector<void*> tables = table(0, p), outs = table(64, p);
  void* ids = ptr(128);
  auto place = [&](int i) -> void** { return i < p ? &tables[i] : i < 2 * p ? &outs[i - p] : &ids; };
  *place(bad) = *place(other);
  expect(ra_embedding(tables.data(), p, 6400, 264, RA_FLOAT16, ids, RA_INT32, T, 1.0f, outs.data(), p, nullptr),
         RA_ERR_ALIAS, "embedding with arrays laid over each other");
}

static void embedding_backward(int p, int bad, int other) {
  std::vector<void*> tables = table(0, p);
  void* more[3] = {ptr(64), ptr(65), ptr(66)};    // dy, ids, workspace
  auto place = [&](int i) -> void** { return i < p ? &tables[i] : &more[i - p]; };
  *place(bad) = *place(other);
  int64_t bytes = 0;
  expect(ra_embedding_backward_workspace(T, 6400, 264, &bytes), RA_OK, "embedding backward workspace");
  expect(ra_embedding_backward(more[0], T, 264, RA_BFLOAT16, more[1], RA_INT64, 1.0f, tables.data(), p, 6400,
                               RA_FLOAT32, 0, more[2], bytes, nullptr),
         RA_ERR_ALIAS, "embedding backward with arrays laid over each other");
}

int main() {
  std::mt19937_64 rng(11);
  // An array that is written, laid over any other one of its call.
  for (int trial = 0; trial < 300; ++trial) {
    const int p = trial < 3 ? RA_MAX_RANKS : 1 + int(rng() % RA_MAX_RANKS);
    auto two = [&](int n, int lo, int hi, int* bad, int* other) {
      *bad = lo + int(rng() % (hi - lo));
      do *other = int(rng() % n);
      while (*other == *bad);
    };
    int bad, other;
    two(3 * p + 4, p, 3 * p, &bad, &other);                     // an output or a scale
    norm(p, 1000, trial % 2 ? 128 : 0, bad, other);
    two(2 * p + 7, 2 * p + 5, 2 * p + 7, &bad, &other);         // dweight or the workspace
    norm_backward(p, bad, other);
    two(2 * p + 5, 2 * p + 2, 2 * p + 5, &bad, &other);         // loss, lse, the workspace
    cross_entropy(p, bad, other);
    two(2 * p + 1, p, 2 * p, &bad, &other);                     // an output
    embedding(p, bad, other);
    two(p + 3, 0, p, &bad, &other);                             // a table's gradient
    embedding_backward(p, bad, other);
  }

  // missing arrays and tables, at the largest p; the last pointer of each list
  const int p = RA_MAX_RANKS;
  std::vector<void*> a = table(0, p), b = table(64, p), none = table(0, p), gap = table(64, p);
  std::vector<float*> s = floats(128, p), no_scale = floats(128, p);
  none[p - 1] = gap[p - 1] = nullptr;
  no_scale[p - 1] = nullptr;
  auto rms = [&](void** in, void** out, float** scales, void* weight, int n_out, int64_t tokens) {
    return ra_allreduce_rmsnorm(in, p, tokens, 512, RA_FLOAT16, ptr(192), ptr(192), RA_FLOAT16, weight, 1e-6f, out,
                                n_out, RA_FLOAT8_E4M3, scales, 64, f32(193), nullptr);
  };
  expect(rms(nullptr, b.data(), s.data(), ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: no buffers");
  expect(rms(none.data(), b.data(), s.data(), ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: a buffer missing");
  expect(rms(a.data(), nullptr, s.data(), ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: no outputs");
  expect(rms(a.data(), gap.data(), s.data(), ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: an output missing");
  expect(rms(a.data(), b.data(), nullptr, ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: no scales");
  expect(rms(a.data(), b.data(), no_scale.data(), ptr(194), p, T), RA_ERR_INVALID_ARG, "norm: a scale missing");
  expect(rms(a.data(), b.data(), s.data(), nullptr, p, T), RA_ERR_INVALID_ARG, "norm: no weight");
  expect(rms(a.data(), b.data(), s.data(), ptr(194), p + 1, T), RA_ERR_INVALID_ARG, "norm: more outputs than ranks");
  expect(rms(a.data(), b.data(), s.data(), ptr(194), p, 0), RA_OK, "norm: no tokens");
  auto ce = [&](void** x, void** dx, const void* targets, int64_t tokens, void* ws, int64_t bytes) {
    return ra_cross_entropy(x, p, tokens, 65536, 65536, RA_FLOAT32, targets, RA_INT32, f32(192), f32(193), dx,
                            nullptr, 1.0f, ws, bytes, nullptr);
  };
  expect(ce(nullptr, b.data(), ptr(194), T, ptr(195), 1 << 20), RA_ERR_INVALID_ARG, "cross entropy: no logits");
  expect(ce(none.data(), b.data(), ptr(194), T, ptr(195), 1 << 20), RA_ERR_INVALID_ARG, "cross entropy: logits missing");
  expect(ce(a.data(), gap.data(), ptr(194), T, ptr(195), 1 << 20), RA_ERR_INVALID_ARG, "cross entropy: a gradient missing");
  expect(ce(a.data(), a.data(), nullptr, T, ptr(195), 1 << 20), RA_ERR_INVALID_ARG, "cross entropy: no targets");
  expect(ce(a.data(), a.data(), ptr(194), T, nullptr, 1 << 20), RA_ERR_INVALID_ARG, "cross entropy: no workspace");
  expect(ce(a.data(), a.data(), ptr(194), T, ptr(195), 16), RA_ERR_INVALID_ARG, "cross entropy: a short workspace");
  expect(ce(a.data(), a.data(), ptr(194), 0, nullptr, 0), RA_OK, "cross entropy: no tokens");
  // pieces without columns or rows may be NULL: 3 over 64 ranks
  std::vector<void*> few(p, nullptr), few_out(p, nullptr);
  for (int r = 0; r < 3; ++r) few[r] = ptr(r), few_out[r] = ptr(64 + r);
  expect(ra_cross_entropy(few.data(), p, T, 3, 2, RA_FLOAT32, nullptr, RA_INT32, f32(192), nullptr, few_out.data(),
                          nullptr, 1.0f, nullptr, 0, nullptr), RA_ERR_INVALID_ARG, "cross entropy of 3 columns");
  expect(ra_embedding(few.data(), p, 3, 8, RA_FLOAT32, nullptr, RA_INT32, T, 1.0f, b.data(), p, nullptr),
         RA_ERR_INVALID_ARG, "embedding of 3 rows");
  expect(ra_embedding_backward(ptr(192), T, 8, RA_FLOAT32, ptr(193), RA_INT32, 1.0f, few.data(), p, 3, RA_FLOAT32, 0,
                               nullptr, 0, nullptr), RA_ERR_INVALID_ARG, "embedding gradient of 3 rows");

  // workspace sizes over the whole range: they ascend with the tokens up to where a call refuses them
  for (int64_t hidden : {int64_t(1), int64_t(1000), int64_t(32768)})
    for (int64_t tokens = 0; tokens < (int64_t(1) << 52) / hidden; tokens = tokens * 3 + 1) {
      int64_t n = -1;
      expect(ra_allreduce_rmsnorm_backward_workspace(tokens, hidden, &n), RA_OK, "norm backward workspace");
      expect(n >= 0 && n <= 512 * hidden * 4, 1, "norm backward workspace size");
      n = -1;
      const int rc = ra_embedding_backward_workspace(tokens, 50000, hidden, &n);
      expect(rc == RA_OK ? n >= 8 * tokens : rc == RA_ERR_UNSUPPORTED && n == -1, 1, "embedding backward workspace");
      n = -1;
      expect(ra_cross_entropy_workspace(tokens, hidden * 100, 8, &n), RA_OK, "cross entropy workspace");
      expect(n >= 0, 1, "cross entropy workspace size");
    }

  std::printf("%s: %d failure(s)\n", failures ? "FAILED" : "PASSED", failures);
  return failures ? 1 : 0;
}
