// host_check_answers.cpp -- the host side of the log probabilities and of the gradients' norm
// and clipping (argument checks, lists of thousands of tensors and their overlaps, workspace
// sizes) exercised without a GPU, built with AddressSanitizer on the library's host code.  No
// call here reaches a kernel: every one is refused, has no tokens, or needs no device.
#include <algorithm>
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
static void* ptr(int i) { return reinterpret_cast<void*>(uintptr_t(0x7f0000000000ull) + uintptr_t(i) * (1 << 20)); }
static float* f32(int i) { return static_cast<float*>(ptr(i)); }
// A pointer table that ends with its last entry, so that a read past it is found.
static std::vector<void*> table(int first, int n) {
  std::vector<void*> v(n);
  for (int i = 0; i < n; ++i) v[i] = ptr(first + i);
  return v;
}

constexpr int64_t T = 64;            // tokens

// `bad` of the call's arrays is laid over another one.
static void logprobs(int p, int bad, int other) {
  std::vector<void*> x = table(0, p);
  void* more[7] = {ptr(64), ptr(65), ptr(66), ptr(67), ptr(68), ptr(69), ptr(70)};   // ids .. workspace
  auto place = [&](int i) -> void** { return i < p ? &x[i] : &more[i - p]; };
  *place(bad) = *place(other);
  const bool both_read = bad <= p && other <= p;       // logits and ids
  if (both_read) return;
  expect(ra_token_logprobs(x.data(), p, T, 4000, 4000, RA_BFLOAT16, 1.0f, more[0], RA_INT64, static_cast<float*>(more[1]),
                           static_cast<float*>(more[2]), static_cast<float*>(more[3]), 20, more[4],
                           static_cast<float*>(more[5]), more[6], 1 << 20, nullptr),
         RA_ERR_ALIAS, "log probabilities with arrays laid over each other");
}

static void backward(int p, int bad, int other) {
  std::vector<void*> x = table(0, p), dx = table(64, p);
  void* more[5] = {ptr(128), ptr(129), ptr(130), ptr(131), ptr(132)};                // ids, lse, entropy, two gradients
  auto place = [&](int i) -> void** { return i < p ? &dx[i] : &more[i - p]; };
  *place(bad) = *place(other);
  if (bad >= p && other >= p) return;                  // read both
  expect(ra_token_logprobs_backward(x.data(), p, T, 4000, 4000, RA_BFLOAT16, 1.0f, more[0], RA_INT64,
                                    static_cast<float*>(more[1]), static_cast<float*>(more[2]), static_cast<float*>(more[3]),
                                    static_cast<float*>(more[4]), dx.data(), nullptr), RA_ERR_ALIAS, "backward with arrays laid over each other");
}

// n tensors in any order, `bad` over another one (bad == other: over the norm).
static void lists(int n, int bad, int other, bool outs, std::mt19937& g) {
  std::vector<void*> x = table(0, n), y = table(n, n);
  std::vector<int64_t> counts(n);
  std::vector<int> types(n), to(n);
  for (int i = 0; i < n; ++i) {
    counts[i] = 1 + (int64_t)(g() % 100000);
    types[i] = RA_FLOAT32 + (int)(g() % 3);
    to[i] = g() % 2 ? types[i] : (int)RA_FLOAT32;
  }
  std::shuffle(x.begin(), x.end(), g);
  int64_t bytes = 0;
  expect(ra_grad_norm_workspace(n, &bytes), RA_OK, "norm workspace");
  float* norm = f32(2 * n);
  if (bad == other) norm = static_cast<float*>(x[bad]);
  else (outs ? y[bad] : x[bad]) = x[other];
  expect(ra_grad_clip(x.data(), counts.data(), types.data(), n, n, 1.0f, 1.0f, outs ? y.data() : nullptr,
                      outs ? to.data() : nullptr, norm, ptr(2 * n + 1), bytes, nullptr), RA_ERR_ALIAS, "clip with tensors laid over each other");
  if (bad == other)
    expect(ra_grad_norm(x.data(), counts.data(), types.data(), n, 1.0f, norm, ptr(2 * n + 1), bytes, nullptr), RA_ERR_ALIAS, "norm over a tensor");
  expect(ra_grad_norm(x.data(), counts.data(), types.data(), n, 1.0f, f32(2 * n), ptr(2 * n + 1), bytes - 1, nullptr), RA_ERR_INVALID_ARG,
         "norm with too small a workspace");
}

static void fold(int p, int bad, int other) {
  std::vector<void*> x = table(0, p), y = table(64, p);
  void* more[2] = {ptr(128), ptr(129)};                 // norm, workspace
  auto place = [&](int i) -> void** { return i < p ? &y[i] : &more[i - p]; };
  *place(bad) = *place(other);
  int64_t bytes = 0;
  expect(ra_allreduce_clip_workspace(5000, &bytes), RA_OK, "all-reduce workspace");
  expect(ra_allreduce_clip(x.data(), p, 5000, RA_FLOAT16, RA_AVG, 1.0f, 1.0f, y.data(), p, static_cast<float*>(more[0]), more[1], bytes,
                           nullptr), RA_ERR_ALIAS, "all-reduce with arrays laid over each other");
}

int main() {
  std::mt19937 g(1);
  for (int p : {1, 2, 3, 8, 63, 64}) {
    for (int k = 0; k < 300; ++k) {
      auto two = [&](int n, auto f) {
        const int bad = (int)(g() % n), other = (int)(g() % n);
        if (bad != other) f(bad, other);
      };
      // the workspace is not used by 64 tokens of 4000 columns: left out
      two(p + 6, [&](int bad, int other) { logprobs(p, bad, other); });
      two(p + 5, [&](int bad, int other) { backward(p, bad, other); });
      two(p + 2, [&](int bad, int other) { fold(p, bad, other); });
    }
    for (int64_t vocab : {1ll, 511ll, 4096ll, 131072ll, 294913ll, 1ll << 24})
      for (int64_t tokens : {0ll, 1ll, 100ll, 1ll << 20}) {
        int64_t bytes = -1;
        expect(ra_token_logprobs_workspace(tokens, vocab, p, (int)std::min<int64_t>(64, vocab), &bytes), RA_OK, "workspace");
        if (bytes < 0) ++failures;
      }
    std::vector<void*> none(p, nullptr);
    expect(ra_token_logprobs(none.data(), p, 0, 4000, 4000, RA_FLOAT32, 1.0f, nullptr, RA_INT32, nullptr, nullptr, nullptr, 5, nullptr,
                             nullptr, nullptr, 0, nullptr), RA_OK, "no tokens");
    expect(ra_token_logprobs_backward(none.data(), p, 0, 4000, 4000, RA_FLOAT32, 1.0f, nullptr, RA_INT32, nullptr, nullptr, nullptr,
                                      nullptr, none.data(), nullptr), RA_OK, "no tokens, backward");
  }
  for (int n : {1, 2, 7, 156, 157, 232, 233, 1000, 5000})
    for (int k = 0; k < 10; ++k) {
      const int bad = (int)(g() % n), other = (int)(g() % n);
      lists(n, bad, bad, false, g);
      if (bad != other) lists(n, bad, other, false, g), lists(n, bad, other, true, g);
    }
  std::printf(failures ? "FAILED %d\n" : "PASSED\n", failures);
  return failures != 0;
}
