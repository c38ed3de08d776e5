// ra_grads.hip -- what follows the gradients of a model: their global 2-norm, over
// many tensors of any sizes and types, and clipping by it; and both in the passes of
// an all-reduce over the ranks.
//
//   norm = s sqrt(sum over all elements of g^2),   c = s min(1, M / (norm + 1e-6))
//   out = g c
//
// Squares and their sums are float64: float32 would lose the range (bfloat16 goes to
// 3.4e38, whose square float32 has not) and, over 10^9 elements, the precision, and
// the pass is bound by memory either way.  The factor is rounded to float32 once, and
// each product once to float32 and once to the output's type.  Gradients whose norm is
// beyond 10^30 need factors that float32 has few bits for: those are kept as two.
//
// The sums have a fixed order: a workgroup's elements, its threads, and the
// workgroups, whose number depends on the sizes alone.
#include "ra_rows.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kTileUnits = 4;                                  // of a thread
constexpr int kTile = kThreads * kTileUnits * kU;              // elements

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  return x;
}

// Over the workgroup, the same in every lane.  `lds` is free again at the next barrier.
__device__ __forceinline__ double block_sum64(double x, double* lds) {
  x = wave_sum64(x);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  double sum = lds[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) sum += lds[w];
  return sum;
}

// The sum of the workgroups' parts.
__device__ __forceinline__ double parts_sum(const double* part, int n, double* lds) {
  double x = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) x += part[i];
  return block_sum64(x, lds);
}

// g times the factor is g hi lo; lo is 1, or 2^-96 where the factor itself would be near
// float32's end (and hi 2^96 times as large: g hi stays below 2^124).
struct Factor {
  float norm, hi, lo;
};
__device__ __forceinline__ float times(float g, const Factor& f) { return g * f.hi * f.lo; }
__device__ __forceinline__ bool is_one(const Factor& f) { return f.hi == 1.0f && f.lo == 1.0f; }

__device__ __forceinline__ Factor factor_of(double total, const ClipRule& r) {
  const double norm = (double)r.scale * __builtin_sqrt(total);
  const double q = (double)r.max_norm / (norm + 1e-6);
  const double c = (double)r.scale * (q > 1.0 ? 1.0 : q);      // NaN stays
  if (c < 0x1p-100) return {(float)norm, (float)(c * 0x1p96), 0x1p-96f};
  return {(float)norm, (float)c, 1.0f};
}

// The factor, the same in every thread: from the parts, or where k_finish left it.
__device__ __forceinline__ Factor factor(const ClipRule& r, double* lds) {
  if (r.factor) return {0.0f, r.factor[0], r.factor[1]};
  const Factor f = factor_of(parts_sum(r.part, r.parts, lds), r);
  if (blockIdx.x == 0 && threadIdx.x == 0) *r.norm = f.norm;
  return f;
}

// The norm, and the factor for the kernels behind this one (or null).
__global__ __launch_bounds__(1024) void k_finish(ClipRule r, float* to) {
  __shared__ double lds[16];
  const double total = parts_sum(r.part, r.parts, lds);
  if (threadIdx.x == 0) {
    const Factor f = factor_of(total, r);
    *r.norm = f.norm;
    if (to) to[0] = f.hi, to[1] = f.lo;
  }
}

// ---------------------------------------------------------------- many tensors

static_assert(sizeof(TensorBatch) + sizeof(ClipRule) + 16 <= 4096, "a launch's arguments");

// The tensor of a batch that has tile t.
__device__ __forceinline__ int tensor_of(const TensorBatch& b, uint32_t t) {
  int n = 0;
  for (int i = 0; i < kBatchTensors; i += 64)
    n += __builtin_popcountll(__ballot(b.first[i + threadIdx.x % 64 + 1] <= t));
  return __builtin_amdgcn_readfirstlane(n);
}

// The tiles of a workgroup: [lo, hi).
__device__ __forceinline__ void tile_range(uint32_t tiles, uint32_t* lo, uint32_t* hi) {
  *lo = (uint32_t)((uint64_t)tiles * blockIdx.x / gridDim.x);
  *hi = (uint32_t)((uint64_t)tiles * (blockIdx.x + 1) / gridDim.x);
}

// The thread's units of a tile of `len` elements at x.
template <int DT>
__device__ __forceinline__ void load_tile(Unit<DT>* t, const void* x, int len) {
#pragma unroll
  for (int u = 0; u < kTileUnits; ++u) {
    const int j = threadIdx.x + u * kThreads;
    t[u] = Unit<DT>{};
    if (j * kU < len) t[u] = load_cut<DT, kOddRows>(x, 0, unit_cut<kOddRows>(j, len));
  }
}

template <int DT>
__device__ __forceinline__ void add_squares(double* acc, const Unit<DT>& t, const Cut& cut) {
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const double x = owns<kOddRows>(cut, k) ? (double)unit_get<DT>(t, k) : 0.0;
    acc[k % 4] = __builtin_fma(x, x, acc[k % 4]);
  }
}

template <int DT>
__device__ __forceinline__ void tile_squares(double* acc, const void* x, int len) {
  Unit<DT> t[kTileUnits];
  load_tile<DT>(t, x, len);
#pragma unroll
  for (int u = 0; u < kTileUnits; ++u) {
    const int j = threadIdx.x + u * kThreads;
    if (j * kU < len) add_squares<DT>(acc, t[u], unit_cut<kOddRows>(j, len));
  }
}

// A workgroup takes a run of tiles, whichever tensors they are of.
__global__ __launch_bounds__(kThreads) void k_squares(TensorBatch b, double* part) {
  __shared__ double lds[kThreads / 64];
  uint32_t t, hi;
  tile_range(b.first[kBatchTensors], &t, &hi);
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int i = tensor_of(b, t); t < hi; ++t) {
    while (t >= b.first[i + 1]) ++i;
    const int64_t at = (int64_t)(t - b.first[i]) * kTile;
    const int len = (int)min((int64_t)kTile, b.count[i] - at);
    const int type = b.type[i] & 15;
    const char* x = static_cast<const char*>(b.in[i]) + at * (type == 1 ? 4 : 2);
    if (type == 1) tile_squares<1>(acc, x, len);
    else if (type == 2) tile_squares<2>(acc, x, len);
    else tile_squares<3>(acc, x, len);
  }
  const double sum = block_sum64((acc[0] + acc[1]) + (acc[2] + acc[3]), lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <int DT, int OUT>
__device__ __forceinline__ void tile_scale(const void* x, void* y, int len, const Factor& c) {
  Unit<DT> t[kTileUnits];
  load_tile<DT>(t, x, len);
#pragma unroll
  for (int u = 0; u < kTileUnits; ++u) {
    const int j = threadIdx.x + u * kThreads;
    if (j * kU < len) {
      float v[kU];
#pragma unroll
      for (int k = 0; k < kU; ++k) v[k] = times(unit_get<DT>(t[u], k), c);
      store_cut<OUT, kOddRows>(y, 0, unit_cut<kOddRows>(j, len), unit_make<OUT>(v));
    }
  }
}

// A factor of one leaves what is scaled in place as it is.
__global__ __launch_bounds__(kThreads) void k_scale(TensorBatch b, ClipRule r) {
  __shared__ double lds[kThreads / 64];
  const Factor c = factor(r, lds);
  uint32_t t, hi;
  tile_range(b.first[kBatchTensors], &t, &hi);
  for (int i = tensor_of(b, t); t < hi; ++t) {
    while (t >= b.first[i + 1]) ++i;
    if (is_one(c) && b.in[i] == b.out[i]) continue;
    const int64_t at = (int64_t)(t - b.first[i]) * kTile;
    const int len = (int)min((int64_t)kTile, b.count[i] - at);
    const int type = b.type[i] & 15, out = b.type[i] >> 4;
    const char* x = static_cast<const char*>(b.in[i]) + at * (type == 1 ? 4 : 2);
    char* y = static_cast<char*>(b.out[i]) + at * (out == 1 ? 4 : 2);
    if (type == 1) tile_scale<1, 1>(x, y, len, c);
    else if (type == 2 && out == 2) tile_scale<2, 2>(x, y, len, c);
    else if (type == 2) tile_scale<2, 1>(x, y, len, c);
    else if (out == 3) tile_scale<3, 3>(x, y, len, c);
    else tile_scale<3, 1>(x, y, len, c);
  }
}

// ---------------------------------------------------------------- ranks

constexpr int kFoldTile = kThreads * kU;

// The sum (mean) over the ranks, rounded to the buffers' type, into `to`, and the
// squares of what was rounded.  `to` may be one of the buffers: a unit is read from all of them
// by the thread that writes it.
template <int DT, int AC>
__global__ __launch_bounds__(kThreads) void k_fold_squares(FoldArgs a, double* part) {
  __shared__ double lds[kThreads / 64];
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int64_t step = (int64_t)gridDim.x * kFoldTile;
  for (int64_t at = (int64_t)blockIdx.x * kFoldTile; at < a.n; at += step) {
    const int len = (int)min((int64_t)kFoldTile, a.n - at), j = threadIdx.x;
    if (j * kU >= len) continue;
    const Cut cut = unit_cut<AC>(j, len);
    float x[kU];
    fold_ranks<DT, AC>(x, a.in, a.p, at, cut);
    if (a.mean) {
#pragma unroll
      for (int k = 0; k < kU; ++k) x[k] = x[k] / (float)a.p;
    }
    const Unit<DT> t = unit_make<DT>(x);
    store_cut<DT, AC>(a.out.b[0], at, cut, t);
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const double g = owns<AC>(cut, k) ? (double)unit_get<DT>(t, k) : 0.0;
      acc[k % 4] = __builtin_fma(g, g, acc[k % 4]);
    }
  }
  const double sum = block_sum64((acc[0] + acc[1]) + (acc[2] + acc[3]), lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// What k_fold_squares left in the first output, times the factor, to all of them.
template <int DT, int AC>
__global__ __launch_bounds__(kThreads) void k_spread(FoldArgs a, ClipRule r) {
  __shared__ double lds[kThreads / 64];
  const Factor c = factor(r, lds);
  const int64_t step = (int64_t)gridDim.x * kFoldTile;
  for (int64_t at = (int64_t)blockIdx.x * kFoldTile; at < a.n; at += step) {
    const int len = (int)min((int64_t)kFoldTile, a.n - at), j = threadIdx.x;
    if (j * kU >= len) continue;
    const Cut cut = unit_cut<AC>(j, len);
    const Unit<DT> t = load_cut<DT, AC>(a.out.b[0], at, cut);
    float v[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) v[k] = times(unit_get<DT>(t, k), c);
    const Unit<DT> y = unit_make<DT>(v);
    for (int o = 0; o < a.n_out; ++o) store_cut<DT, AC>(a.out.b[o], at, cut, y);
  }
}

// More parts than this are summed once, by a launch of their own, and not by every
// workgroup that needs the factor.
constexpr int kPartsMost = 2048;

// Where k_finish leaves the factor: in front of the parts.
float* factor_at(void* work) { return static_cast<float*>(work); }
double* parts_at(void* work) { return static_cast<double*>(work) + 2; }

hipError_t finish(const ClipRule& r, float* to, hipStream_t s) {
  k_finish<<<1, 1024, 0, s>>>(r, to);
  return hipGetLastError();
}

// Parts or the factor, for the kernel that scales.
hipError_t rule_for(ClipRule* r, void* work, hipStream_t s) {
  if (r->parts <= kPartsMost) return hipSuccess;
  hipError_t e = finish(*r, factor_at(work), s);
  r->factor = factor_at(work);
  return e;
}

unsigned batch_grid(const TensorBatch& b) { return std::min<uint32_t>(b.first[kBatchTensors], kSquaresGrid); }

// Runs `go` on the tensors [from, to) of a list, as many of them at a time as a launch takes.
template <typename F>
hipError_t each_batch(const TensorListArgs& a, int64_t from, int64_t to, F go) {
  TensorBatch b;
  while (from < to) {
    uint32_t tiles = 0;
    int n = 0;
    for (; n < kBatchTensors && from < to; ++from) {
      const int64_t count = a.counts[from];
      if (count == 0) continue;
      b.in[n] = a.in[from];
      b.out[n] = a.out ? a.out[from] : nullptr;
      b.count[n] = count;
      b.type[n] = (uint8_t)(a.types[from] | (a.out_types ? a.out_types[from] : a.types[from]) << 4);
      b.first[n++] = tiles;
      tiles += (uint32_t)((count + kTile - 1) / kTile);
    }
    for (int i = n; i <= kBatchTensors; ++i) b.first[i] = tiles;
    if (n == 0) break;
    hipError_t e = go(b);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The squares' parts; their number goes to *parts.
hipError_t squares(const TensorListArgs& a, void* work, int* parts, hipStream_t s) {
  int n = 0;
  hipError_t e = each_batch(a, 0, a.counted, [&](const TensorBatch& b) {
    const unsigned grid = batch_grid(b);
    k_squares<<<grid, kThreads, 0, s>>>(b, parts_at(work) + n);
    n += (int)grid;
    return hipGetLastError();
  });
  *parts = n;
  return e;
}

template <int DT, int AC>
hipError_t fold_go(const FoldArgs& a, ClipRule r, void* work, hipStream_t s) {
  const int64_t tiles = (a.n + kFoldTile - 1) / kFoldTile;
  r.parts = (int)fold_clip_parts(a.n);
  r.part = parts_at(work);
  k_fold_squares<DT, AC><<<(unsigned)r.parts, kThreads, 0, s>>>(a, parts_at(work));
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = rule_for(&r, work, s);
  if (e != hipSuccess) return e;
  k_spread<DT, AC><<<(unsigned)std::min<int64_t>(tiles, kMaxGrid), kThreads, 0, s>>>(a, r);
  return hipGetLastError();
}

template <int DT>
hipError_t fold_access(const FoldArgs& a, const ClipRule& r, int access, void* work, hipStream_t s) {
  if (access == kStreamRows) return fold_go<DT, kStreamRows>(a, r, work, s);
  if (access == kAlignedRows) return fold_go<DT, kAlignedRows>(a, r, work, s);
  return fold_go<DT, kOddRows>(a, r, work, s);
}

}  // namespace

int64_t grad_norm_bytes(int64_t n) {
  const int64_t batches = (n + kBatchTensors - 1) / kBatchTensors;
  return 16 + batches * kSquaresGrid * (int64_t)sizeof(double);
}

// One part for each of the first pass's workgroups, which take tiles in a stride where there
// are more.
int64_t fold_clip_parts(int64_t n) { return std::min<int64_t>((n + kFoldTile - 1) / kFoldTile, kFoldGrid); }
int64_t fold_clip_bytes(int64_t n) { return 16 + fold_clip_parts(n) * (int64_t)sizeof(double); }

hipError_t launch_grad_norm(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s) {
  hipError_t e = squares(a, work, &r.parts, s);
  r.part = parts_at(work);
  return e != hipSuccess ? e : finish(r, nullptr, s);
}

hipError_t launch_grad_clip(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s) {
  hipError_t e = squares(a, work, &r.parts, s);
  r.part = parts_at(work);
  if (e == hipSuccess) e = rule_for(&r, work, s);
  if (e != hipSuccess) return e;
  bool any = false;
  e = each_batch(a, 0, a.n, [&](const TensorBatch& b) {
    any = true;
    k_scale<<<batch_grid(b), kThreads, 0, s>>>(b, r);
    return hipGetLastError();
  });
  // without an element to scale, the norm of none
  return e != hipSuccess || any ? e : finish(r, nullptr, s);
}

hipError_t launch_fold_clip(const FoldArgs& a, int dtype, const ClipRule& r, int access, void* work, hipStream_t s) {
  if (a.n == 0) {
    ClipRule none = r;
    none.parts = 0;
    none.part = nullptr;
    return finish(none, nullptr, s);
  }
  if (dtype == 1) return fold_access<1>(a, r, access, work, s);
  if (dtype == 2) return fold_access<2>(a, r, access, work, s);
  return fold_access<3>(a, r, access, work, s);
}

}  // namespace ra
