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
//
// All of it is bound by memory, and each pass moves 1.00 times the bytes that it has to
// (HBM counters).  What decides the rate is how the accesses go past the caches, how much a thread
// has under way, and whether streams are read and written in turns.  Measured on MI355X, where a copy of
// 8 GiB runs at 6.55 TB/s and reads alone at 7.0:
//   norm of 1.2 10^9 bfloat16 gradients, 219 tensors    345 us, 6.9 TB/s
//   the same clipped into other buffers                 1128 us: the norm, and 775 us at 6.1 TB/s
//   8 x 256 MiB float32 averaged, clipped, to all 8     784 us: 393 us for 2.4 GB, 9 streams at equal offsets,
//                                                       332 us for 2.4 GB of which the caches have some
//   9 x 1,000,003 bfloat16 summed, clipped, to all 9    14.2 us: 5.5 and 7.0 in two launches
//   norm of 75 tensors, 24 MB in the caches             5.4 us and 2.4 for the sum of the parts
#include "ra_rows.h"

namespace ra {
namespace {

constexpr int kThreads = 256;

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
// float32's end (and hi 2^96 times as large: g hi stays below 2^124), or 2^-126 where that
// would be, too (and g hi stays below 2^32).  Such factors belong to gradients near float32's
// other end, which they bring back into its range.
struct Factor {
  float norm, hi, lo;
};
__device__ __forceinline__ float times(float g, const Factor& f) { return g * f.hi * f.lo; }
__device__ __forceinline__ bool is_one(const Factor& f) { return f.hi == 1.0f && f.lo == 1.0f; }

__device__ __forceinline__ Factor factor_of(double total, const ClipRule& r) {
  const double norm = (double)r.scale * __builtin_sqrt(total);
  const double q = (double)r.max_norm / (norm + 1e-6);
  const double c = (double)r.scale * (q > 1.0 ? 1.0 : q);      // NaN stays
  if (c < 0x1p-222) return {(float)norm, (float)(c * 0x1p126), 0x1p-126f};
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

// ---------------------------------------------------------------- elements

// A lane moves N consecutive elements of each array at a time, at most 16 bytes, so that a wave's
// accesses are whole lines: 8 elements, or 4 where one of the arrays is float32.  (A lane that
// moved 8 float32, as two accesses 16 bytes apart, wrote half lines: the pass that writes 8 x 256 MiB
// took 889 us, and 497 with 16 bytes a lane, before what makes it 332 now.)  Arrays start on any
// boundary of their elements, for which gfx950 issues the same accesses.  Where a run of elements ends
// inside a lane's, those are moved back to end there, and the first `lo` of them, which are another
// lane's, are loaded and not used.  Runs shorter than N go a lane to an element.
template <int N> struct Some {
  float x[N];
};
struct Own {
  int at, lo;         // elements [at + lo, at + N) are the lane's
};
template <int N>
__device__ __forceinline__ Own own_of(int j, int len) {
  const int at = min(j * N, len - N);
  return {at, j * N - at};
}

typedef uint32_t u32x2_by2 __attribute__((ext_vector_type(2), aligned(2)));

// What a lane's N elements are in registers and in memory.
template <int DT, int N> struct Word { typedef u32x2 R; typedef u32x2_by2 M; };
template <> struct Word<1, 4> { typedef u32x4 R; typedef u32x4_by4 M; };
template <int DT> struct Word<DT, 8> { typedef u32x4 R; typedef u32x4_by2 M; };

// NT: past the caches.
template <int DT, int N, bool NT>
__device__ __forceinline__ typename Word<DT, N>::R load_word(const void* p, int64_t i) {
  typedef typename Word<DT, N>::M M;
  const M* q = reinterpret_cast<const M*>(static_cast<const char*>(p) + i * ElemSize<DT>::value);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  else return *q;
}

template <int DT, int N>
__device__ __forceinline__ Some<N> values(const typename Word<DT, N>::R w) {
  Some<N> s;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (DT == 1) s.x[k] = __uint_as_float(w[k]);
    else if constexpr (DT == 2) s.x[k] = __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    else s.x[k] = f16_to_f32((uint16_t)(w[k / 2] >> (k % 2 * 16)));
  }
  return s;
}

// Rounded to nearest, ties to even.
template <int DT, int N>
__device__ __forceinline__ typename Word<DT, N>::R word_of(const Some<N>& s) {
  typename Word<DT, N>::R w;
  if constexpr (DT == 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __float_as_uint(s.x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      const f32x2 two = {s.x[2 * k], s.x[2 * k + 1]};
      if constexpr (DT == 2) w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
      else w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
    }
  }
  return w;
}

// The lane's elements of the run at element `run` of p.
template <int DT, int N, bool NT>
__device__ __forceinline__ void store_own(void* p, int64_t run, const Own& o, const typename Word<DT, N>::R w) {
  typedef typename Elem<DT>::S S;
  S* q = static_cast<S*>(p) + run + o.at;
  if (o.lo == 0) {
    typedef typename Word<DT, N>::M M;
    if constexpr (NT) __builtin_nontemporal_store((M)w, reinterpret_cast<M*>(q));
    else *reinterpret_cast<M*>(q) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k < o.lo) continue;
    if constexpr (DT == 1) q[k] = w[k];
    else q[k] = (S)(w[k / 2] >> (k % 2 * 16));
  }
}

// One element.
template <int DT>
__device__ __forceinline__ float value_of(typename Elem<DT>::S x) {
  if constexpr (DT == 1) return __uint_as_float(x);
  else return Elem<DT>::to_w(x);
}
template <int DT>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  return value_of<DT>(static_cast<const typename Elem<DT>::S*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::S one_of(float x) {
  if constexpr (DT == 1) return __float_as_uint(x);
  else return Elem<DT>::from_w(x);
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, int64_t i, float x) {
  static_cast<typename Elem<DT>::S*>(p)[i] = one_of<DT>(x);
}

template <int N>
__device__ __forceinline__ void add_squares(double* acc, const Some<N>& s, int lo) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const double x = k >= lo ? (double)s.x[k] : 0.0;
    acc[k % 4] = __builtin_fma(x, x, acc[k % 4]);
  }
}

// ---------------------------------------------------------------- many tensors

// The tensors of a launch, cut into tiles, which go one tensor's behind the other's.  A launch's
// arguments have to stay within 4 KiB, with the 256 bytes that the compiler adds of its own (the
// grid's size among them).
template <int N, bool OUT> struct Batch {
  const void* in[N];
  void* out[OUT ? N : 1];
  uint32_t first[N + 1];    // tiles before each tensor's; from the last one on, all tiles
  // Elements of a tensor's last tile, less 1, and its Kind.  32 bits, of which 16 would do: where an
  // index counts by 2 bytes in one array and by 4 in another, the compiler shares sums of it between
  // their addresses and splits one into parts that are no multiples of 4, of which a scalar load
  // drops the low bits.
  uint32_t last[N];
};
typedef Batch<232, false> Read;
typedef Batch<156, true> Scale;
enum Kind { kHalf = 1 << 13, kFull = 1 << 14, kWiden = 1 << 15 };   // float16 (neither: bfloat16), float32; out is float32
constexpr int kArgsMost = 4096 - 256;
static_assert(sizeof(Read) + sizeof(double*) <= kArgsMost && sizeof(Scale) + sizeof(ClipRule) <= kArgsMost, "arguments");

template <int N, bool OUT> constexpr int tensors(const Batch<N, OUT>&) { return N; }

// Accesses of a thread to a tile.  What the norm reads: 32 elements, all under way together.  The pass
// that scales beyond the caches has one access: read and written streams go best that way (2.4 GB into
// 2.4 GB: 742 us, two accesses 820, four 833), in workgroups that take a tile each (884 in ones that stay).
// Where the caches serve it, four, in workgroups that stay (44 MB into 88 MB: 24.6 us, one access 27).
template <bool NT> constexpr int kScaleLoads = NT ? 1 : 4;
constexpr int kReadTile = kThreads * 32;
template <bool OUT>
__host__ __device__ constexpr int tile_elements(int kind, bool stream) {
  return OUT ? kThreads * (stream ? kScaleLoads<true> : kScaleLoads<false>) * (kind & (kFull | kWiden) ? 4 : 8) : kReadTile;
}
static_assert(kReadTile <= kHalf, "a last tile's elements have 13 bits");

// The tensor that has tile t: as many end before it.  One round trip for the whole list, which in a
// small launch no cache holds yet.  The whole wave has to be active.
template <int N, bool OUT>
__device__ __forceinline__ int tensor_of(const Batch<N, OUT>& b, uint32_t t) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; i += 64) {
    const int k = i + threadIdx.x % 64;
    n += __builtin_popcountll(__ballot(k < N && b.first[min(k, N - 1) + 1] <= t));
  }
  return __builtin_amdgcn_readfirstlane(n);
}

// The same by halving: eight scalar loads, one behind the other, from the scalar cache.  For launches
// of many workgroups that look up one tile each (2.4 GB into 2.4 GB: 775 us).
template <int N, bool OUT>
__device__ __forceinline__ int tensor_by_halving(const Batch<N, OUT>& b, uint32_t t) {
  int lo = 0;
#pragma unroll
  for (int step = 128; step > 0; step /= 2)
    if (lo + step < N && b.first[lo + step] <= t) lo += step;
  return lo;
}

// Tile t of tensor i.
struct Tile {
  int64_t at;       // its first element
  int len, kind;
};
template <bool NT, int N, bool OUT>
__device__ __forceinline__ Tile tile_of(const Batch<N, OUT>& b, int i, uint32_t t) {
  const int last = (int)b.last[i], kind = last & ~(kHalf - 1), all = tile_elements<OUT>(kind, NT);
  return {(int64_t)(t - b.first[i]) * all, t + 1 == b.first[i + 1] ? (last & (kHalf - 1)) + 1 : all, kind};
}

template <int DT, bool NT>
__device__ __forceinline__ void tile_squares(double* acc, const void* p, const Tile& tile) {
  constexpr int N = DT == 1 ? 4 : 8;
  const char* x = static_cast<const char*>(p) + tile.at * ElemSize<DT>::value;
  const int len = tile.len;
  if (len < N) {
    const double g = (int)threadIdx.x < len ? (double)load_one<DT>(x, threadIdx.x) : 0.0;
    acc[0] = __builtin_fma(g, g, acc[0]);
    return;
  }
  // All loads go out before the first is used.  Lanes behind the end read what the last one does, and
  // own none of it.
  constexpr int kLoads = kReadTile / kThreads / N;
  typename Word<DT, N>::R t[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) t[u] = load_word<DT, N, NT>(x, own_of<N>(threadIdx.x + u * kThreads, len).at);
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    if (len == kReadTile) add_squares<N>(acc, values<DT, N>(t[u]), 0);
    else add_squares<N>(acc, values<DT, N>(t[u]), own_of<N>(threadIdx.x + u * kThreads, len).lo);
  }
}

// Workgroups take the tiles in turn, whichever tensors they are of, so that all of them
// together go through the tensors from front to back.
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_squares(Read b, double* part) {
  __shared__ double lds[kThreads / 64];
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  uint32_t t = blockIdx.x;
  for (int i = tensor_of(b, t); t < b.first[tensors(b)]; t += gridDim.x) {
    while (t >= b.first[i + 1]) ++i;
    const Tile tile = tile_of<NT>(b, i, t);
    if (tile.kind & kFull) tile_squares<1, NT>(acc, b.in[i], tile);
    else if (tile.kind & kHalf) tile_squares<3, NT>(acc, b.in[i], tile);
    else tile_squares<2, NT>(acc, b.in[i], tile);
  }
  const double sum = block_sum64((acc[0] + acc[1]) + (acc[2] + acc[3]), lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <int DT, int OUT, bool NT>
__device__ __forceinline__ void tile_scale(const void* from, void* to, const Tile& tile, const Factor& c) {
  constexpr int N = DT == 1 || OUT == 1 ? 4 : 8;
  const char* x = static_cast<const char*>(from) + tile.at * ElemSize<DT>::value;
  char* y = static_cast<char*>(to) + tile.at * ElemSize<OUT>::value;
  const int len = tile.len;
  if (len < N) {
    if ((int)threadIdx.x < len) store_one<OUT>(y, threadIdx.x, times(load_one<DT>(x, threadIdx.x), c));
    return;
  }
  typename Word<DT, N>::R w[kScaleLoads<NT>];
#pragma unroll
  for (int u = 0; u < kScaleLoads<NT>; ++u) w[u] = load_word<DT, N, NT>(x, own_of<N>(threadIdx.x + u * kThreads, len).at);
#pragma unroll
  for (int u = 0; u < kScaleLoads<NT>; ++u) {
    const Own o = own_of<N>(threadIdx.x + u * kThreads, len);
    if (o.lo >= N) continue;
    Some<N> s = values<DT, N>(w[u]);
#pragma unroll
    for (int k = 0; k < N; ++k) s.x[k] = times(s.x[k], c);
    store_own<OUT, N, NT>(y, 0, o, word_of<OUT, N>(s));
  }
}

// A factor of one leaves what is scaled in place as it is.  From the last tile to the first:
// what the pass before read last may still be cached.
template <bool NT>
__global__ __launch_bounds__(kThreads) void k_scale(Scale b, ClipRule r) {
  __shared__ double lds[kThreads / 64];
  const Factor c = factor(r, lds);
  uint32_t n = b.first[tensors(b)] - blockIdx.x;           // tiles up to the workgroup's
  for (int i = NT ? tensor_by_halving(b, n - 1) : tensor_of(b, n - 1);; n -= gridDim.x) {
    while (n - 1 < b.first[i]) --i;
    if (!is_one(c) || b.in[i] != b.out[i]) {
      const Tile tile = tile_of<NT>(b, i, n - 1);
      if (tile.kind & kFull) tile_scale<1, 1, NT>(b.in[i], b.out[i], tile, c);
      else if (tile.kind == 0) tile_scale<2, 2, NT>(b.in[i], b.out[i], tile, c);
      else if (tile.kind == kWiden) tile_scale<2, 1, NT>(b.in[i], b.out[i], tile, c);
      else if (tile.kind == kHalf) tile_scale<3, 3, NT>(b.in[i], b.out[i], tile, c);
      else tile_scale<3, 1, NT>(b.in[i], b.out[i], tile, c);
    }
    if (n <= gridDim.x) return;
  }
}

// ---------------------------------------------------------------- ranks

// A workgroup's tile: kRuns<NT> times what its lanes move at a time.
template <int DT> constexpr int kLane = DT == 1 ? 4 : 8;
template <bool NT> constexpr int kRuns = NT ? 2 : 1;
template <int DT, bool NT> constexpr int kFoldTile = kThreads * kLane<DT> * kRuns<NT>;

// The sum over the ranks, in rank order from 0, of each of the lane's runs; up to eight ranks'
// loads are in flight together.
template <int DT, int N, int RUNS, bool NT>
__device__ __forceinline__ void fold_words(Some<N>* s, const RankPtrs& P, int p, int64_t at, const Own* o) {
  constexpr int kBatch = 8;
#pragma unroll
  for (int u = 0; u < RUNS; ++u) s[u] = Some<N>{};
  auto add = [&](int u, const typename Word<DT, N>::R w) {
    const Some<N> v = values<DT, N>(w);
#pragma unroll
    for (int k = 0; k < N; ++k) s[u].x[k] += v.x[k];
  };
  int r = 0;
  for (; r + kBatch <= p; r += kBatch) {
    typename Word<DT, N>::R t[kBatch][RUNS];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int u = 0; u < RUNS; ++u) t[b][u] = load_word<DT, N, NT>(P.b[r + b], at + o[u].at);
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int u = 0; u < RUNS; ++u) add(u, t[b][u]);
  }
  for (; r + 2 <= p; r += 2) {
    typename Word<DT, N>::R t[2][RUNS];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < RUNS; ++u) t[b][u] = load_word<DT, N, NT>(P.b[r + b], at + o[u].at);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < RUNS; ++u) add(u, t[b][u]);
  }
  if (r < p) {
#pragma unroll
    for (int u = 0; u < RUNS; ++u) add(u, load_word<DT, N, NT>(P.b[r], at + o[u].at));
  }
}

// The sum (mean) over the ranks, rounded to the buffers' type, into the first output, and the
// squares of what was rounded.  An output may be one of the buffers: an element is read from all of
// them by the thread that writes it.  The sum is written to the caches, for the next pass.
template <int DT, bool NT>
__global__ __launch_bounds__(kThreads) void k_fold_squares(FoldArgs a, double* part) {
  constexpr int N = kLane<DT>, RUNS = kRuns<NT>, kTile = kFoldTile<DT, NT>;
  __shared__ double lds[kThreads / 64];
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int64_t step = (int64_t)gridDim.x * kTile;
  for (int64_t at = (int64_t)blockIdx.x * kTile; at < a.n; at += step) {
    const int len = (int)min((int64_t)kTile, a.n - at);
    if (len < N) {
      if ((int)threadIdx.x >= len) continue;
      float x = 0.0f;
      for (int r = 0; r < a.p; ++r) x += load_one<DT>(a.in.b[r], at + threadIdx.x);
      if (a.mean) x = x / (float)a.p;
      store_one<DT>(a.out.b[0], at + threadIdx.x, x);
      const double g = value_of<DT>(one_of<DT>(x));
      acc[0] = __builtin_fma(g, g, acc[0]);
      continue;
    }
    Own o[RUNS];
    Some<N> s[RUNS];
#pragma unroll
    for (int u = 0; u < RUNS; ++u) o[u] = own_of<N>(threadIdx.x + u * kThreads, len);
    fold_words<DT, N, RUNS, NT>(s, a.in, a.p, at, o);
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      if (o[u].lo >= N) continue;
      if (a.mean) {
#pragma unroll
        for (int k = 0; k < N; ++k) s[u].x[k] = s[u].x[k] / (float)a.p;
      }
      const typename Word<DT, N>::R w = word_of<DT, N>(s[u]);
      store_own<DT, N, false>(a.out.b[0], at, o[u], w);
      add_squares<N>(acc, values<DT, N>(w), o[u].lo);
    }
  }
  const double sum = block_sum64((acc[0] + acc[1]) + (acc[2] + acc[3]), lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// What k_fold_squares left in the first output, times the factor, to all of them; from the last
// tile to the first, since what was written last is still cached.
template <int DT, bool NT>
__global__ __launch_bounds__(kThreads) void k_spread(FoldArgs a, ClipRule r) {
  constexpr int N = kLane<DT>, kTile = kThreads * N;
  __shared__ double lds[kThreads / 64];
  const int64_t last = (a.n + kTile - 1) / kTile - 1 - blockIdx.x;
  Factor c;
  for (int64_t t = last; t >= 0; t -= gridDim.x) {
    const int64_t at = t * kTile;
    const int len = (int)min((int64_t)kTile, a.n - at);
    if (len < N) {            // the very last tile: the workgroup's first
      c = factor(r, lds);
      if ((int)threadIdx.x >= len) continue;
      const float x = times(load_one<DT>(a.out.b[0], at + threadIdx.x), c);
      for (int q = 0; q < a.n_out; ++q) store_one<DT>(a.out.b[q], at + threadIdx.x, x);
      continue;
    }
    const Own o = own_of<N>(threadIdx.x, len);
    const typename Word<DT, N>::R w = load_word<DT, N, false>(a.out.b[0], at + o.at);
    if (t == last) c = factor(r, lds);     // while the first load is under way
    if (o.lo >= N) continue;
    Some<N> s = values<DT, N>(w);
#pragma unroll
    for (int k = 0; k < N; ++k) s.x[k] = times(s.x[k], c);
    const typename Word<DT, N>::R y = word_of<DT, N>(s);
    for (int q = 0; q < a.n_out; ++q) store_own<DT, N, NT>(a.out.b[q], at, o, y);
  }
}

// ---------------------------------------------------------------- launches

// Workgroups of the pass over a batch of tensors that sums, and of the first pass over the ranks'
// buffers.  Constants, so that the order of the sums does not depend on the GPU.
constexpr int kListGrid = 1024;
constexpr unsigned kScaleGrid = 2048;     // of the pass that scales, where the caches serve it
constexpr int kFoldGrid = 1 << 18;

// Where k_finish leaves the factor: in front of the parts.
float* factor_at(void* work) { return static_cast<float*>(work); }
double* parts_at(void* work) { return static_cast<double*>(work) + 2; }

hipError_t finish(const ClipRule& r, float* to, hipStream_t s) {
  k_finish<<<1, 1024, 0, s>>>(r, to);
  return hipGetLastError();
}

// Parts or the factor, for the kernels that scale: few parts are summed by every one of few workgroups,
// more by a launch of their own.
constexpr int64_t kSumMost = 2048;
hipError_t rule_for(ClipRule* r, int64_t workgroups, void* work, hipStream_t s) {
  if (r->parts <= kSumMost && workgroups <= kSumMost) return hipSuccess;
  hipError_t e = finish(*r, factor_at(work), s);
  r->factor = factor_at(work);
  return e;
}

// The tiles of a tensor.
template <bool OUT>
int64_t tiles_of(const TensorListArgs& a, int64_t i, int* kind) {
  const int type = a.types[i], out = OUT && a.out_types ? a.out_types[i] : type;
  *kind = (type == 1 ? kFull : type == 3 ? kHalf : 0) | (out != type ? kWiden : 0);
  const int all = tile_elements<OUT>(*kind, a.stream);
  return (a.counts[i] + all - 1) / all;
}

// Runs go(batch, tiles) on the first n tensors of a list, as many of them at a time as a launch takes.
template <int N, bool OUT, typename F>
hipError_t each_batch(const TensorListArgs& a, int64_t n, F go) {
  Batch<N, OUT> b;
  for (int64_t i = 0; i < n;) {
    uint32_t tiles = 0;
    int m = 0;
    for (; m < N && i < n; ++i) {
      if (a.counts[i] == 0) continue;
      int kind;
      const int64_t mine = tiles_of<OUT>(a, i, &kind);
      b.in[m] = a.in[i];
      if (OUT) b.out[m] = a.out[i];
      b.last[m] = (uint32_t)((a.counts[i] - 1) % tile_elements<OUT>(kind, a.stream) | kind);
      b.first[m++] = tiles;
      tiles += (uint32_t)mine;
    }
    if (m == 0) break;
    for (; m <= N; ++m) b.first[m] = tiles;
    hipError_t e = go(b, tiles);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The squares' parts; their number goes to *parts.
hipError_t squares(const TensorListArgs& a, void* work, int* parts, hipStream_t s) {
  int n = 0;
  hipError_t e = each_batch<232, false>(a, a.counted, [&](const Read& b, uint32_t tiles) {
    const unsigned grid = std::min<unsigned>(tiles, kListGrid);
    if (a.stream) k_squares<true><<<grid, kThreads, 0, s>>>(b, parts_at(work) + n);
    else k_squares<false><<<grid, kThreads, 0, s>>>(b, parts_at(work) + n);
    n += (int)grid;
    return hipGetLastError();
  });
  *parts = n;
  return e;
}

template <int DT, bool NT>
hipError_t fold_go(const FoldArgs& a, ClipRule r, void* work, hipStream_t s) {
  const int64_t tiles = (a.n + kFoldTile<DT, NT> - 1) / kFoldTile<DT, NT>;
  const int64_t spread = (a.n + kThreads * kLane<DT> - 1) / (kThreads * kLane<DT>);
  r.parts = (int)std::min<int64_t>(tiles, kFoldGrid);
  r.part = parts_at(work);
  k_fold_squares<DT, NT><<<(unsigned)r.parts, kThreads, 0, s>>>(a, parts_at(work));
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = rule_for(&r, spread, work, s);
  if (e != hipSuccess) return e;
  k_spread<DT, NT><<<(unsigned)std::min<int64_t>(spread, kMaxGrid), kThreads, 0, s>>>(a, r);
  return hipGetLastError();
}

template <int DT>
hipError_t fold_access(const FoldArgs& a, const ClipRule& r, bool stream, void* work, hipStream_t s) {
  return stream ? fold_go<DT, true>(a, r, work, s) : fold_go<DT, false>(a, r, work, s);
}

}  // namespace

int64_t grad_norm_bytes(int64_t n) {
  const int64_t batches = (n + tensors(Read{}) - 1) / tensors(Read{});
  return 16 + batches * kListGrid * (int64_t)sizeof(double);
}

// A part for each of the first pass's workgroups (float32's tiles are the smallest), which take tiles
// in a stride where there are more of them.
int64_t fold_clip_bytes(int64_t n) {
  constexpr int kLeast = kFoldTile<1, false>;
  return 16 + std::min<int64_t>((n + kLeast - 1) / kLeast, kFoldGrid) * (int64_t)sizeof(double);
}

hipError_t launch_grad_norm(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s) {
  hipError_t e = squares(a, work, &r.parts, s);
  r.part = parts_at(work);
  return e != hipSuccess ? e : finish(r, nullptr, s);
}

hipError_t launch_grad_clip(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s) {
  hipError_t e = squares(a, work, &r.parts, s);
  r.part = parts_at(work);
  int64_t tiles = 0;
  int kind;
  for (int64_t i = 0; i < a.n; ++i) tiles += tiles_of<true>(a, i, &kind);
  if (e == hipSuccess) e = rule_for(&r, a.stream ? tiles : kScaleGrid, work, s);
  if (e == hipSuccess)
    e = each_batch<156, true>(a, a.n, [&](const Scale& b, uint32_t tiles) {
      if (a.stream) k_scale<true><<<std::min<uint32_t>(tiles, kMaxGrid), kThreads, 0, s>>>(b, r);
      else k_scale<false><<<std::min<uint32_t>(tiles, kScaleGrid), kThreads, 0, s>>>(b, r);
      return hipGetLastError();
    });
  // without an element to scale, the norm of none
  return e != hipSuccess || tiles > 0 ? e : finish(r, nullptr, s);
}

hipError_t launch_fold_clip(const FoldArgs& a, int dtype, const ClipRule& r, bool stream, void* work, hipStream_t s) {
  if (a.n == 0) {
    ClipRule none = r;
    none.parts = 0;
    none.part = nullptr;
    return finish(none, nullptr, s);
  }
  if (dtype == 1) return fold_access<1>(a, r, stream, work, s);
  if (dtype == 2) return fold_access<2>(a, r, stream, work, s);
  return fold_access<3>(a, r, stream, work, s);
}

}  // namespace ra
