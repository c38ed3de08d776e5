// ra_logprob.hip -- log probabilities of given tokens, the entropy and the best
// alternatives, from logits whose vocabulary is cut over the ranks; and the gradient of
// the first two.
//
//   y_j = s x_j,  m = max_j y_j,  z = sum_j exp(y_j - m),  w = sum_j exp(y_j - m) (y_j - m)
//   lse = m + ln z,  ln p_j = y_j - m - ln z,  H = ln z - w / z
//   dx_j = s (a [j = id] - p_j (a + b (ln p_j + H))),   a, b: gradients of ln p_id and of H
//
// One pass over the logits.  Like the cross entropy's (ra_xent.hip) it takes 2^(x s log2 e - c)
// with one fused multiply-add and the hardware's exponential, c = m log2 e rounded, and
// keeps what that rounding leaves: in the end z and w are brought to the true m.  w is
// kept in units of ln 2.  A row where that leaves float32 (only -inf or the type's lowest
// value, NaN, +inf, logits beyond 10^7) is done again with m subtracted first.
//
// The k best columns by (logit descending, column ascending): in the same pass each thread
// keeps the largest logit of every 32 that it reads.  The k-th largest of the maxima of 128
// sets of threads bounds the k-th best logit from below, and only the groups whose maximum reaches
// that bound are read again, some k of a row's thousands, a thread to each unit of eight columns.
// The elements at or above the bound are put in order by counting, for each, the ones in front of it.
// Where too many reach the bound (ties), it is raised first, by halving the interval of (logit, column).
// Few rows are cut into parts, a workgroup each, whose sums and best columns a second launch joins.
//
// Large calls are bound by memory, and by the search for the best columns at the end of each row.  Measured on
// MI355X (GPU time; a copy of 8 GiB runs at 6.55 TB/s, reads alone at 7.0):
//   4096 x 131072 bfloat16, 8 ranks     158 to 179 us from card to card and from buffers to buffers, 6.0 to 6.8 TB/s;
//                                       top 20 172 to 185, top 64 197
//   the same with three columns left in every row, or all of them equal, top 20   5.9 ms: 22 halvings and a reading
//                                       of the row for each; 16 x 128000 262 us, 1 x 32000 300
//   16384 x 131072                      641 us, 6.7 TB/s
//   1003 x 50017 float32, 9 ranks       35.5 us, 5.7 TB/s; top 64 45 to 46
//   16 x 128000 bfloat16, top 20        12.4 us in two launches
//   1 x 32000 float16, top 5            9.3 us in one
//   64 x 4096 bfloat16, top 5           7.0 us, of which the search is 3, half of that the second reading
//   gradient of 4096 x 131072           348 us, 6.2 TB/s
// It reads 1.05 times the logits' bytes with 20 alternatives of 131072 bfloat16 columns, 1.28 times with 64
// of 50017 float32 ones (HBM counters): the groups that are read again, a line for each unit.  The gradient reads
// and writes 1.00 times what it has to.
#include "ra_vocab.h"

namespace ra {
namespace {

constexpr float kNone = -1e38f;      // c of no logit
constexpr float kFloor = -200.0f;    // 2^-200 is 0: a product with it is 0, where -inf would make NaN
constexpr int kMore = 4;             // units of a group, in flight together

// A row, or what one wave or workgroup has of it.
struct Stat {
  float m, c, z, w;     // the largest logit; c near m s log2 e; z, w relative to 2^c
};
__device__ __forceinline__ Stat none() { return {-INFINITY, kNone, 0.0f, 0.0f}; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(a) : "v"(a), "v"(b), "v"(c));
  return a;
}

// Joins a unit; `top` becomes the largest of itself and the unit's logits.  m and c are the wave's: after
// a row's first units a larger m is rare, and c costs a comparison.  NaN is passed over by the maxima,
// and makes z NaN.
template <int DT>
__device__ __forceinline__ void take(Stat& t, float& top, const Unit<DT>& u, float s2) {
  float x[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) x[i] = unit_get<DT>(u, i);
  const float most = max3(max3(max3(x[0], x[1], x[2]), x[3], x[4]), max3(x[5], x[6], x[7]), -INFINITY);
  top = __builtin_fmaxf(top, most);
  if (__any(most > t.m)) {
    t.m = wave_max(__builtin_fmaxf(most, t.m));
    const float c = __builtin_fmaxf(kNone, t.m * s2), d = t.c - c, r = exp2_of(d);
    t.w = r * __builtin_fmaf(d, t.z, t.w);
    t.z *= r;
    t.c = c;
  }
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const float y = __builtin_fmaf(x[i], s2, -t.c), e = exp2_of(y);
    t.z += e;
    t.w = __builtin_fmaf(e, __builtin_fmaxf(y, kFloor), t.w);
  }
}

// Over 16 neighbouring lanes: the same c, then the sums.
__device__ __forceinline__ Stat row_join(Stat t) {
  const float c = row_max(t.c), d = t.c - c, r = exp2_of(d);
  return {row_max(t.m), c, row_sum(r * t.z), row_sum(r * __builtin_fmaf(d, t.z, t.w))};
}
__device__ __forceinline__ Stat lane_stat(const Stat& t, int lane) {
  return {lane_value(t.m, lane), lane_value(t.c, lane), lane_value(t.z, lane), lane_value(t.w, lane)};
}

// Over the workgroup of at most 16 waves, in each of which m and c are the same; every lane gets it.
// `lds` is free again at the next barrier.
__device__ __forceinline__ Stat block_join(Stat t, Stat* lds, int waves) {
  t.z = wave_sum(t.z);
  t.w = wave_sum(t.w);
  const int lane = threadIdx.x % 64;
  if (lane == 0) lds[threadIdx.x / 64] = t;
  __syncthreads();
  t = row_join(lane % 16 < waves ? lds[lane % 16] : none());
  return lane_stat(t, 0);
}

// Relative to the true m, as y - m is: c was rounded.
__device__ __forceinline__ bool settle(Stat& t, float s2) {
  const float d = __builtin_fmaf(t.m, s2, -t.c), r = exp2_of(-d);
  const bool good = t.z > 0x1p-100f && t.z < 0x1p120f && __builtin_fabsf(d) < 0.5f && __builtin_fabsf(t.w) < 1e30f;
  t.w = r * __builtin_fmaf(-d, t.z, t.w);
  t.z *= r;
  return good;
}

// s (x - m) for x <= m.  The difference of logits near both of float32's ends is beyond it, s times it
// perhaps not: those are multiplied first, |m s| being at most s (m - x) then.
__device__ __forceinline__ float below(float x, float m, float s) {
  const float d = x - m;
  return d == -INFINITY && x != -INFINITY ? __builtin_fmaf(x, s, -(m * s)) : d * s;
}

// The same as exponents of 2, s log2 e (x - m).  The product s log2 e leaves float32 for an s beyond
// 2.3 10^38 (0 times it would be NaN, and all rows are settled by the difference then): s goes first there.
struct Exponent {
  float s, more;
  __device__ __forceinline__ float operator()(float x, float m) const { return below(x, m, s) * more; }
};
__device__ __forceinline__ Exponent exponent_of(float scale) {
  const float s2 = scale * kLog2e;
  return s2 < INFINITY ? Exponent{s2, 1.0f} : Exponent{scale, kLog2e};
}

// The chunks of a workgroup: lo, lo + step, ... below hi, its waves taking one each in turn.  The parts of
// a row take turns, too: the last chunks, which are short where pieces end in them, go to many.
struct Range {
  int lo, hi, step;
};
__device__ __forceinline__ Range range_of(const VocabArgs& a, int part) { return {part, a.total, a.splits}; }

// The statistics of a range with the largest logit subtracted first, by the workgroup.
template <int DT, int MODE>
__device__ __forceinline__ Stat plain_stat(const LogpArgs& a, int64_t row, Range g, float* lds) {
  const Exponent exponent = exponent_of(a.scale);
  const int w = wave_id(), waves = blockDim.x / 64;
  float m = -INFINITY;
  for (int q = g.lo + w * g.step; q < g.hi; q += waves * g.step) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, waves * g.step, g.hi);
#pragma unroll
    for (int i = 0; i < kU; ++i) m = __builtin_fmaxf(m, unit_get<DT>(u[0], i));
  }
  m = wave_max(m);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = m;
  __syncthreads();
  const int lane = threadIdx.x % 16;
  m = lane_value(row_max(lane < waves ? lds[lane] : -INFINITY), 0);
  __syncthreads();
  const float at = m == -INFINITY ? 0.0f : m;
  float z = 0.0f, v = 0.0f;
  for (int q = g.lo + w * g.step; q < g.hi; q += waves * g.step) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, waves * g.step, g.hi);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const float y = exponent(unit_get<DT>(u[0], i), at), e = exp2_of(y);
      z += e;
      v = __builtin_fmaf(e, __builtin_fmaxf(y, kFloor), v);
    }
  }
  z = block_sum(z, lds, waves);
  __syncthreads();
  v = block_sum(v, lds, waves);
  __syncthreads();
  return {m, 0.0f, z, v};
}

// ---------------------------------------------------------------- the best columns

// Logits as whole numbers of the same order: NaN the largest, -0 like +0; 0 is none's.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) != 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key == 0xffffffffu ? 0x7fc00000u : key ^ ((key >> 31) != 0 ? 0x80000000u : 0xffffffffu));
}
// ... with the column, of which lower ones come first.
__device__ __forceinline__ uint64_t place_of(uint32_t key, int col) { return (uint64_t)key << 32 | ~(uint32_t)col; }

constexpr int kCap = 1024;      // columns that are kept
constexpr int kOrder = 256;     // ... and that are put in order as they are; of more, kFew at most
constexpr int kFew = 128;
constexpr int kWork = 512;      // groups that are read again at once
constexpr int kSets = 128;      // threads are taken together in so many sets for the bound
// A bound that so many more sets or columns reach than have to will do.
__device__ __forceinline__ int slack(int k) { return 4 + k / 4; }

template <int G> struct Pick {
  uint64_t best[kCap];
  const void* x[kMaxRanks];      // the pieces, for threads that read different ones
  uint32_t lanes[G];
  union {
    uint16_t work[kWork];
    uint64_t few[kFew];
  };
  uint64_t from;
  uint32_t bound;
  int n, groups, sum[2];
};

// Runs f(place) on the elements of a unit that count.
template <int DT, typename F>
__device__ __forceinline__ void each_of(const LogpArgs& a, const Chunk& s, const Lane& l, const Unit<DT>& u, F f) {
#pragma unroll
  for (int i = 0; i < kU; ++i)
    if (counts(s, l, a.valid, i)) f(place_of(order_of(unit_get<DT>(u, i)), s.col0 - s.c0 + l.c + i));
}

// Runs f(place) on the elements of the thread's groups whose maximum reaches `key`.  `top`: the largest
// order of every group, as the threads read them.
template <int DT, int MODE, typename F>
__device__ __forceinline__ void each_in(const LogpArgs& a, int64_t row, Range g, const uint32_t* top, uint32_t key,
                                        F f) {
  const int waves = blockDim.x / 64, next = waves * g.step;
  for (int q0 = g.lo + wave_id() * g.step, b = 0; q0 < g.hi; q0 += kMore * waves * g.step, ++b) {
    if (top[b * blockDim.x + threadIdx.x] < key) continue;
    Unit<DT> u[kMore];
#pragma unroll
    for (int k = 0; k < kMore; ++k) u[k] = fetch<DT, MODE>(a, row, chunk(a, min(q0 + k * next, g.hi - 1)));
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      if (q0 + k * next >= g.hi) continue;
      const Chunk s = chunk(a, q0 + k * next);
      each_of<DT>(a, s, lane_of<MODE>(s), u[k], f);
    }
  }
}

template <int G>
__device__ __forceinline__ void keep(Pick<G>* P, uint64_t x) {
  const int i = atomicAdd(&P->n, 1);
  if (i < kCap) P->best[i] = x;
}

// Element i of a unit, where i is known at run time only.
template <int DT>
__device__ __forceinline__ float unit_at(const Unit<DT>& u, int i) {
  float x = unit_get<DT>(u, 0);
#pragma unroll
  for (int j = 1; j < kU; ++j) x = i == j ? unit_get<DT>(u, j) : x;
  return x;
}

// Keeps the elements of a unit whose order reaches the bound.
template <int DT, int G>
__device__ __forceinline__ void keep_unit(const LogpArgs& a, const Chunk& s, const Lane& l, const Unit<DT>& u,
                                          uint32_t bound, Pick<G>* P) {
  const float least = logit_of(bound);
  const bool nan = bound == 0xffffffffu;      // only NaN reaches it
  uint32_t hits = 0;
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const float x = unit_get<DT>(u, i);
    const bool hit = !(x < least) && !(nan && x == x) && counts(s, l, a.valid, i);
    hits |= hit ? 1u << i : 0u;
  }
  if (hits == 0) return;
  for (int at = atomicAdd(&P->n, __builtin_popcount(hits)); hits != 0; hits &= hits - 1, ++at) {
    const int i = __builtin_ctz(hits);
    if (at < kCap) P->best[at] = place_of(order_of(unit_at<DT>(u, i)), s.col0 - s.c0 + l.c + i);
  }
}

// The k-th largest of the maxima of kSets sets of threads, or a smaller one that at most slack(k) more sets
// reach; by one wave.  (With a set for each thread, more of the k best are sets' maxima, and the
// bound is higher; 128 sets bring 22 of the row's elements for 20, 89 for 64, in a quarter of the
// steps.)
template <int G>
__device__ __forceinline__ uint32_t bound_of(const uint32_t* v, int k) {
  const int lane = threadIdx.x % 64;
  uint32_t x = 0, y = 0;
#pragma unroll
  for (int i = 0; i < G; i += kSets) {
    x = max(x, v[i + lane]);
    y = max(y, v[i + 64 + lane]);
  }
  auto reach = [&](uint32_t at) { return __builtin_popcountll(__ballot(x >= at)) + __builtin_popcountll(__ballot(y >= at)); };
  uint32_t hi = wave_max_u32(max(x, y)), lo = ~wave_max_u32(~min(x, y));
  if (reach(hi) >= k) return hi;
  while (hi - lo > 1) {            // lo is reached by k at least, hi by fewer
    // three at once take as long as one
    const uint32_t d = (hi - lo) / 4 + (hi - lo < 4), m1 = lo + d, m2 = min(m1 + d, hi), m3 = min(m2 + d, hi);
    const int n1 = reach(m1), n2 = reach(m2), n3 = reach(m3);
    const int n = n3 >= k ? n3 : n2 >= k ? n2 : n1;
    if (n3 >= k) lo = m3;
    else if (n2 >= k) lo = m2, hi = m3;
    else if (n1 >= k) lo = m1, hi = m2;
    else hi = m1;
    if (n >= k && n <= k + slack(k)) break;
  }
  return lo;
}

// A place that at least k of n > k places reach, and at most slack(k) more; all reach lo.  By one wave.
__device__ __forceinline__ uint64_t place_bound(const uint64_t* v, int n, int k, uint64_t lo) {
  uint64_t hi = ~0ull;
  while (hi - lo > 1) {
    const uint64_t mid = lo + (hi - lo) / 2;
    int m = 0;
    for (int i = 0; i < n; i += 64) {
      const int j = i + threadIdx.x % 64;
      m += __builtin_popcountll(__ballot(j < n && v[min(j, n - 1)] >= mid));
    }
    if (m < k) {
      hi = mid;
    } else {
      lo = mid;
      if (m <= k + slack(k)) break;
    }
  }
  return lo;
}

// The k best places that a workgroup's threads have (all, if there are fewer), and a few more perhaps.
// mine: the largest order that the thread has.  quick(bound): keeps the places whose order reaches the
// bound, or only counts groups beyond kWork.  each(key, f): runs f(place) on the thread's places, where it may
// pass over orders below the key.
struct Picked {
  const uint64_t* list;
  int n;
};
template <int G, typename Quick, typename Each>
__device__ __forceinline__ Picked pick(int k, uint32_t mine, Pick<G>* P, Quick quick, Each each) {
  P->lanes[threadIdx.x] = mine;
  if (threadIdx.x == 0) P->n = P->groups = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t t = bound_of<G>(P->lanes, k);
    if (threadIdx.x == 0) P->bound = max(t, 1u);
  }
  __syncthreads();
  const uint32_t bound = P->bound;
  quick(bound);
  __syncthreads();
  uint64_t lo = (uint64_t)bound << 32;
  int n = P->groups > kWork ? kCap + 1 : P->n;
  if (n > kCap) {
    // ties, or many of the best in few threads.  lo is reached by more than k, hi by fewer (or is the
    // last place there is)
    uint64_t hi = ~0ull;
    uint64_t mid = bound == 0xffffffffu ? lo + (1ull << 31) : (uint64_t)(bound + 1) << 32;
    for (int turn = 0; hi - lo > 1; turn ^= 1, mid = lo + (hi - lo) / 2) {
      if (threadIdx.x == 0) P->sum[turn] = 0;
      __syncthreads();
      int m = 0;
      each((uint32_t)(mid >> 32), [&](uint64_t x) { m += x >= mid; });
      atomicAdd(&P->sum[turn], m);
      __syncthreads();
      n = P->sum[turn];         // zeroed again two turns and three barriers later
      if (n < k) {
        hi = mid;
      } else {
        lo = mid;
        if (n <= kCap) break;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) P->n = 0;
    __syncthreads();
    each((uint32_t)(lo >> 32), [&](uint64_t x) {
      if (x >= lo) keep(P, x);
    });
    __syncthreads();
    n = P->n;
  }
  if (n <= kOrder) return {P->best, n};
  if (threadIdx.x < 64) {
    const uint64_t t = place_bound(P->best, n, k, lo);
    if (threadIdx.x == 0) P->from = t, P->groups = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += G)
    if (P->best[i] >= P->from) P->few[atomicAdd(&P->groups, 1)] = P->best[i];
  __syncthreads();
  return {P->few, P->groups};
}

// The k best of a row's range.
template <int DT, int MODE, int G>
__device__ __forceinline__ Picked pick_row(const LogpArgs& a, int64_t row, Range g, int k, const uint32_t* top,
                                           Pick<G>* P) {
  constexpr int waves = G / 64;
  uint32_t mine = 0;
  for (int q0 = g.lo + wave_id() * g.step, b = 0; q0 < g.hi; q0 += kMore * waves * g.step, ++b) mine = max(mine, top[b * G + threadIdx.x]);
  return pick<G>(k, mine, P, [&](uint32_t bound) {
    // the groups that reach the bound, then a thread to each unit of them: one round trip to memory
    for (int q0 = g.lo + wave_id() * g.step, b = 0; q0 < g.hi; q0 += kMore * waves * g.step, ++b) {
      if (top[b * G + threadIdx.x] < bound) continue;
      const int i = atomicAdd(&P->groups, 1);
      if (i < kWork) P->work[i] = (uint16_t)(b * G + threadIdx.x);
    }
    __syncthreads();
    const int units = min(P->groups, kWork) * kMore;
    for (int i = threadIdx.x; i < units; i += G) {
      const int e = P->work[i / kMore], from = e % G;
      const int q = g.lo + (from / 64 + (e / G * kMore + i % kMore) * waves) * g.step;
      if (q >= g.hi) continue;
      const Chunk s = chunk_of(a, q);
      const Lane l = lane_of<MODE>(s, from % 64);
      keep_unit<DT, G>(a, s, l, fetch_of<DT, MODE>(P->x[s.r], row, s, l), bound, P);
    }
  }, [&](uint32_t key, auto f) { each_in<DT, MODE>(a, row, g, top, key, f); });
}

// f(rank, place) for the first k of some places, four threads to each.
template <int G, typename F>
__device__ __forceinline__ void in_order(const Picked& t, int k, F f) {
  const int sub = threadIdx.x % 4;
  for (int i = threadIdx.x / 4; i < t.n; i += G / 4) {
    const uint64_t x = t.list[i];
    uint32_t rank = 0;
#pragma unroll 4
    for (int j = sub; j < t.n; j += 4) rank += t.list[j] > x;
    rank += dpp<kDppNeighbour>(rank);
    rank += dpp<kDppPair>(rank);
    if (sub == 0 && rank < (uint32_t)k) f((int)rank, x);
  }
}

// ---------------------------------------------------------------- results

// A row's statistics when they are settled.
struct Row {
  float m, ln_z, z, w;
};
__device__ __forceinline__ Row row_of(const Stat& t) { return {t.m, log2_of(t.z) * kLn2, t.z, t.w}; }
__device__ __forceinline__ bool empty(const Row& t) { return t.m == -INFINITY && t.z == 0.0f; }
__device__ __forceinline__ float log_p(const Row& t, float x, float scale) {
  return empty(t) ? -INFINITY : below(x, t.m, scale) - t.ln_z;
}

// The given token's logit and its column, or what there is instead: kNoToken, kNoColumn.
constexpr int kNoToken = -1, kNoColumn = -2;
struct Given {
  int col;
  float x;
};
template <int DT>
__device__ __forceinline__ Given given(const LogpArgs& a, int64_t row) {
  if (!a.logprob) return {kNoToken, 0.0f};
  const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[row]
                             : (int64_t)static_cast<const int32_t*>(a.ids)[row];
  const int col = id < 0 ? kNoToken : id < a.valid ? (int)id : kNoColumn;
  return {col, logit<DT>(a, row, col)};
}

// One thread's work.
__device__ __forceinline__ void write_row(const LogpArgs& a, int64_t row, const Row& t, const Given& y) {
  if (a.lse) a.lse[row] = empty(t) ? -INFINITY : __builtin_fmaf(t.m, a.scale, t.ln_z);
  if (a.entropy) a.entropy[row] = empty(t) ? 0.0f : t.ln_z - t.w / t.z * kLn2;
  if (a.logprob)
    a.logprob[row] = y.col == kNoToken ? 0.0f : y.col == kNoColumn ? __uint_as_float(0x7fc00000u) : log_p(t, y.x, a.scale);
}

__device__ __forceinline__ void write_top(const LogpArgs& a, int64_t row, const Row& t, int rank, uint64_t place) {
  const int64_t at = row * a.top + rank;
  const uint32_t col = ~(uint32_t)place;
  if (a.top_ids) {
    if (a.ids64) static_cast<int64_t*>(a.top_ids)[at] = col;
    else static_cast<int32_t*>(a.top_ids)[at] = (int32_t)col;
  }
  if (a.top_logprobs) a.top_logprobs[at] = log_p(t, logit_of((uint32_t)(place >> 32)), a.scale);
}

// The workspace of a part of a row: m, z, w and a spare word, then its best places in order.
__device__ __forceinline__ float* part_space(const LogpArgs& a, int64_t part) {
  return a.part + part * (4 + 2 * a.top);
}

// ---------------------------------------------------------------- kernels

// A workgroup of G threads to a row, or to one of a row's `splits` parts.
template <int DT, int G, int MODE, bool TOP>
__global__ __launch_bounds__(G) void k_logp(LogpArgs a) {
  extern __shared__ uint32_t top[];        // TOP: for each group of 32 that a thread reads, its maximum's order
  __shared__ Stat stats[16];
  __shared__ Pick<G> pool;
  const int waves = G / 64, w = wave_id();
  const unsigned splits = a.splits;
  const int64_t row = a.row0 + blockIdx.x / splits;
  const int part = blockIdx.x % splits;
  const Range g = range_of(a, part);
  const float s2 = a.scale * kLog2e;
  const Given y = a.splits > 1 ? Given{kNoToken, 0.0f} : given<DT>(a, row);     // under way with the logits
  const void* piece = TOP && (int)threadIdx.x < a.p ? a.x.b[threadIdx.x] : nullptr;
  Stat t = none();
  for (int q = g.lo + w * g.step, b = 0; q < g.hi; q += kMore * waves * g.step, ++b) {
    Unit<DT> u[kMore];
    fetch_all<DT, MODE, kMore>(u, a, row, q, waves * g.step, g.hi);
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      // short rows: what lies behind them is not computed (16384 x 1024 bfloat16: 28 us, 22.5 so; with more
      // threads, where few units lie behind a row's end, the branches cost 2%)
      if (G > 128 || k == 0 || q + k * waves * g.step < g.hi) take<DT>(t, most, u[k], s2);
    }
    if (TOP) top[b * G + threadIdx.x] = order_of(most);
  }
  if (TOP && (int)threadIdx.x < a.p) pool.x[threadIdx.x] = piece;
  t = block_join(t, stats, waves);
  if (!settle(t, s2)) {        // the same in all waves
    __syncthreads();
    t = plain_stat<DT, MODE>(a, row, g, reinterpret_cast<float*>(stats));
    if (TOP && t.z != t.z) {
      // the maxima passed over NaN, which is the largest
      for (int q = g.lo + w * g.step, b = 0; q < g.hi; q += kMore * waves * g.step, ++b) {
        Unit<DT> u[kMore];
        fetch_all<DT, MODE, kMore>(u, a, row, q, waves * g.step, g.hi);
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < kMore; ++k)
#pragma unroll
          for (int i = 0; i < kU; ++i) most = max(most, order_of(unit_get<DT>(u[k], i)));
        top[b * G + threadIdx.x] = most;
      }
    }
  }
  const Row r = row_of(t);
  if (a.splits > 1) {
    float* to = part_space(a, row * a.splits + part);
    if (threadIdx.x == G - 64) {
      to[0] = t.m;
      to[1] = t.z;
      to[2] = t.w;
    }
    if constexpr (TOP) {
      uint64_t* list = reinterpret_cast<uint64_t*>(to + 4);
      const Picked best = pick_row<DT, MODE, G>(a, row, g, a.top, top, &pool);
      for (int i = best.n + threadIdx.x; i < a.top; i += G) list[i] = 0;
      in_order<G>(best, a.top, [&](int rank, uint64_t place) { list[rank] = place; });
    }
  } else {
    if (threadIdx.x == G - 64) write_row(a, row, r, y);      // while the first wave looks for the bound
    if constexpr (TOP) {
      const Picked best = pick_row<DT, MODE, G>(a, row, g, a.top, top, &pool);
      in_order<G>(best, a.top, [&](int rank, uint64_t place) { write_top(a, row, r, rank, place); });
    }
  }
}

// The parts of a row, at most 64.  Their best columns, at most 64 of each, lie in LDS.
constexpr int kJoinThreads = 256;

template <int DT, bool TOP>
__global__ __launch_bounds__(TOP ? kJoinThreads : 64) void k_logp_join(LogpArgs a) {
  extern __shared__ uint64_t places[];
  __shared__ Pick<kJoinThreads> pool;
  constexpr int G = TOP ? kJoinThreads : 64;
  const int64_t row = a.row0 + blockIdx.x;
  const int lane = threadIdx.x % 64;
  const float* parts = part_space(a, row * a.splits);
  Stat t = {-INFINITY, 0.0f, 0.0f, 0.0f};
  if (lane < a.splits) {
    const float* from = parts + lane * (4 + 2 * a.top);
    t = {from[0], 0.0f, from[1], from[2]};
  }
  const Given y = given<DT>(a, row);
  uint32_t mine = 0;
  const int n = a.splits * a.top;
  if constexpr (TOP) {
    for (int i = threadIdx.x; i < n; i += G) {
      // the parts' first ones first, so that they go to many threads
      const int k = i / a.splits, part = i - k * a.splits;
      const uint64_t x = reinterpret_cast<const uint64_t*>(parts + part * (4 + 2 * a.top) + 4)[k];
      places[i] = x;
      mine = max(mine, (uint32_t)(x >> 32));
    }
  }
  // every wave for itself
  const float m = wave_max(t.m);
  // NaN (of -inf - -inf) becomes the floor, too
  const float d = __builtin_fmaxf(exponent_of(a.scale)(t.m, m), kFloor), r = exp2_of(d);
  const Row all = row_of({m, 0.0f, wave_sum(r * t.z), wave_sum(r * __builtin_fmaf(d, t.z, t.w))});
  if (threadIdx.x == 0) write_row(a, row, all, y);
  if constexpr (TOP) {
    auto each = [&](uint32_t, auto f) {
      for (int i = threadIdx.x; i < n; i += G) f(places[i]);
    };
    const Picked best = pick<G>(a.top, mine, &pool, [&](uint32_t bound) {
      each(bound, [&](uint64_t x) {
        if (x >> 32 >= bound) keep(&pool, x);
      });
    }, each);
    in_order<G>(best, a.top, [&](int rank, uint64_t place) { write_top(a, row, all, rank, place); });
  }
}

// The gradient: `splits` workgroups to a row, each wave with M chunks.  16-bit types: four where that leaves
// the GPU eight workgroups to a compute unit, one where not (us with one, two and four; 64 rows of 32000
// bfloat16: 5.2, 5.5, 6.5; 256 of 128000: 28.6, 28.2, 25.3; 4096 of 32000: 145, 123, 111).  Beyond the caches, two
// where all chunks are whole ones (4096 x 131072: 451, 348, 367; 4096 x 110592: -, 309, 322), four where pieces
// leave a rest (4096 x 128000: -, 418, 357).  float32, whose chunks are twice as large: one, beyond the caches two
// (517 x 50017: 45.5, 48, 49.2; 2048 x 131072: 424, 412, 423).
constexpr int kGradThreads = 256, kGradWaves = kGradThreads / 64;

// A token's weights and what its gradient is made with.
struct Weights {
  float a, b, lse, entropy;
  int col;          // of the given token, or -1
};

// WHOLE: all of the chunk's columns are valid.
template <int DT, int MODE, bool ENT, bool WHOLE>
__device__ __forceinline__ void write_grad(const LogpArgs& a, int64_t row, const Chunk& s, const Unit<DT>& u,
                                           const Weights& w) {
  Lane l = lane_of<MODE>(s);
  if (WHOLE) l.c = l.from;
  const int col = s.col0 - s.c0 + l.c;
  float d[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    // x - lse first: a product lse log2 e would be rounded once more
    const float ln_p = __builtin_fmaf(unit_get<DT>(u, i), a.scale, -w.lse), p = exp_of(ln_p);
    d[i] = ENT ? -p * __builtin_fmaf(w.b, __builtin_fmaxf(ln_p, kFloor) + w.entropy, w.a) : -p * w.a;
  }
  if (w.col >= s.col0 && w.col < s.col0 + kChunk) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i == w.col) d[i] += w.a;
  }
  if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i >= a.valid) d[i] = 0.0f;       // padding's gradient is zero, whatever the weights are
  }
  put<DT, MODE, WHOLE>(a, row, s, l, unit_make<DT>(d));
}

template <int DT, int MODE, int M, bool ENT>
__global__ __launch_bounds__(kGradThreads) void k_logp_grad(LogpArgs a) {
  const unsigned splits = a.splits;
  const int64_t row = a.row0 + blockIdx.x / splits;
  const int q0 = blockIdx.x % splits * (kGradWaves * M) + wave_id();
  if (q0 >= a.total) return;
  Unit<DT> u[M];
  fetch_all<DT, MODE, M>(u, a, row, q0, kGradWaves, a.total);
  int64_t id = -1;
  if (a.dlogprob)
    id = a.ids64 ? static_cast<const int64_t*>(a.ids)[row] : (int64_t)static_cast<const int32_t*>(a.ids)[row];
  Weights w = {a.dlogprob ? a.dlogprob[row] : 0.0f, ENT ? a.dentropy[row] : 0.0f, a.lse_in[row],
               ENT ? a.entropy_in[row] : 0.0f, id >= 0 && id < a.valid ? (int)id : -1};
  if (id < 0) w.a = 0.0f;
  // a token without weights, or all of whose columns are -inf, gets zeros whatever else its row holds
  const bool zero = id < a.valid && ((w.a == 0.0f && w.b == 0.0f) || w.lse == -INFINITY);
  if (id >= a.valid || !(w.lse < INFINITY)) w.a = __uint_as_float(0x7fc00000u);
  w.a *= a.scale;
  w.b *= a.scale;
#pragma unroll
  for (int k = 0; k < M; ++k) {
    const int q = q0 + k * kGradWaves;
    if (q >= a.total) continue;
    const Chunk s = chunk(a, q);
    if (zero) put<DT, MODE, false>(a, row, s, lane_of<MODE>(s), Unit<DT>{});
    else if (q < a.full) write_grad<DT, MODE, ENT, true>(a, row, s, u[k], w);
    else write_grad<DT, MODE, ENT, false>(a, row, s, u[k], w);
  }
}

template <int DT, int G, int MODE>
hipError_t rows_go(const LogpArgs& args, hipStream_t s) {
  LogpArgs a = args;
  const int64_t most = std::max<int64_t>(1, 0xFFFFFFFFll / G / a.splits);
  const int per = (a.total + a.splits - 1) / a.splits, step = G / 64 * kMore;
  const unsigned groups = (unsigned)((per + step - 1) / step) * G * 4;
  const unsigned lists = (unsigned)(a.splits * a.top) * 8;
  for (; a.row0 < a.tokens; a.row0 += most) {
    const int64_t rows = std::min(most, a.tokens - a.row0);
    const unsigned grid = (unsigned)(rows * a.splits);
    if (a.top > 0) k_logp<DT, G, MODE, true><<<grid, G, groups, s>>>(a);
    else k_logp<DT, G, MODE, false><<<grid, G, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.splits == 1) continue;
    if (a.top > 0) k_logp_join<DT, true><<<(unsigned)rows, kJoinThreads, lists, s>>>(a);
    else k_logp_join<DT, false><<<(unsigned)rows, 64, 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Beyond the caches, past them: 4096 x 131072 bfloat16 176 us against 186 (within them, 1003 x 50017 float32,
// 46 against 36).
template <int DT, int MODE>
hipError_t logp_size(const LogpArgs& a, hipStream_t s) {
  if (a.splits > 1) return rows_go<DT, 256, MODE>(a, s);
  // threads to a row: fewer for short rows, of which a compute unit then holds more, and the others' loads
  // cover a row's end; as many as pay off where rows are too few for that (top 20, us with 512, 256 and 128
  // before later steps; 4096 x 32000: 66, 59, 70; 16384 x 8192: 147, 83, 73; 300 x 32000: 14.3, 15.4, 22.7)
  const bool many = a.tokens >= 2048;
  if (a.total <= (many ? 16 : 8)) return rows_go<DT, 128, MODE>(a, s);
  return many && a.total <= 128 ? rows_go<DT, 256, MODE>(a, s) : rows_go<DT, 512, MODE>(a, s);
}

template <int DT>
hipError_t logp_go(const LogpArgs& a, int access, hipStream_t s) {
  if (a.cut.base < kU) return rows_go<DT, 128, kTiny>(a, s);
  if (access == kStreamRows) return logp_size<DT, kStream>(a, s);
  return access == kAlignedRows ? logp_size<DT, kAligned>(a, s) : logp_size<DT, kOdd>(a, s);
}

template <int DT, int MODE, int M>
hipError_t grad_go(const LogpArgs& args, hipStream_t s) {
  LogpArgs a = args;
  a.splits = (a.total + kGradWaves * M - 1) / (kGradWaves * M);
  const int64_t most = 0xFFFFFFFFll / kGradThreads / a.splits;
  for (; a.row0 < a.tokens; a.row0 += most) {
    const unsigned grid = (unsigned)(std::min(most, a.tokens - a.row0) * a.splits);
    if (a.dentropy) k_logp_grad<DT, MODE, M, true><<<grid, kGradThreads, 0, s>>>(a);
    else k_logp_grad<DT, MODE, M, false><<<grid, kGradThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int M>
hipError_t grad_rows(const LogpArgs& a, bool al, hipStream_t s) {
  return al ? grad_go<DT, kAligned, M>(a, s) : grad_go<DT, kOdd, M>(a, s);
}

constexpr int64_t kGradFew = 2048 * kGradWaves * 4;      // chunks

// Past the caches where they do not hold the call (4096 x 128000 bfloat16: 354 us against 392), but not
// float32, of which a lane's accesses are half lines (2048 x 131072: 412 against 388).
template <int DT>
hipError_t bwd_go(const LogpArgs& a, bool al, bool big, hipStream_t s) {
  if (a.cut.base < kU) return grad_go<DT, kTiny, 1>(a, s);
  if constexpr (DT == 1) {
    return big ? grad_rows<DT, 2>(a, al, s) : grad_rows<DT, 1>(a, al, s);
  } else {
    if (al && big) return a.total == a.whole * a.p ? grad_go<DT, kStream, 2>(a, s) : grad_go<DT, kStream, 4>(a, s);
    return a.tokens * a.total < kGradFew ? grad_rows<DT, 1>(a, al, s) : grad_rows<DT, 4>(a, al, s);
  }
}

}  // namespace

int64_t logp_bytes(int64_t tokens, int splits, int top) { return splits > 1 ? tokens * splits * (16 + 8 * top) : 0; }

// Workgroups share a row where tokens are few, and where it is longer than what one of them
// keeps the maxima of (36 KiB; at most 64 parts for the longest row there is).
constexpr int kPartChunks = 576;
int logp_splits(int64_t tokens, int vocab, int p) {
  const int chunks = vocab_chunks(vocab, p);
  const int need = (chunks + kPartChunks - 1) / kPartChunks;
  if (vocab / p < kU || tokens < 1) return 1;
  if (need > 1 && tokens > chunks / 2) return need;
  if (chunks <= 64 || tokens > chunks / 2) return 1;
  // two chunks at least for each of the four waves of a part
  return (int)std::max<int64_t>(need, std::min<int64_t>(std::min(64, chunks / 8), (1024 + tokens - 1) / tokens));
}

hipError_t launch_logp(const LogpArgs& a, int dtype, int access, hipStream_t s) {
  if (dtype == 1) return logp_go<1>(a, access, s);
  if (dtype == 2) return logp_go<2>(a, access, s);
  return logp_go<3>(a, access, s);
}

hipError_t launch_logp_bwd(const LogpArgs& a, int dtype, bool al, bool big, hipStream_t s) {
  if (dtype == 1) return bwd_go<1>(a, al, big, s);
  if (dtype == 2) return bwd_go<2>(a, al, big, s);
  return bwd_go<3>(a, al, big, s);
}

}  // namespace ra
