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
// keeps the largest logit of every 32 that it reads.  The k-th largest of the threads' own
// maxima bounds the k-th best logit from below, and only the groups whose maximum reaches
// that bound are read again, some k of a row's thousands.  Their elements at or above the
// bound are put in order by counting, for each, the ones in front of it.  Where too many
// reach the bound (ties), it is raised first, by halving the interval of (logit, column).
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

// Joins a unit; `top` becomes the largest of itself and the unit's logits.  NaN is passed over
// by the maxima, and makes z NaN.
template <int DT>
__device__ __forceinline__ void take(Stat& t, float& top, const Unit<DT>& u, float s2) {
  float x[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) x[i] = unit_get<DT>(u, i);
  const float most = max3(max3(max3(x[0], x[1], x[2]), x[3], x[4]), max3(x[5], x[6], x[7]), -INFINITY);
  top = __builtin_fmaxf(top, most);
  t.m = __builtin_fmaxf(t.m, most);
  const float c = __builtin_fmaxf(kNone, t.m * s2);
  const float d = t.c - c, r = exp2_of(d);
  t.w = r * __builtin_fmaf(d, t.z, t.w);
  t.z *= r;
  t.c = c;
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const float y = __builtin_fmaf(x[i], s2, -c), e = exp2_of(y);
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
__device__ __forceinline__ Stat join2(const Stat& a, const Stat& b) {
  const float c = __builtin_fmaxf(a.c, b.c), da = a.c - c, db = b.c - c, ra = exp2_of(da), rb = exp2_of(db);
  return {__builtin_fmaxf(a.m, b.m), c, a.z * ra + b.z * rb,
          ra * __builtin_fmaf(da, a.z, a.w) + rb * __builtin_fmaf(db, b.z, b.w)};
}

// Over the workgroup of at most 16 waves; every lane gets it.  `lds` is free again at the next
// barrier.
__device__ __forceinline__ Stat block_join(Stat t, Stat* lds, int waves) {
  t = row_join(t);
  t = join2(join2(lane_stat(t, 0), lane_stat(t, 16)), join2(lane_stat(t, 32), lane_stat(t, 48)));
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

// The chunks of a workgroup: [lo, hi), its waves taking one each in turn.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range range_of(const VocabArgs& a, int part) {
  const int per = (a.total + a.splits - 1) / a.splits, lo = min(a.total, part * per);
  return {lo, min(a.total, lo + per)};
}

// The statistics of a range with the largest logit subtracted first, by the workgroup.
template <int DT, int MODE>
__device__ __forceinline__ Stat plain_stat(const LogpArgs& a, int64_t row, Range g, float s2, float* lds) {
  const int w = wave_id(), waves = blockDim.x / 64;
  float m = -INFINITY;
  for (int q = g.lo + w; q < g.hi; q += waves) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, waves, g.hi);
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
  for (int q = g.lo + w; q < g.hi; q += waves) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, waves, g.hi);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const float y = (unit_get<DT>(u[0], i) - at) * s2, e = exp2_of(y);
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

constexpr int kCap = 1024;      // columns that are put in order
constexpr int kSlack = 32;      // a bound that this many more threads reach than have to will do

struct Pick {
  uint64_t best[kCap];
  uint32_t bound;
  int n, sum[2];
};

// Runs f(place) on the elements of the thread's groups whose maximum reaches `key`.
template <int DT, int MODE, typename F>
__device__ __forceinline__ void each_in(const LogpArgs& a, int64_t row, Range g, const uint32_t* top, uint32_t key,
                                        F f) {
  const int waves = blockDim.x / 64;
  for (int q0 = g.lo + wave_id(), b = 0; q0 < g.hi; q0 += kMore * waves, ++b) {
    if (top[b * blockDim.x + threadIdx.x] < key) continue;
    Unit<DT> u[kMore];
#pragma unroll
    for (int k = 0; k < kMore; ++k) u[k] = fetch<DT, MODE>(a, row, chunk(a, min(q0 + k * waves, g.hi - 1)));
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      if (q0 + k * waves >= g.hi) continue;
      const Chunk s = chunk(a, q0 + k * waves);
      const Lane l = lane_of<MODE>(s);
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (counts(s, l, a.valid, i)) f(place_of(order_of(unit_get<DT>(u[k], i)), s.col0 - s.c0 + l.c + i));
    }
  }
}

// Elements of the range at or above a place.
template <int DT, int MODE>
__device__ __forceinline__ int count_from(const LogpArgs& a, int64_t row, Range g, const uint32_t* top, Pick* P,
                                          int turn, uint64_t from) {
  int n = 0;
  each_in<DT, MODE>(a, row, g, top, (uint32_t)(from >> 32), [&](uint64_t x) { n += x >= from; });
  if (threadIdx.x == 0) P->sum[turn] = 0;
  __syncthreads();
  atomicAdd(&P->sum[turn], n);
  __syncthreads();
  return P->sum[turn];     // zeroed again two calls and a barrier later
}

// Keeps the elements at or above a place, in any order, and returns their number.
template <int DT, int MODE>
__device__ __forceinline__ int keep_from(const LogpArgs& a, int64_t row, Range g, const uint32_t* top, Pick* P,
                                         uint64_t from) {
  if (threadIdx.x == 0) P->n = 0;
  __syncthreads();
  each_in<DT, MODE>(a, row, g, top, (uint32_t)(from >> 32), [&](uint64_t x) {
    if (x < from) return;
    const int i = atomicAdd(&P->n, 1);
    if (i < kCap) P->best[i] = x;
  });
  __syncthreads();
  return P->n;
}

// The k-th largest of G values, or a smaller one that at most kSlack more reach; by one wave.
template <int G>
__device__ __forceinline__ uint32_t bound_of(const uint32_t* v, int k) {
  uint32_t x[G / 64], least = 0xffffffffu, most = 0;
#pragma unroll
  for (int i = 0; i < G / 64; ++i) {
    x[i] = v[i * 64 + threadIdx.x % 64];
    least = min(least, x[i]);
    most = max(most, x[i]);
  }
  auto reach = [&](uint32_t at) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < G / 64; ++i) n += __builtin_popcountll(__ballot(x[i] >= at));
    return n;
  };
  uint32_t hi = wave_max_u32(most), lo = ~wave_max_u32(~least);
  if (reach(hi) >= k) return hi;
  while (hi - lo > 1) {            // lo is reached by k at least, hi by fewer
    const uint32_t mid = lo + (hi - lo) / 2;
    const int n = reach(mid);
    if (n < k) {
      hi = mid;
    } else {
      lo = mid;
      if (n <= k + kSlack) break;
    }
  }
  return lo;
}

// Leaves the k best elements of a range (all, if it has fewer), and a few more perhaps, in P->best and
// returns how many.  `top`: the largest order of every group, as the threads read them; `lanes`: room
// for G words.
template <int DT, int MODE, int G>
__device__ __forceinline__ int pick(const LogpArgs& a, int64_t row, Range g, int k, const uint32_t* top,
                                    uint32_t* lanes, Pick* P) {
  uint32_t mine = 0;
  const int waves = G / 64;
  for (int q0 = g.lo + wave_id(), b = 0; q0 < g.hi; q0 += kMore * waves, ++b) mine = max(mine, top[b * G + threadIdx.x]);
  lanes[threadIdx.x] = mine;
  __syncthreads();
  if (threadIdx.x < 64) {
    const uint32_t t = bound_of<G>(lanes, k);
    if (threadIdx.x == 0) P->bound = max(t, 1u);
  }
  __syncthreads();
  const uint32_t bound = P->bound;
  uint64_t lo = (uint64_t)bound << 32;
  int n = keep_from<DT, MODE>(a, row, g, top, P, lo);
  if (n <= kCap) return n;
  // lo is reached by more than k, hi by fewer (or is the last place there is)
  uint64_t hi = ~0ull, mid = bound == 0xffffffffu ? lo + (1ull << 31) : (uint64_t)(bound + 1) << 32;
  for (int turn = 0; hi - lo > 1; turn ^= 1, mid = lo + (hi - lo) / 2) {
    n = count_from<DT, MODE>(a, row, g, top, P, turn, mid);
    if (n < k) {
      hi = mid;
    } else {
      lo = mid;
      if (n <= kCap) break;
    }
  }
  __syncthreads();
  return keep_from<DT, MODE>(a, row, g, top, P, lo);
}

// f(rank, place) for the first k of P->best's n.
template <typename F>
__device__ __forceinline__ void in_order(const Pick* P, int n, int k, F f) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t x = P->best[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += P->best[j] > x;
    if (rank < k) f(rank, x);
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
  return empty(t) ? -INFINITY : (x - t.m) * scale - t.ln_z;
}

// One thread's work.
template <int DT>
__device__ __forceinline__ void write_row(const LogpArgs& a, int64_t row, const Row& t) {
  if (a.lse) a.lse[row] = empty(t) ? -INFINITY : __builtin_fmaf(t.m, a.scale, t.ln_z);
  if (a.entropy) a.entropy[row] = empty(t) ? 0.0f : t.ln_z - t.w / t.z * kLn2;
  if (!a.logprob) return;
  const int64_t id = a.ids64 ? static_cast<const int64_t*>(a.ids)[row]
                             : (int64_t)static_cast<const int32_t*>(a.ids)[row];
  float r = 0.0f;
  if (id >= a.valid) r = __uint_as_float(0x7fc00000u);
  else if (id >= 0) r = log_p(t, logit<DT>(a, row, (int)id), a.scale);
  a.logprob[row] = r;
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
  __shared__ Pick pool;
  __shared__ uint32_t lanes[TOP ? G : 1];
  const int waves = G / 64, w = wave_id();
  const unsigned splits = a.splits;
  const int64_t row = a.row0 + blockIdx.x / splits;
  const int part = blockIdx.x % splits;
  const Range g = range_of(a, part);
  const float s2 = a.scale * kLog2e;
  Stat t = none();
  for (int q = g.lo + w, b = 0; q < g.hi; q += kMore * waves, ++b) {
    Unit<DT> u[kMore];
    fetch_all<DT, MODE, kMore>(u, a, row, q, waves, g.hi);
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMore; ++k) take<DT>(t, most, u[k], s2);
    if (TOP) top[b * G + threadIdx.x] = order_of(most);
  }
  t = block_join(t, stats, waves);
  if (!settle(t, s2)) {        // the same in all waves
    __syncthreads();
    t = plain_stat<DT, MODE>(a, row, g, s2, reinterpret_cast<float*>(stats));
    if (TOP && t.z != t.z) {
      // the maxima passed over NaN, which is the largest
      for (int q = g.lo + w, b = 0; q < g.hi; q += kMore * waves, ++b) {
        Unit<DT> u[kMore];
        fetch_all<DT, MODE, kMore>(u, a, row, q, waves, g.hi);
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
    if (threadIdx.x == 0) {
      to[0] = t.m;
      to[1] = t.z;
      to[2] = t.w;
    }
    if constexpr (TOP) {
      uint64_t* list = reinterpret_cast<uint64_t*>(to + 4);
      const int n = pick<DT, MODE, G>(a, row, g, a.top, top, lanes, &pool);
      for (int i = n + threadIdx.x; i < a.top; i += G) list[i] = 0;
      in_order(&pool, n, a.top, [&](int rank, uint64_t place) { list[rank] = place; });
    }
  } else {
    if (threadIdx.x == 0) write_row<DT>(a, row, r);
    if constexpr (TOP) {
      const int n = pick<DT, MODE, G>(a, row, g, a.top, top, lanes, &pool);
      in_order(&pool, n, a.top, [&](int rank, uint64_t place) { write_top(a, row, r, rank, place); });
    }
  }
}

// The parts of a row, at most 64: a wave to a row.  Its best columns are the parts' merged:
// the largest of the parts' first ones, k times.
template <int DT>
__global__ __launch_bounds__(64) void k_logp_join(LogpArgs a) {
  extern __shared__ uint64_t lists[];
  const int64_t row = a.row0 + blockIdx.x;
  const int lane = threadIdx.x;
  const float s2 = a.scale * kLog2e;
  Stat t = {-INFINITY, 0.0f, 0.0f, 0.0f};
  if (lane < a.splits) {
    const float* from = part_space(a, row * a.splits + lane);
    t = {from[0], 0.0f, from[1], from[2]};
  }
  const float m = wave_max(t.m);
  // NaN (of -inf - -inf) becomes the floor, too
  const float d = __builtin_fmaxf((t.m - m) * s2, kFloor), r = exp2_of(d);
  const Row all = row_of({m, 0.0f, wave_sum(r * t.z), wave_sum(r * __builtin_fmaf(d, t.z, t.w))});
  if (lane == 0) write_row<DT>(a, row, all);
  if (a.top == 0) return;
  for (int i = lane; i < a.splits * a.top; i += 64) {
    const int part = i / a.top, k = i % a.top;
    lists[i] = reinterpret_cast<const uint64_t*>(part_space(a, row * a.splits + part) + 4)[k];
  }
  __syncthreads();
  uint64_t mine = 0;
  int next = 0;
  uint64_t head = lane < a.splits ? lists[lane * a.top] : 0;
  for (int k = 0; k < a.top; ++k) {
    const uint32_t hi = wave_max_u32((uint32_t)(head >> 32));
    const uint32_t lo = wave_max_u32((uint32_t)(head >> 32) == hi ? (uint32_t)head : 0u);
    const uint64_t best = (uint64_t)hi << 32 | lo;
    if (lane == k) mine = best;
    if (head == best) {
      ++next;
      head = next < a.top ? lists[lane * a.top + next] : 0;
    }
  }
  if (lane < a.top) write_top(a, row, all, lane, mine);
}

// The gradient: `splits` workgroups to a row.
constexpr int kGradThreads = 256;

template <int DT, int MODE, bool ENT>
__global__ __launch_bounds__(kGradThreads) void k_logp_grad(LogpArgs a) {
  constexpr int kWaves = kGradThreads / 64;
  const unsigned splits = a.splits;
  const int64_t row = a.row0 + blockIdx.x / splits;
  const Range g = range_of(a, blockIdx.x % splits);
  int64_t id = -1;
  if (a.dlogprob)
    id = a.ids64 ? static_cast<const int64_t*>(a.ids)[row] : (int64_t)static_cast<const int32_t*>(a.ids)[row];
  float da = id < 0 ? 0.0f : a.dlogprob[row];
  float db = ENT ? a.dentropy[row] : 0.0f;
  const float lse = a.lse_in[row], ent = ENT ? a.entropy_in[row] : 0.0f;
  // a token without weights, or all of whose columns are -inf, gets zeros whatever else its row holds
  const bool zero = id < a.valid && ((da == 0.0f && db == 0.0f) || lse == -INFINITY);
  if (id >= a.valid || !(lse < INFINITY)) da = __uint_as_float(0x7fc00000u);
  const int y = id >= 0 && id < a.valid ? (int)id : -1;
  da *= a.scale;
  db *= a.scale;
  for (int q0 = g.lo + wave_id(); q0 < g.hi; q0 += kMore * kWaves) {
    Unit<DT> u[kMore];
    if (!zero) fetch_all<DT, MODE, kMore>(u, a, row, q0, kWaves, g.hi);
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      const int q = q0 + k * kWaves;
      if (q >= g.hi) continue;
      const Chunk s = chunk(a, q);
      const Lane l = lane_of<MODE>(s);
      const int col = s.col0 - s.c0 + l.c;
      float d[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (zero) {
          d[i] = 0.0f;
          continue;
        }
        // x - lse first: a product lse log2 e would be rounded once more
        const float ln_p = __builtin_fmaf(unit_get<DT>(u[k], i), a.scale, -lse);
        const float p = exp_of(ln_p);
        d[i] = ENT ? -p * __builtin_fmaf(db, __builtin_fmaxf(ln_p, kFloor) + ent, da) : -p * da;
        if (col + i == y) d[i] += da;
        if (col + i >= a.valid) d[i] = 0.0f;       // padding's gradient is zero, whatever the weights are
      }
      put<DT, MODE, false>(a, row, s, l, unit_make<DT>(d));
    }
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
    k_logp_join<DT><<<(unsigned)rows, 64, lists, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int MODE>
hipError_t logp_size(const LogpArgs& a, hipStream_t s) {
  if (a.splits > 1) return rows_go<DT, 256, MODE>(a, s);
  return a.total <= 8 ? rows_go<DT, 128, MODE>(a, s) : rows_go<DT, 512, MODE>(a, s);
}

template <int DT>
hipError_t logp_go(const LogpArgs& a, bool al, hipStream_t s) {
  if (a.cut.base < kU) return rows_go<DT, 128, kTiny>(a, s);
  return al ? logp_size<DT, kAligned>(a, s) : logp_size<DT, kOdd>(a, s);
}

template <int DT, int MODE>
hipError_t grad_go(const LogpArgs& args, hipStream_t s) {
  LogpArgs a = args;
  const int64_t most = 0xFFFFFFFFll / kGradThreads / a.splits;
  for (; a.row0 < a.tokens; a.row0 += most) {
    const unsigned grid = (unsigned)(std::min(most, a.tokens - a.row0) * a.splits);
    if (a.dentropy) k_logp_grad<DT, MODE, true><<<grid, kGradThreads, 0, s>>>(a);
    else k_logp_grad<DT, MODE, false><<<grid, kGradThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t bwd_go(const LogpArgs& a, bool al, hipStream_t s) {
  if (a.cut.base < kU) return grad_go<DT, kTiny>(a, s);
  return al ? grad_go<DT, kAligned>(a, s) : grad_go<DT, kOdd>(a, s);
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

hipError_t launch_logp(const LogpArgs& a, int dtype, bool al, hipStream_t s) {
  if (dtype == 1) return logp_go<1>(a, al, s);
  if (dtype == 2) return logp_go<2>(a, al, s);
  return logp_go<3>(a, al, s);
}

hipError_t launch_logp_bwd(const LogpArgs& a, int dtype, bool al, hipStream_t s) {
  if (dtype == 1) return bwd_go<1>(a, al, s);
  if (dtype == 2) return bwd_go<2>(a, al, s);
  return bwd_go<3>(a, al, s);
}

}  // namespace ra
