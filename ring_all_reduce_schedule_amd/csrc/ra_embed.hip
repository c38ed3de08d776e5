// ra_embed.hip -- rows of an embedding table whose vocabulary is cut over the
// ranks, and the gradient of those rows.
//
//   y_t = scale W[id_t],     dW[v] = scale * sum over {t: id_t = v} of dy_t  (+ dW[v])
//
// A rank that does not hold id_t would add a row of zeros to the sum over the
// ranks; here the one row that counts is read from the rank that holds it and
// written to every rank.
//
// The gradient adds up the rows of equal tokens in the order of their positions,
// so it does not depend on how the work was scheduled: positions are sorted by
// token (a stable sort), the sorted positions are cut into stretches of equal
// length, and each stretch adds up its runs of equal tokens in float32.  A run
// inside one stretch is written at once; the sums of a run that crosses stretches
// go to the workspace and are joined afterwards in order.  Cutting by positions
// and not by tokens keeps the work even: in text the most frequent token makes up
// several percent of all.  No atomics on floats are used.
//
// Both are bound by writing.  Measured on MI355X (fills reach 6.9 TB/s, copies 6.55):
//   16384 tokens x 4096 bfloat16 to 8 ranks              213 us, 5.3 TB/s
//   its gradient, float32, into 131,072 rows              445 us, 5.1 TB/s, of which
//     sorting takes 20, joining long runs 12
//   1003 tokens x 1001 float16 into 5003 rows              20 us in three launches: sort
//     5.4, runs and zeros 11, joins 3.5
#include "ra_rows.h"

namespace ra {
namespace {

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t t) {
  return ids64 ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
}

// G lanes and 256 / G tokens of a workgroup at a time, kTokens of them one after
// the other in a thread; a token's units go over gridDim.y and the lanes.  A thread
// writes its tokens rank by rank: longer pieces of fewer streams at a time (16384
// x 4096 to 8 ranks: 226 us against 229 with one token, 220 past the caches).
constexpr int kTokens = 4;
template <int DT, int G, int AC>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a) {
  const int64_t t0 = a.row0 + ((int64_t)blockIdx.x * (256 / G) + threadIdx.x / G) * kTokens;
  const int j = blockIdx.y * G + threadIdx.x % G;
  if (t0 >= a.tokens || j * kU >= a.hidden) return;
  const Cut u = unit_cut<AC>(j, a.hidden);
  const int n = (int)min((int64_t)kTokens, a.tokens - t0);
  int64_t id[kTokens];
  Unit<DT> w[kTokens];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) id[k] = load_id(a.ids, a.ids64, min(t0 + k, a.tokens - 1));
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const int64_t i = id[k] >= 0 && id[k] < a.vocab ? id[k] : 0;
    const int r = piece_of(a.cut, (int)i);
    w[k] = load_cut<DT, AC != 0>(a.table.b[r], (i - piece_lo(a.cut, r)) * a.hidden, u);
  }
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    float y[kU];
    const float none = id[k] < 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    const bool ok = id[k] >= 0 && id[k] < a.vocab;
#pragma unroll
    for (int i = 0; i < kU; ++i) y[i] = ok ? unit_get<DT>(w[k], i) * a.scale : none;
    w[k] = unit_make<DT>(y);
  }
  for (int r = 0; r < a.n_out; ++r)
#pragma unroll
    for (int k = 0; k < kTokens; ++k)
      if (k < n) store_cut<DT, AC>(a.out.b[r], (t0 + k) * a.hidden, u, w[k]);
}

// ---------------------------------------------------------------- sorting positions by token

// Keys: the token, or `vocab` for what has no row, which sorts behind all rows.
__device__ __forceinline__ int key_of(const EmbedBwdArgs& a, int64_t t) {
  const int64_t id = load_id(a.ids, a.ids64, t);
  return id >= 0 && id < a.vocab ? (int)id : a.vocab;
}

// Few positions: each finds its place by counting the keys before it.  A workgroup
// has all keys in LDS and 64 positions, and each of its 16 waves counts a
// sixteenth of the keys for all 64.  That is quadratic work, but in one launch: 1003
// positions take 5.4 us; 16384 took 49 us, where two passes of the other sort
// take 20.
constexpr int kCountMost = 4096, kCountThreads = 1024;
__global__ __launch_bounds__(kCountThreads) void k_sort_count(EmbedBwdArgs a, int* keys, int* pos) {
  __shared__ __align__(16) int lds[kCountMost];
  constexpr int kWaves = kCountThreads / 64, kStep = kWaves * 4;
  const int n = (int)a.tokens, up = (n + kStep - 1) / kStep * kStep;
  for (int i = threadIdx.x; i < up; i += kCountThreads) lds[i] = i < n ? key_of(a, i) : 0x7fffffff;
  __syncthreads();
  const int w = threadIdx.x / 64, lane = threadIdx.x % 64, me = blockIdx.x * 64 + lane;
  const int key = lds[min(me, n - 1)];
  const int per = up / kWaves, lo = w * per;
  int at = 0;
  typedef int i32x4 __attribute__((ext_vector_type(4)));
#pragma unroll 4
  for (int i = lo; i < lo + per; i += 4) {
    const i32x4 k = *reinterpret_cast<const i32x4*>(lds + i);
    // keys before mine, or equal ones before me: k < key + (their position < mine)
#pragma unroll
    for (int c = 0; c < 4; ++c) at += k[c] < key + (i + c < me ? 1 : 0) ? 1 : 0;
  }
  __syncthreads();
  lds[threadIdx.x] = at;
  __syncthreads();
  if (w == 0 && me < n) {
    at = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) at += lds[i * 64 + lane];
    keys[at] = key;
    pos[at] = me;
  }
}

// More: passes over digits of kBits bits, lowest first, each a stable counting
// sort of blocks of PER * kSortThreads keys.  A block looks through the counts of
// all blocks, so large calls take larger ones; small ones, with two keys to a
// thread, put more compute units to work.
constexpr int kBits = 9, kBins = 1 << kBits, kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSmallTile = 2 * kSortThreads, kLargeTile = 8 * kSortThreads, kSmallMost = 1 << 16;

// Key and position number i of a pass's input; the first pass reads the tokens.
struct SortIn {
  const int* keys;     // null: the tokens themselves
  const int* pos;
};

template <int PER>
__global__ __launch_bounds__(kSortThreads) void k_sort_hist(EmbedBwdArgs a, SortIn in, int shift, int* hist) {
  __shared__ int bins[kBins];
  for (int i = threadIdx.x; i < kBins; i += kSortThreads) bins[i] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * (PER * kSortThreads);
  int key[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int64_t i = min(lo + k * kSortThreads + threadIdx.x, a.tokens - 1);
    key[k] = in.keys ? in.keys[i] : key_of(a, i);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (lo + k * kSortThreads + threadIdx.x < a.tokens) atomicAdd(&bins[(key[k] >> shift) & (kBins - 1)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSortThreads) hist[(int64_t)blockIdx.x * kBins + i] = bins[i];
}

// A block's keys go behind all keys of lower digits, and behind the earlier
// blocks' keys of the same digit; inside the block wave by wave (a wave has
// neighbouring keys), inside a wave round by round and lane by lane.
template <int PER>
__global__ __launch_bounds__(kSortThreads) void k_sort_place(EmbedBwdArgs a, SortIn in, int shift,
                                                             const int* hist, int blocks, int* keys, int* pos) {
  __shared__ int place[kSortWaves][kBins];   // keys of a digit in a wave, then where they start
  __shared__ int waves[kSortWaves];          // sums of the digits' counts, by wave
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64;
  static_assert(kSortThreads == kBins, "a thread to a digit");
  // digit tid: how many keys there are, and how many in earlier blocks
  const int64_t lo = ((int64_t)blockIdx.x * kSortWaves + w) * (PER * 64);
  int key[PER], rank[PER], from[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int64_t i = min(lo + k * 64 + lane, a.tokens - 1);
    key[k] = in.keys ? in.keys[i] : key_of(a, i);
    from[k] = in.pos ? in.pos[i] : (int)i;
  }
  int before = 0, all = 0;
#pragma unroll 8
  for (int b = 0; b < blocks; ++b) {
    const int n = hist[(int64_t)b * kBins + tid];
    before += b < (int)blockIdx.x ? n : 0;
    all += n;
  }
  for (int i = 0; i < kSortWaves; ++i) place[i][tid] = 0;
  // sum over the lower digits: in the wave, then of the waves before
  int lower_digits = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int add = __shfl_up(lower_digits, d);
    lower_digits += lane >= d ? add : 0;
  }
  if (lane == 63) waves[w] = lower_digits;
  lower_digits -= all;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) lower_digits += i < w ? waves[i] : 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const bool in_range = lo + k * 64 + lane < a.tokens;
    const int digit = (key[k] >> shift) & (kBins - 1);
    uint64_t same = __ballot(in_range);
#pragma unroll
    for (int b = 0; b < kBits; ++b) {
      const bool bit = (digit >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    const uint64_t lower = same & ((1ull << lane) - 1);
    rank[k] = 0;
    if (in_range) {
      // the lanes of a digit read its count before the last of them raises it
      const int at = place[w][digit];
      rank[k] = at + __popcll(lower);
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) place[w][digit] = rank[k] + 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __syncthreads();
  int at = lower_digits + before;
  for (int i = 0; i < kSortWaves; ++i) {
    const int n = place[i][tid];
    place[i][tid] = at;
    at += n;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (lo + k * 64 + lane < a.tokens) {
      const int to = place[w][(key[k] >> shift) & (kBins - 1)] + rank[k];
      keys[to] = key[k];
      pos[to] = from[k];
    }
  }
}

// ---------------------------------------------------------------- adding up the runs

// Sorted positions of one stretch, and the most rows that one workgroup clears.
constexpr int kRun = 16, kClearMost = 256;

// Two launches after the sort's: the stretches' runs, together with zeros for the
// rows that have no tokens; then the runs that cross stretches.
struct RunArgs {
  const int* keys;
  const int* pos;
  float* part;        // [stretches][2][hidden]: a stretch's first and last run, where they cross its ends
  int32_t sorted;     // positions
  int32_t stretches;
  int32_t columns;    // workgroups to a stretch, of 256 units
  int32_t clear;      // rows that a workgroup clears, at most kClearMost
};

template <int TT, int AC>
__device__ __forceinline__ void put_row(const EmbedBwdArgs& a, int key, const Cut& u, const float* sum) {
  const int r = piece_of(a.cut, key);
  const int64_t row = (int64_t)(key - piece_lo(a.cut, r)) * a.hidden;
  float y[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) y[i] = sum[i] * a.scale;
  if (a.accumulate) {
    const Unit<TT> old = load_cut<TT, AC>(a.table.b[r], row, u);
#pragma unroll
    for (int i = 0; i < kU; ++i) y[i] += unit_get<TT>(old, i);
  }
  store_cut<TT, AC>(a.table.b[r], row, u, unit_make<TT>(y));
}

// First sorted place whose key is at least `key`, by the whole wave: each round
// looks at 64 places.
__device__ __forceinline__ int lower_bound(const int* keys, int n, int key) {
  int lo = 0, hi = n;                  // the answer is in [lo, hi]
  const int lane = threadIdx.x % 64;
  while (hi > lo) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const bool less = at < hi && keys[at] < key;
    const int below = __popcll(__ballot(less));      // keys ascend: the first lanes
    if (below == 0) return lo;
    const int from = lo + (below - 1) * step + 1;
    hi = min(hi, lo + below * step);
    lo = from;
  }
  return lo;
}

// Zeros for those of rows [v0, v0 + g.clear) that no token has.  A workgroup that
// waits for a search has to write more than a few KiB: it has eight rows of 16 KiB
// (131,072 of them, with the runs of 16384 tokens beside them, 400 us; four rows
// 415; a bit for each row, set by a launch before, in place of the search, and a
// workgroup to a row 443 for the zeros alone), and more of shorter ones (70,144 rows
// of 768 bytes: 16 us with 68 to a workgroup, 38 with eight).
template <int TT, int AC>
__device__ __forceinline__ void clear_rows(const EmbedBwdArgs& a, const RunArgs& g, int v0) {
  __shared__ int taken[kClearMost];
  const int v1 = min(a.vocab, v0 + g.clear);
  taken[threadIdx.x] = 0;
  __syncthreads();
  const int from = lower_bound(g.keys, g.sorted, v0), to = lower_bound(g.keys, g.sorted, v1);
  for (int i = from + (int)threadIdx.x; i < to; i += 256) taken[g.keys[i] - v0] = 1;
  __syncthreads();
  // 16 bytes to a thread where rows are aligned, else a unit: neighbouring threads
  // next to each other, and several short rows at a time
  constexpr int kV = AC != 0 ? 16 / ElemSize<TT>::value : kU;
  const int vecs = (a.hidden + kV - 1) / kV;
  const int sub = vecs < 256 ? (int)threadIdx.x / vecs : 0, subs = vecs < 256 ? 256 / vecs : 1;
  if (sub >= subs) return;
  for (int v = v0 + sub; v < v1; v += subs) {
    if (taken[v - v0]) continue;
    const int r = piece_of(a.cut, v);
    const int64_t row = (int64_t)(v - piece_lo(a.cut, r)) * a.hidden;
    u32x4* at = reinterpret_cast<u32x4*>(static_cast<char*>(a.table.b[r]) + row * ElemSize<TT>::value);
    for (int j = (int)threadIdx.x - sub * vecs; j < vecs; j += 256) {
      if constexpr (AC != 0) at[j] = u32x4{0, 0, 0, 0};
      else store_cut<TT, AC>(a.table.b[r], row, unit_cut<AC>(j, a.hidden), Unit<TT>{});
    }
  }
}

template <int DT, int TT, int AC>
__global__ __launch_bounds__(256) void k_embed_runs(EmbedBwdArgs a, RunArgs g) {
  const int stretch = blockIdx.x / g.columns, j = blockIdx.x % g.columns * 256 + threadIdx.x;
  if (stretch >= g.stretches) {
    clear_rows<TT, AC>(a, g, ((int)blockIdx.x - g.stretches * g.columns) * g.clear);
    return;
  }
  const int lo = stretch * kRun, n = min(g.sorted - lo, kRun), lane = threadIdx.x % 64;
  // the stretch's keys with the one before and the one behind, and its positions:
  // one load each, a lane to a key
  const int near = lo - 1 + lane;
  const int keys = lane < n + 2 && near >= 0 && near < g.sorted ? g.keys[near] : -1;
  const int places = lane < n ? g.pos[lo + lane] : 0;
  // A wave stays whole as long as any lane has a unit: keys and places are read from
  // lanes, and what a lane that has left holds may be anything.  (All of them read into
  // scalars before lanes leave: 14 scalars of the odd-row kernels do not fit.)
  if ((j - lane) * kU >= a.hidden) return;
  const bool in = j * kU < a.hidden;
  const Cut u = unit_cut<AC>(in ? j : (a.hidden - 1) / kU, a.hidden);
  // all the stretch's rows at once
  Unit<DT> rows[kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k)
    rows[k] = load_cut<DT, AC>(a.dy, (int64_t)__builtin_amdgcn_readlane(places, k < n ? k : 0) * a.hidden, u);
  float sum[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) sum[i] = 0.0f;
  bool open = __builtin_amdgcn_readlane(keys, 0) == __builtin_amdgcn_readlane(keys, 1);   // began earlier
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int key = __builtin_amdgcn_readlane(keys, k + 1), next = __builtin_amdgcn_readlane(keys, k + 2);
    if (k < n && key < a.vocab) {
      unit_add<DT>(sum, rows[k]);
      if (k + 1 == n || next != key) {
        if (open || next == key) {
          const int64_t slot = ((int64_t)stretch * 2 + (open ? 0 : 1)) * a.hidden;
          if (in) store_cut<1, AC>(g.part, slot, u, unit_make<1>(sum));
        } else if (in) {
          put_row<TT, AC>(a, key, u, sum);
        }
        open = false;
#pragma unroll
        for (int i = 0; i < kU; ++i) sum[i] = 0.0f;
      }
    }
  }
}

// Runs that cross stretches: the stretch a run begins in adds up its parts, its
// own first, then the following stretches' first parts.  64 units of the row to a
// workgroup, four threads to a unit that take every fourth part: the run of a
// frequent token has many.
constexpr int kJoinUnits = 64;
template <int TT, int AC>
__global__ __launch_bounds__(256) void k_embed_join(EmbedBwdArgs a, RunArgs g) {
  __shared__ float lds[3][kU][kJoinUnits];
  const int columns = (a.hidden + kJoinUnits * kU - 1) / (kJoinUnits * kU);
  const int stretch = blockIdx.x / columns, x = threadIdx.x % kJoinUnits, y = threadIdx.x / kJoinUnits;
  const int j = blockIdx.x % columns * kJoinUnits + x;
  const int lo = stretch * kRun, hi = lo + kRun;
  if (hi >= g.sorted) return;                       // the last stretch: nothing follows
  const int key = g.keys[hi - 1];
  if (key >= a.vocab || g.keys[hi] != key) return;
  // it began before this stretch, which all belongs to it
  if (lo > 0 && g.keys[lo] == key && g.keys[lo - 1] == key) return;
  // where it ends: the place after its last position (whole waves search)
  const int end = lower_bound(g.keys, g.sorted, key + 1);
  const int parts = (end - 1) / kRun - stretch + 1;
  const bool in = j * kU < a.hidden;
  const Cut u = unit_cut<AC>(j, a.hidden);
  float sum[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) sum[i] = 0.0f;
  if (in) {
#pragma unroll 4
    for (int s = y; s < parts; s += 4)
      unit_add<1>(sum, load_cut<1, AC>(g.part, ((int64_t)(stretch + s) * 2 + (s == 0 ? 1 : 0)) * a.hidden, u));
  }
  if (y > 0) {
#pragma unroll
    for (int i = 0; i < kU; ++i) lds[y - 1][i][x] = sum[i];
  }
  __syncthreads();
  if (y > 0 || !in) return;
#pragma unroll
  for (int i = 0; i < kU; ++i) sum[i] += lds[0][i][x] + (lds[1][i][x] + lds[2][i][x]);
  put_row<TT, AC>(a, key, u, sum);
}

}  // namespace

// ---------------------------------------------------------------- launches

template <int DT, int G>
static hipError_t embed_go(const EmbedArgs& args, int access, hipStream_t s) {
  constexpr int64_t kMost = 1ll << 20;      // x blocks; with y the dispatch counts 32 bits of threads
  EmbedArgs a = args;
  const int units = (a.hidden + kU - 1) / kU, cols = (units + G - 1) / G;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMost, 0xFFFFFFFFll / 256 / cols));
  for (; a.row0 < a.tokens; a.row0 += most * (256 / G) * kTokens) {
    const dim3 grid((unsigned)std::min<int64_t>(most, (a.tokens - a.row0 + 256 / G * kTokens - 1) / (256 / G * kTokens)), cols);
    if (access == kStreamRows) k_embed<DT, G, kStreamRows><<<grid, 256, 0, s>>>(a);
    else if (access == kAlignedRows) k_embed<DT, G, kAlignedRows><<<grid, 256, 0, s>>>(a);
    else k_embed<DT, G, kOddRows><<<grid, 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
static hipError_t embed_size(const EmbedArgs& a, int access, hipStream_t s) {
  const int units = (a.hidden + kU - 1) / kU;
  return units <= 64 ? embed_go<DT, 64>(a, access, s) : embed_go<DT, 256>(a, access, s);
}

hipError_t launch_embed(const EmbedArgs& a, int dtype, int access, hipStream_t s) {
  if (dtype == 1) return embed_size<1>(a, access, s);
  if (dtype == 2) return embed_size<2>(a, access, s);
  return embed_size<3>(a, access, s);
}

// The workspace: sorted keys and positions (twice where the sort takes passes),
// the passes' counts, the open runs' sums.  Each part starts on 16 bytes.
static int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }
static int tile_of(int64_t tokens) { return tokens <= kSmallMost ? kSmallTile : kLargeTile; }
static int sort_blocks(int64_t tokens) {
  return tokens <= kCountMost ? 0 : (int)((tokens + tile_of(tokens) - 1) / tile_of(tokens));
}
static int64_t stretches_of(int64_t tokens) { return (tokens + kRun - 1) / kRun; }

int64_t embed_bwd_words(int64_t tokens, int hidden) {
  const int64_t blocks = sort_blocks(tokens);
  return (blocks ? 4 : 2) * up4(tokens) + blocks * kBins + stretches_of(tokens) * 2 * hidden;
}

static int columns_of(int hidden, int units) { return (hidden + units * kU - 1) / (units * kU); }

// Rows to a workgroup that clears: 65,536 elements of them, but 1024 workgroups if there
// are rows for that, and eight at least.
static int clear_of(int vocab, int hidden) {
  const int most = std::min({kClearMost, 65536 / hidden, std::max(vocab / 1024, 8)});
  return std::max(most, 8);
}

// One dispatch counts threads in 32 bits.
bool embed_bwd_fits(int64_t tokens, int vocab, int hidden) {
  return tokens < (1ll << 31) - kLargeTile &&
         stretches_of(tokens) * columns_of(hidden, kJoinUnits) + (vocab + 7) / 8 <=
             0xFFFFFFFFll / 256;
}

template <int DT, int TT>
static hipError_t runs_go(const EmbedBwdArgs& a, const RunArgs& g, bool al, hipStream_t s) {
  const int clears = a.accumulate ? 0 : (a.vocab + g.clear - 1) / g.clear;
  const unsigned grid = (unsigned)(g.stretches * g.columns + clears);
  if (grid == 0) return hipSuccess;
  if (al) k_embed_runs<DT, TT, kAlignedRows><<<grid, 256, 0, s>>>(a, g);
  else k_embed_runs<DT, TT, kOddRows><<<grid, 256, 0, s>>>(a, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.stretches < 2) return e;
  const unsigned joins = (unsigned)((g.stretches - 1) * columns_of(a.hidden, kJoinUnits));
  if (al) k_embed_join<TT, kAlignedRows><<<joins, 256, 0, s>>>(a, g);
  else k_embed_join<TT, kOddRows><<<joins, 256, 0, s>>>(a, g);
  return hipGetLastError();
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, int dtype, int table_dtype, bool al, hipStream_t s) {
  const int64_t n = a.tokens, blocks = sort_blocks(n);
  int* keys = a.work;
  int* pos = keys + up4(n);
  int* spare_keys = pos + up4(n);
  int* spare_pos = spare_keys + up4(n);
  int* hist = spare_pos + up4(n);
  RunArgs g = {};
  g.part = reinterpret_cast<float*>(blocks ? hist + blocks * kBins : spare_keys);
  if (n > 0 && blocks == 0) {
    k_sort_count<<<(unsigned)((n + 63) / 64), kCountThreads, 0, s>>>(a, keys, pos);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else if (n > 0) {
    int bits = 1;
    while ((a.vocab >> bits) != 0) ++bits;          // keys are 0 .. vocab
    SortIn in = {nullptr, nullptr};
    for (int shift = 0; shift < bits; shift += kBits) {
      if (tile_of(n) == kSmallTile) {
        k_sort_hist<2><<<(unsigned)blocks, kSortThreads, 0, s>>>(a, in, shift, hist);
        k_sort_place<2><<<(unsigned)blocks, kSortThreads, 0, s>>>(a, in, shift, hist, (int)blocks, keys, pos);
      } else {
        k_sort_hist<8><<<(unsigned)blocks, kSortThreads, 0, s>>>(a, in, shift, hist);
        k_sort_place<8><<<(unsigned)blocks, kSortThreads, 0, s>>>(a, in, shift, hist, (int)blocks, keys, pos);
      }
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      in = {keys, pos};
      std::swap(keys, spare_keys);
      std::swap(pos, spare_pos);
    }
    keys = const_cast<int*>(in.keys);
    pos = const_cast<int*>(in.pos);
  }
  g.keys = keys;
  g.pos = pos;
  g.sorted = (int32_t)n;
  g.stretches = (int32_t)stretches_of(n);
  g.columns = columns_of(a.hidden, 256);
  g.clear = clear_of(a.vocab, a.hidden);
  if (dtype == 1) return runs_go<1, 1>(a, g, al, s);
  if (dtype == 2) return table_dtype == 1 ? runs_go<2, 1>(a, g, al, s) : runs_go<2, 2>(a, g, al, s);
  return table_dtype == 1 ? runs_go<3, 1>(a, g, al, s) : runs_go<3, 3>(a, g, al, s);
}

}  // namespace ra
