// ra_internal.h -- interface between the host API (ra_api.cpp) and the kernel
// launchers in the .hip files, plus small host helpers.
// Not installed; the public ABI is include/ra.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ra_elem.h"

namespace ra {

struct WsHeader;

// Kernel families of the step-by-step schedule run by launch_steps().
enum StepMode { kModeRing = 0, kModeBidir = 1, kModeTree = 2, kModeHier = 3 };

// What the step and pipelined launchers need besides the data.
struct SyncCfg {
  WsHeader* ws;           // device workspace of this (device, stream); null when the call
                          // cannot run a persistent grid (its launches have no waits)
  uint64_t limit_ticks;   // bound of one device-side wait, device clock ticks
  uint32_t expect_extra;  // 1 = first wait expects an arrival that never comes (test hook)
  uint32_t stress;        // nonzero: pseudo-random delays before arrivals and hops (test hook)
  uint64_t* step_ts;      // optional device array of step timestamps
  int grid;               // 0 = as many workgroups as are co-resident
  int channels;           // step kernels: independent channels (1 = whole grid, 0 = automatic)
  int group;              // kModeHier: ranks per node g (g divides p)
  bool may_probe;         // may run (and allocate for) the one-time XCD placement probe;
                          // false: an unprobed device counts as unplaced
};

// Launch descriptions return the number of workgroups used through *grid_used.

// Whether a one-pass call runs with read and write phases (k_fused_phased):
// where the library finds it pays, always where the grid fits, or never.
enum PhaseMode { kPhasesAuto = 0, kPhasesForce = 1, kPhasesOff = 2 };

// One pass: each element folded in its chunk's ring order with reduction `op`
// (wide: accumulated in the wider type).  mode 0 stores the result to all ranks
// (all-reduce), 1 only to the chunk's owner (reduce-scatter), 2 copies each
// owner's chunk to the other ranks (all-gather; op and wide unused).  phases: a
// PhaseMode.
hipError_t launch_fused(const RankPtrs& P, int p, int64_t n, int dtype, int op, bool wide,
                        int mode, int phases, hipStream_t s, int* grid_used);

// Steps [step_begin, step_end) of a step-by-step schedule, in order.  Steps
// that move at most 256 vectors run on one workgroup (its own barrier between
// steps); larger ones as one launch per step, or -- when sc asks for a grid,
// channels, step timestamps or a test hook -- as one persistent cooperative
// launch with a grid barrier between steps.  Ring/bidir: steps 0..p-2
// reduce-scatter, p-1..2p-3 all-gather.  Tree: L reduce levels then L broadcast
// levels.  Hier (g = sc.group, m = p / g): g-1 intra-node reduce-scatter steps,
// 2(m-1) inter-node all-reduce steps on the shards, g-1 intra-node all-gather
// steps.
hipError_t launch_steps(const RankPtrs& P, int p, int64_t n, int dtype, int op, StepMode mode,
                        int step_begin, int step_end, const SyncCfg& sc, hipStream_t s,
                        int* grid_used, int* launches);

// One pass in the two-level order: node partials folded over local ranks,
// then folded over nodes (g ranks per node), stored to every rank.
hipError_t launch_fused_hier(const RankPtrs& P, int p, int64_t n, int dtype, int op, int g,
                             hipStream_t s, int* grid_used);

// Hops [hop_begin, hop_end) of the forward ring with chunks cut into slices of
// `slice` elements and per-slice ready counters in `flags` (p * kmax entries,
// all <= `base` on entry).
hipError_t launch_pipelined(const RankPtrs& P, int p, int64_t n, int dtype, int op, int hop_begin,
                            int hop_end, int64_t slice, int64_t kmax, uint32_t* flags,
                            uint32_t base, const SyncCfg& sc, hipStream_t s, int* grid_used);

// The pipelined ring with every slice carried through all its hops by one
// workgroup (no flags, no barriers).  mode 0: all-reduce, 1: reduce-scatter
// (leaves the step-by-step partials), 2: all-gather.  slice_elems 0 = one tile
// (kBlock vectors) per slice; stress != 0 adds the test hook's delays.
hipError_t launch_rider(const RankPtrs& P, int p, int64_t n, int dtype, int op, int mode,
                        int64_t slice_elems, uint32_t stress, hipStream_t s, int* grid_used);

// Slices per chunk for the pipelined kernel (the host sizes `flags` with it).
int64_t pipelined_slices_per_chunk(int p, int64_t n, int dtype, int64_t slice);

// Slice length used when the caller does not choose one.
int64_t pipelined_default_slice(int p, int64_t n, int dtype, int grid_override);

// dst[0 .. count) = value, a kernel on stream s (a fill that a graph capture
// records as a kernel, not as a memset).
hipError_t launch_fill_u32(uint32_t* dst, uint32_t value, int64_t count, hipStream_t s);

// Plain streaming copy (measurement helpers): one-shot grid, and a resident
// grid of `grid` workgroups looping over tiles handed out in order from tile
// counters at ctr (8 of them, 32 words apart; zeroed here, on s).
hipError_t launch_copy(void* dst, const void* src, int64_t bytes, hipStream_t s);
hipError_t launch_copy_resident(void* dst, const void* src, int64_t bytes, int grid,
                                uint32_t* ctr, hipStream_t s);

// Workgroups a persistent step kernel runs by default on the current device.
int default_persistent_workgroups();

// ---------------------------------------------------------------- row operators
// What a tensor-parallel model does where it folds its ranks' buffers.  `al`:
// every row of every array starts on a 16-byte boundary (and its length is a
// multiple of 8).  `access`: an Access of ra_rows.h.

struct NormArgs {
  RankPtrs in, out, scale;   // scale: used by 8-bit outputs
  const void* res;           // or null
  void* res_out;             // or null
  const void* weight;
  float* rstd;               // or null
  int64_t tokens, row0;
  int32_t hidden, p, n_out, group;
  float eps, inv_h;
};

struct NormBwdArgs {
  RankPtrs in, dx;
  const void* h;
  const float* rstd;
  const void* weight;
  const void* dh_in;         // or null
  void* dh;
  float* part;               // [norm_bwd_blocks()][hidden]: the workgroups' sums for dw, or null
  int64_t tokens;
  int32_t hidden, p, n_dx;
  float inv_h;
};

// Rows longer than this would not stay in the registers of one workgroup.
constexpr int kNormMaxHidden = 32768;

// Workgroups of the backward pass: two for each of 256 compute units.  Those of 1024
// threads run one after the other, since they take more than the 64 registers that
// would let two of them share a unit.  A constant, so that the order in which dw is
// summed does not depend on the GPU.
constexpr int kNormBwdBlocks = 512;

hipError_t launch_norm(const NormArgs& a, int dtype, int res_dtype, bool f8, int access, hipStream_t s);
int norm_bwd_blocks(int64_t tokens);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int h_dtype, float* dweight, int access,
                           hipStream_t s);

// How a length (a vocabulary) is cut over the ranks.
struct Pieces {
  int32_t base;    // floor(n / p)
  int32_t extra;   // n mod p: the first `extra` pieces hold one more
};

// Logits whose vocabulary is cut over the ranks.
struct VocabArgs {
  RankPtrs x, dx;            // the ranks' logits; their gradients (dx.b[0..p) null: not wanted)
  int64_t tokens, row0;
  Pieces cut;
  int32_t p, vocab, valid, splits;
  // set by vocab_geometry() from cut, p, vocab and valid:
  int32_t whole;             // chunks of 512 columns in a piece
  int32_t total;             // chunks of a row: those, and what is left of each piece
  int32_t full;              // the first chunks, all of whose columns are valid
  uint32_t magic;            // ceil(2^32 / whole): q / whole = (q magic) >> 32 while q whole < 2^32
};
int vocab_chunks(int vocab, int p);
void vocab_geometry(VocabArgs* a);

struct XentArgs : VocabArgs {
  const void* target;
  const float* dloss;        // or null: 1 for every token
  const float* lse_in;       // backward only
  float* loss;
  float* lse;
  float* part;               // split rows: xent_words() of workspace
  int32_t target64;
  float grad_scale;
};

// Workgroups that share a row, 1 where a workgroup takes a whole row.
int xent_splits(int64_t tokens, int vocab, int p, bool grad);
int64_t xent_words(int64_t tokens, int splits);   // 32-bit words of workspace

// Columns of a vocabulary: chunk numbers times chunks stay below 2^32.
constexpr int kXentMaxVocab = 1 << 24;
hipError_t launch_xent(const XentArgs& a, int dtype, bool grad, bool al, hipStream_t s);
hipError_t launch_xent_bwd(const XentArgs& a, int dtype, bool al, hipStream_t s);

struct LogpArgs : VocabArgs {
  const void* ids;           // or null: none wanted
  float* logprob;            // these five or null
  float* entropy;
  float* lse;
  void* top_ids;
  float* top_logprobs;
  const float* lse_in;       // backward only, as the next three
  const float* entropy_in;
  const float* dlogprob;     // or null
  const float* dentropy;     // or null
  float* part;               // split rows: logp_bytes() of workspace
  int32_t ids64, top;
  float scale;
};
constexpr int kTopMost = 64;   // a lane for each
int logp_splits(int64_t tokens, int vocab, int p);
int64_t logp_bytes(int64_t tokens, int splits, int top);
hipError_t launch_logp(const LogpArgs& a, int dtype, int access, hipStream_t s);
hipError_t launch_logp_bwd(const LogpArgs& a, int dtype, bool al, bool big, hipStream_t s);   // big: more than the caches hold

struct EmbedArgs {
  RankPtrs table, out;
  const void* ids;
  int64_t tokens;
  Pieces cut;
  int64_t row0;
  int32_t p, vocab, hidden, n_out, ids64;
  float scale;
};
hipError_t launch_embed(const EmbedArgs& a, int dtype, int access, hipStream_t s);

struct EmbedBwdArgs {
  RankPtrs table;            // the ranks' gradients
  const void* dy;
  const void* ids;
  int32_t* work;             // see embed_bwd_words
  int64_t tokens;
  Pieces cut;
  int32_t p, vocab, hidden, ids64, accumulate;
  float scale;
};
int64_t embed_bwd_words(int64_t tokens, int hidden);   // 32-bit words of workspace
bool embed_bwd_fits(int64_t tokens, int vocab, int hidden);

// Elements of an embedding's row (columns of workgroups in one dispatch).
constexpr int kEmbedMaxHidden = 1 << 20;
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, int dtype, int table_dtype, bool al, hipStream_t s);

// ---------------------------------------------------------------- gradients

// A caller's list.
struct TensorListArgs {
  const void* const* in;
  void* const* out;          // null: not written
  const int64_t* counts;
  const int* types;
  const int* out_types;      // null: the same
  int64_t n, counted;        // the first `counted` make the norm
  bool stream;               // larger than the caches
};

// How a norm and a factor come from the sum of squares.
struct ClipRule {
  const double* part;        // `parts` sums
  const float* factor;       // two floats, or null: from the parts
  float* norm;
  int32_t parts;
  float max_norm, scale;
};

struct FoldArgs {
  RankPtrs in, out;
  int64_t n;
  int32_t p, n_out, mean;
};

int64_t grad_norm_bytes(int64_t n);        // of workspace, for n tensors
int64_t fold_clip_bytes(int64_t n);        // ... for n elements
hipError_t launch_grad_norm(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s);
hipError_t launch_grad_clip(const TensorListArgs& a, ClipRule r, void* work, hipStream_t s);
hipError_t launch_fold_clip(const FoldArgs& a, int dtype, const ClipRule& r, bool stream, void* work, hipStream_t s);

// ---------------------------------------------------------------- errors
// Sets the calling thread's error message and returns `code` (ra_api.cpp).
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail_hip(hipError_t e, const char* what);
bool debug_on();

// ---------------------------------------------------------------- host helpers

inline int elem_bytes(int dtype) {
  switch (dtype) {
    case 2: case 3: return 2;
    case 4: case 5: return 8;
    default: return 4;
  }
}

inline int elems_per_vec(int dtype) { return 16 / elem_bytes(dtype); }

// Whole 16-byte vectors inside [lo, hi) (host mirror of split_span).
inline int64_t vecs_in(int64_t lo, int64_t hi, int V) {
  int64_t a0 = (lo + V - 1) / V * V;
  int64_t a1 = hi / V * V;
  return a1 > a0 ? (a1 - a0) / V : 0;
}

// Vectors the tiles of [lo, hi) span, counted from the line their first tile
// starts on (Span::vb): the whole vectors plus up to kLineVecs - 1 before them.
inline int64_t tiled_vecs_in(int64_t lo, int64_t hi, int V) {
  int64_t a0 = (lo + V - 1) / V, a1 = hi / V;
  return a1 > a0 ? a1 - a0 / kLineVecs * kLineVecs : 0;
}

// Whether a segment of `vecs` tiled vectors ends in a tile (of `tile` vectors)
// at most half full: then launches number every segment's last tile after the
// others (tile_of in ra_elem.h).  Fuller last tiles gain nothing from it (p = 64
// with 15,625 bfloat16 per chunk, last tiles 62% full: 53.4 against 52.2 us).
inline int short_tail(int64_t vecs, int64_t tile) {
  const int64_t rem = vecs % tile;
  return rem != 0 && 2 * rem <= tile;
}

// The most workgroups of 256 threads an MI355X holds at once (256 compute units,
// 8 each).  Up to that many, a launch's workgroups are all placed in the first
// rounds of the dispatcher, and which compute unit gets which tile is decided by
// their order; beyond it, workgroups wait for free slots and the order of the
// short tiles no longer decides anything (launches keep the plain order).
constexpr int64_t kResidentTiles = 2048;

// Where a launch's edge workgroups sit in its workgroup order (e0):
// first, so their chains of round trips start at once, or -- when the segments'
// last tiles are short (tail_last) -- right after the other tiles and before the
// short ones, so that the first round of compute units gets whole tiles and the
// edge workgroups share the second round with the short tiles.  Measured at
// p = 64 (one-pass all-reduce, us): 524,365 bfloat16 per rank (short last tiles)
// 30.4-30.8 with the edge workgroups placed so (31.4 with them first, and the
// short tiles numbered like the others); 1,000,003 (last tiles 62% full) 52.6-54.5
// with them first against 55.4-56.7 with them last.
inline int64_t edge_start(int64_t ntiles, int64_t nseg, int tail_last, int edges, int64_t grid) {
  const int64_t after_whole = ntiles - nseg;          // the tiles before the short ones
  return tail_last && after_whole + edges <= grid ? after_whole : 0;
}

inline int64_t host_chunk_lo(int64_t off, int64_t len, int p, int c) {
  int64_t base = len / p, extra = len % p;
  return off + (int64_t)c * base + std::min<int64_t>(c, extra);
}

inline ChunkGeo make_geo(int64_t off, int64_t len, int p) {
  ChunkGeo g;
  g.off = off;
  g.base = len / p;
  g.extra = len % p;
  return g;
}

// Buffers larger than this in total (p * S) are streamed with non-temporal
// loads and stores: they are far beyond the 256 MB Infinity Cache, and the
// streaming hint measured +3.7% for the fused kernel at 8 x 16 GiB.  Smaller
// working sets keep normal caching so that repeated calls can hit the cache.
constexpr int64_t kStreamingBytes = 512ll << 20;

inline bool streaming(int p, int64_t n, int dtype) {
  return (int64_t)p * n * elem_bytes(dtype) > kStreamingBytes;
}

// Non-persistent grids are capped here; beyond it, workgroups loop over tiles.
// The dispatch counts the grid in work-items in 32 bits, so this is the largest
// grid of kBlock-thread workgroups there is.  A grid that covers the data once
// streams faster than one that loops: the tree at 8 x 16 GB (whole-buffer steps
// of up to 15.6 million tiles) took 89.9 ms against 91.1 with a cap of 2^22.
constexpr int64_t kMaxGrid = 0xFFFFFFFFll / kBlock;

}  // namespace ra
