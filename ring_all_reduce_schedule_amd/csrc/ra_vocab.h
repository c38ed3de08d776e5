// ra_vocab.h -- rows of logits whose vocabulary is cut over the ranks: how a
// workgroup's waves share a row, and how their lanes read and write it (cross
// entropy, log probabilities).
#pragma once

#include "ra_rows.h"

namespace ra {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }

// A row's units over all ranks go in chunks of 64, one to each lane of a wave; a
// chunk lies in one piece, so that its pointers are the wave's and not the lanes'.
// First come the chunks of whole 512 columns, a.whole of each piece, in the order
// of their columns; then what is left of each piece, if anything is.
struct Chunk {
  int r;        // piece (rank)
  int len;      // the piece's columns
  int c0;       // the chunk's first column in its piece
  int col0;     // ... and in the vocabulary
};
constexpr int kChunk = 64 * kU;

__device__ __forceinline__ Chunk chunk_of(const VocabArgs& a, int q) {
  Chunk s;
  const int wholes = a.whole * a.p;
  if (q < wholes) {
    s.r = a.whole == 1 ? q : (int)__umulhi((uint32_t)q, a.magic);
    s.c0 = (q - s.r * a.whole) * kChunk;
  } else {
    s.r = q - wholes;
    s.c0 = a.whole * kChunk;
  }
  s.len = piece_len(a.cut, s.r);
  s.col0 = piece_lo(a.cut, s.r) + s.c0;
  return s;
}

// A wave's chunk.
__device__ __forceinline__ Chunk chunk(const VocabArgs& a, int q) {
  // Computed where it is used: kept over a row's passes, the places of sixteen
  // chunks would not fit the scalar registers.
  asm volatile("" : "+s"(q));
  return chunk_of(a, q);
}

// How a kernel reads and writes units.
enum Mode {
  kAligned,   // rows of whole units on 16-byte boundaries
  kStream,    // those, past the caches
  kOdd,       // any rows of pieces of at least a unit
  kTiny       // pieces shorter than a unit are among them: element by element
};

constexpr int access_of(int mode) { return mode == kStream ? kStreamRows : mode == kAligned ? kAlignedRows : kOddRows; }

// The lane's unit of a chunk: it loads elements [c, c + 8) of the piece's row,
// and its own are those from `from` on that the piece has.  The unit that would
// pass the row's end is moved back to end there, and so are the units of lanes
// behind it, which then own nothing: every lane loads without a branch.
struct Lane {
  int c, from;
};
template <int MODE>
__device__ __forceinline__ Lane lane_of(const Chunk& s, int lane) {
  const int from = s.c0 + lane * kU;
  if (MODE == kTiny) return {from, from};
  return {min(from, s.len - kU), from};
}
template <int MODE>
__device__ __forceinline__ Lane lane_of(const Chunk& s) { return lane_of<MODE>(s, (int)(threadIdx.x % 64)); }

// Which elements count: the lane's own, before the first column that is not valid.
__device__ __forceinline__ bool counts(const Chunk& s, const Lane& l, int valid, int i) {
  return l.c + i >= l.from && l.c + i < s.len && s.col0 - s.c0 + l.c + i < valid;
}

// Element i of a unit becomes -inf.
template <int DT>
__device__ __forceinline__ void mask_out(Unit<DT>* t, int i) {
  if constexpr (DT == 1) {
    t->v[i / 4][i % 4] = 0xff800000u;
  } else {
    const uint32_t ninf = DT == 2 ? 0xff80u : 0xfc00u;
    const uint32_t w = t->v[0][i / 2];
    t->v[0][i / 2] = i % 2 ? (w & 0xffffu) | ninf << 16 : (w & 0xffff0000u) | ninf;
  }
}

// The lane's unit of a chunk, as memory holds it, of the piece at p.
template <int DT, int MODE>
__device__ __forceinline__ Unit<DT> fetch_of(const void* p, int64_t row, const Chunk& s, const Lane& l) {
  const char* x = static_cast<const char*>(p) + row * s.len * ElemSize<DT>::value;
  if constexpr (MODE != kTiny) {
    return load_unit<DT, access_of(MODE)>(x, l.c);
  } else {
    return load_cut<DT, false>(x, 0, {l.c, 0, max(0, min(kU, s.len - l.c))});
  }
}

template <int DT, int MODE>
__device__ __forceinline__ Unit<DT> fetch(const VocabArgs& a, int64_t row, const Chunk& s) {
  return fetch_of<DT, MODE>(a.x.b[s.r], row, s, lane_of<MODE>(s));
}

// ... with -inf for what does not count: the first a.full chunks count as a whole.
template <int DT, int MODE>
__device__ __forceinline__ void mask(Unit<DT>* t, const VocabArgs& a, int q, const Chunk& s) {
  if (q < a.full) return;
  const Lane l = lane_of<MODE>(s);
#pragma unroll
  for (int i = 0; i < kU; ++i)
    if (!counts(s, l, a.valid, i)) mask_out<DT>(t, i);
}

template <int DT>
__device__ __forceinline__ void mask_all(Unit<DT>* t) {
#pragma unroll
  for (int i = 0; i < kU; ++i) mask_out<DT>(t, i);
}

// The masked units of N chunks q0, q0 + step, ...; -inf from chunk `end` on.  All
// loads go out before the first is looked at.
template <int DT, int MODE, int N>
__device__ __forceinline__ void fetch_all(Unit<DT>* u, const VocabArgs& a, int64_t row, int q0, int step, int end) {
#pragma unroll
  for (int k = 0; k < N; ++k) u[k] = fetch<DT, MODE>(a, row, chunk(a, min(q0 + k * step, end - 1)));
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int q = q0 + k * step;
    if (q < end) mask<DT, MODE>(&u[k], a, q, chunk(a, q));
    else mask_all<DT>(&u[k]);
  }
}

// Keeps the compiler from holding on to a unit's unpacked values: they would take
// twice the unit's registers from one pass over it to the next.
template <int DT>
__device__ __forceinline__ void forget(Unit<DT>* t) {
  asm volatile("" : "+v"(t->v[0]));
  if constexpr (DT == 1) asm volatile("" : "+v"(t->v[1]));
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// The target's logit; not read where there is none.
template <int DT>
__device__ __forceinline__ float logit(const VocabArgs& a, int64_t row, int y) {
  if (y < 0) return 0.0f;
  const int r = piece_of(a.cut, y);
  const typename Elem<DT>::S* x = static_cast<const typename Elem<DT>::S*>(a.x.b[r]);
  const int64_t at = row * piece_len(a.cut, r) + (y - piece_lo(a.cut, r));
  if constexpr (DT == 1) return __uint_as_float(x[at]);
  else return Elem<DT>::to_w(x[at]);
}

// Writes a lane's own elements of a chunk's gradient.  WHOLE: 512 columns.
template <int DT, int MODE, bool WHOLE>
__device__ __forceinline__ void put(const VocabArgs& a, int64_t row, const Chunk& s, const Lane& l, const Unit<DT>& t) {
  char* dx = static_cast<char*>(a.dx.b[s.r]) + row * s.len * ElemSize<DT>::value;
  if (WHOLE) {
    store_unit<DT, access_of(MODE)>(dx, l.from, t);
  } else if (l.from < s.len) {
    store_cut<DT, access_of(MODE)>(dx, 0, {l.c, l.from - l.c, min(kU, s.len - l.c)}, t);
  }
}

}  // namespace ra
