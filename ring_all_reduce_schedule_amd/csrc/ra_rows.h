// ra_rows.h -- what the row operators (norm, cross entropy, embedding) share:
// eight consecutive elements of a row as the unit a lane moves, their values in
// float32, and reductions over a wave or a workgroup.
//
// A lane's eight elements are one 16-byte access for the 16-bit types and two
// for float32.  Rows need not start on a 16-byte boundary (an odd row length
// puts every second row of 16-bit elements 2 bytes off): the kOddRows forms
// promise the compiler the element's own alignment only, for which gfx950 issues
// the same 16-byte accesses.  Large calls stream past the caches.  Where the last unit of a row would pass its end,
// it is moved back to end there: it loads a whole unit, of which its first
// elements belong to the unit before it and count as absent.  (One load instead
// of up to seven: they would be one round trip to memory for each rank.)
#pragma once

#include "ra_elem.h"
#include "ra_internal.h"

namespace ra {

constexpr int kU = 8;   // elements of a unit

// Piece r of a length cut over the ranks, and the piece that holds element i.
__device__ __forceinline__ int piece_len(const Pieces& c, int r) { return c.base + (r < c.extra ? 1 : 0); }
__device__ __forceinline__ int piece_lo(const Pieces& c, int r) {
  return r * c.base + (r < c.extra ? r : c.extra);
}
__device__ __forceinline__ int piece_of(const Pieces& c, int i) {
  const int cut = c.extra * (c.base + 1);
  return i < cut ? i / (c.base + 1) : c.extra + (i - cut) / c.base;
}

// Storage of a unit.
template <int DT> struct Unit {
  u32x4 v[DT == 1 ? 2 : 1];
};

template <int DT> struct ElemSize { static constexpr int value = DT == 1 ? 4 : 2; };

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));
typedef u32x2 u32x2_by1 __attribute__((aligned(1)));

// How a kernel reaches its rows: any rows; rows of whole units that start on
// 16-byte boundaries; those, past the caches (a call whose arrays together are
// larger than kStreamingBytes: norm of 4096 x 8192 bfloat16 over 8 ranks, 8-bit
// outputs, 173 us against 186, its gradient 147 against 165).
enum Access { kOddRows = 0, kAlignedRows = 1, kStreamRows = 2 };

template <int DT, bool AL> struct UnitWord;
template <> struct UnitWord<1, false> { typedef u32x4_by4 T; };
template <> struct UnitWord<2, false> { typedef u32x4_by2 T; };
template <> struct UnitWord<3, false> { typedef u32x4_by2 T; };
template <int DT> struct UnitWord<DT, true> { typedef u32x4 T; };

// Elements [i, i + 8) of the row at p.
template <int DT, int AC>
__device__ __forceinline__ Unit<DT> load_unit(const void* p, int64_t i) {
  typedef typename UnitWord<DT, AC != 0>::T W;
  const W* q = reinterpret_cast<const W*>(static_cast<const char*>(p) + i * ElemSize<DT>::value);
  Unit<DT> u;
  if constexpr (AC == kStreamRows) {
    u.v[0] = __builtin_nontemporal_load(q);
    if constexpr (DT == 1) u.v[1] = __builtin_nontemporal_load(q + 1);
  } else {
    u.v[0] = q[0];
    if constexpr (DT == 1) u.v[1] = q[1];
  }
  return u;
}

// Unit j of a row of `len` elements: it loads elements [c, c + 8), of which
// [c + lo, c + hi) are its own.  hi < 8 only in rows shorter than a unit.
struct Cut {
  int c, lo, hi;
};
template <int AC>
__device__ __forceinline__ Cut unit_cut(int j, int len) {
  const int c = j * kU;
  if (AC != 0 || c + kU <= len) return {c, 0, kU};
  if (len >= kU) return {len - kU, c + kU - len, kU};
  return {0, 0, len};
}
template <int AC>
__device__ __forceinline__ bool owns(const Cut& u, int i) { return AC != 0 || (i >= u.lo && i < u.hi); }

// Unit u of the row that starts at element `row` of p.  What is not its own is
// whatever memory holds (in rows shorter than a unit: zero).
template <int DT, int AC>
__device__ __forceinline__ Unit<DT> load_cut(const void* p, int64_t row, const Cut& u) {
  if (AC != 0 || u.hi == kU) return load_unit<DT, AC>(p, row + u.c);
  typedef typename Elem<DT>::S S;
  const S* q = static_cast<const S*>(p) + row;
  Unit<DT> x{};
#pragma unroll
  for (int k = 0; k < kU - 1; ++k) {
    if (k < u.hi) {
      if constexpr (DT == 1) x.v[k / 4][k % 4] = q[k];
      else x.v[0][k / 2] |= (uint32_t)q[k] << (k % 2 * 16);
    }
  }
  return x;
}

template <int DT, int AC>
__device__ __forceinline__ void store_unit(void* p, int64_t i, const Unit<DT>& u) {
  typedef typename UnitWord<DT, AC != 0>::T W;
  W* q = reinterpret_cast<W*>(static_cast<char*>(p) + i * ElemSize<DT>::value);
  if constexpr (AC == kStreamRows) {
    __builtin_nontemporal_store(u.v[0], q);
    if constexpr (DT == 1) __builtin_nontemporal_store(u.v[1], q + 1);
  } else {
    q[0] = u.v[0];
    if constexpr (DT == 1) q[1] = u.v[1];
  }
}

// Writes a unit's own elements.
template <int DT, int AC>
__device__ __forceinline__ void store_cut(void* p, int64_t row, const Cut& u, const Unit<DT>& x) {
  if (AC != 0 || u.hi - u.lo == kU) {
    store_unit<DT, AC>(p, row + u.c, x);
    return;
  }
  typedef typename Elem<DT>::S S;
  S* q = static_cast<S*>(p) + row + u.c;
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    if (owns<AC>(u, k)) {
      if constexpr (DT == 1) q[k] = x.v[k / 4][k % 4];
      else q[k] = (S)(x.v[0][k / 2] >> (k % 2 * 16));
    }
  }
}

// Element k of a unit as float32 (exact).
template <int DT>
__device__ __forceinline__ float unit_get(const Unit<DT>& u, int k) {
  if constexpr (DT == 1) {
    return __uint_as_float(u.v[k / 4][k % 4]);
  } else if constexpr (DT == 2) {
    const uint32_t w = u.v[0][k / 2];
    return __uint_as_float(k % 2 ? w & 0xffff0000u : w << 16);
  } else {
    return f16_to_f32((uint16_t)(u.v[0][k / 2] >> (k % 2 * 16)));
  }
}

// Eight float32 values rounded (to nearest, ties to even) to a unit.
template <int DT>
__device__ __forceinline__ Unit<DT> unit_make(const float* x) {
  Unit<DT> u;
  if constexpr (DT == 1) {
#pragma unroll
    for (int k = 0; k < kU; ++k) u.v[k / 4][k % 4] = __float_as_uint(x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kU / 2; ++k) {
      const f32x2 two = {x[2 * k], x[2 * k + 1]};
      if constexpr (DT == 2) {
        u.v[0][k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
      } else {
        u.v[0][k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
      }
    }
  }
  return u;
}

// acc += u, in float32.
template <int DT>
__device__ __forceinline__ void unit_add(float* acc, const Unit<DT>& u) {
#pragma unroll
  for (int k = 0; k < kU; ++k) acc[k] += unit_get<DT>(u, k);
}

// x = sum over the ranks, in rank order from 0, of unit u of each rank's row;
// elements that are not its own as zeros.  Up to kBatch ranks' loads are in
// flight together.
template <int DT, int AC>
__device__ __forceinline__ void fold_ranks(float* x, const RankPtrs& P, int p, int64_t row, const Cut& u) {
  constexpr int kBatch = DT == 1 ? 4 : 8;
#pragma unroll
  for (int k = 0; k < kU; ++k) x[k] = 0.0f;
  int r = 0;
  for (; r + kBatch <= p; r += kBatch) {
    Unit<DT> t[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) t[b] = load_cut<DT, AC>(P.b[r + b], row, u);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) unit_add<DT>(x, t[b]);
  }
  for (; r + 2 <= p; r += 2) {
    const Unit<DT> t0 = load_cut<DT, AC>(P.b[r], row, u), t1 = load_cut<DT, AC>(P.b[r + 1], row, u);
    unit_add<DT>(x, t0);
    unit_add<DT>(x, t1);
  }
  if (r < p) unit_add<DT>(x, load_cut<DT, AC>(P.b[r], row, u));
  if constexpr (AC == 0) {
#pragma unroll
    for (int k = 0; k < kU; ++k) x[k] = owns<AC>(u, k) ? x[k] : 0.0f;
  }
}

// ---------------------------------------------------------------- reductions

// x from another lane of the same 16, by the lane pattern CTRL.  Four patterns in a
// row give every lane what all 16 have: neighbours, pairs, fours (mirrored in 8),
// eights (mirrored in 16).  They take an instruction each; a shuffle through LDS
// takes a round trip.
constexpr int kDppNeighbour = 0xB1, kDppPair = 0x4E, kDppFour = 0x141, kDppEight = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) { return __uint_as_float(dpp<CTRL>(__float_as_uint(x))); }

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

// Over 16 neighbouring lanes, the same in all of them.
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<kDppNeighbour>(x);
  x += dpp<kDppPair>(x);
  x += dpp<kDppFour>(x);
  x += dpp<kDppEight>(x);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
  x = __builtin_fmaxf(x, dpp<kDppNeighbour>(x));
  x = __builtin_fmaxf(x, dpp<kDppPair>(x));
  x = __builtin_fmaxf(x, dpp<kDppFour>(x));
  x = __builtin_fmaxf(x, dpp<kDppEight>(x));
  return x;
}
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t row_max_u32(uint32_t x) {
  x = max_u32(x, dpp<kDppNeighbour>(x));
  x = max_u32(x, dpp<kDppPair>(x));
  x = max_u32(x, dpp<kDppFour>(x));
  x = max_u32(x, dpp<kDppEight>(x));
  return x;
}

// Over the wave, the same in every lane.  The whole wave has to be active.
__device__ __forceinline__ float wave_sum(float x) {
  x = row_sum(x);
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}
__device__ __forceinline__ float wave_max(float x) {
  x = row_max(x);
  return __builtin_fmaxf(__builtin_fmaxf(lane_value(x, 0), lane_value(x, 16)),
                         __builtin_fmaxf(lane_value(x, 32), lane_value(x, 48)));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  x = row_max_u32(x);
  const uint32_t a = __builtin_amdgcn_readlane(x, 0), b = __builtin_amdgcn_readlane(x, 16);
  const uint32_t c = __builtin_amdgcn_readlane(x, 32), d = __builtin_amdgcn_readlane(x, 48);
  return max_u32(max_u32(a, b), max_u32(c, d));
}

// Over the workgroup's `waves` waves (at most 16), the same in every lane.  `lds` is
// this call's alone until every wave has passed the next barrier.
__device__ __forceinline__ float block_sum(float x, float* lds, int waves) {
  x = wave_sum(x);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  const int lane = threadIdx.x % 16;
  return lane_value(row_sum(lane < waves ? lds[lane] : 0.0f), 0);
}
__device__ __forceinline__ uint32_t block_max_u32(uint32_t x, uint32_t* lds, int waves) {
  x = wave_max_u32(x);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  const int lane = threadIdx.x % 16;
  return (uint32_t)__builtin_amdgcn_readlane((int)row_max_u32(lane < waves ? lds[lane] : 0u), 0);
}

}  // namespace ra
