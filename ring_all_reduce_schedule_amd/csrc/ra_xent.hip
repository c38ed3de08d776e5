// ra_xent.hip -- softmax cross entropy over logits whose vocabulary is cut over
// the ranks, with its gradient.
//
//   m = max_j x_j,  z = sum_j exp(x_j - m),  lse = m + ln z,  loss = ln z + (m - x_y)
//   dx_j = c (exp(x_j - m) / z - [j = y]),   c = grad_scale * dloss
//
// Maxima, sums and exponentials are float32; dx is rounded once.  exp(x) is
// 2^(x log2 e) by the hardware's exponential, which is within 1 ulp.  A partial
// sum over some of the logits is kept with the maximum it is relative to, and
// two of them join as z = z1 exp(m1 - m) + z2 exp(m2 - m).
//
// The pass is bound by memory: reading the logits once and writing the gradient
// once is all it cannot avoid, so a workgroup keeps as much of its row in
// registers as they hold and only what is beyond that is read a second time.
#include "ra_rows.h"

namespace ra {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float ln_of(float x) { return __builtin_amdgcn_logf(x) * kLn2; }

// A sum of exponentials relative to a maximum.  An empty one is (-inf, 0).
struct Part {
  float m, z;
};
__device__ __forceinline__ bool empty(Part t) { return t.m == -INFINITY && t.z == 0.0f; }

// Relative to a maximum of -inf every logit is -inf and every term zero; using 0
// in its place keeps (-inf) - (-inf) out.
__device__ __forceinline__ float anchor(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ Part join(Part a, Part b) {
  const float m = __builtin_fmaxf(a.m, b.m), at = anchor(m);
  return {m, a.z * exp_of(a.m - at) + b.z * exp_of(b.m - at)};
}

__device__ __forceinline__ Part wave_join(Part a) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) a = join(a, {__shfl_xor(a.m, d), __shfl_xor(a.z, d)});
  return a;
}

// Over the workgroup; every lane gets it.
template <int WAVES>
__device__ __forceinline__ Part block_join(Part a, Part* lds) {
  a = wave_join(a);
  const int lane = threadIdx.x % 64;
  if (lane == 0) lds[threadIdx.x / 64] = a;
  __syncthreads();
  // every wave joins the waves' parts itself, in the same order
  return wave_join(lane < WAVES ? lds[lane] : Part{-INFINITY, 0.0f});
}

// A row's units over all ranks go in chunks of 64, one to each lane of a wave; a
// chunk lies in one piece, so that its pointers are the wave's and not the
// lanes'.  Chunk q is chunk q mod a.chunks of piece q / a.chunks.
struct Chunk {
  int r;        // piece (rank)
  int len;      // the piece's columns
  int c0;       // the chunk's first column in its piece
  int col0;     // ... and in the vocabulary
  bool whole;   // 512 columns of the piece, all valid
};
constexpr int kChunk = 64 * kU;

__device__ __forceinline__ Chunk chunk(const XentArgs& a, int q) {
  Chunk s;
  s.r = a.chunks == 1 ? q : (int)__umulhi((uint32_t)q, a.magic);
  s.len = piece_len(a.cut, s.r);
  s.c0 = (q - s.r * a.chunks) * kChunk;
  s.col0 = piece_lo(a.cut, s.r) + s.c0;
  s.whole = s.c0 + kChunk <= s.len && s.col0 + kChunk <= a.valid;
  return s;
}

// The lane's unit of a chunk, and whether it has one.
template <bool AL>
__device__ __forceinline__ bool lane_cut(const Chunk& s, Cut* u) {
  const int j = s.c0 / kU + (int)(threadIdx.x % 64);
  *u = unit_cut<AL>(j, s.len);
  return j * kU < s.len;
}

// Which of a unit's elements count: its own, before the first column that is not valid.
template <bool AL>
__device__ __forceinline__ bool counts(const Chunk& s, const Cut& u, int valid, int i) {
  return owns<AL>(u, i) && s.col0 - s.c0 + u.c + i < valid;
}

template <int DT, bool AL>
__device__ __forceinline__ Unit<DT> fetch(const XentArgs& a, int64_t row, const Chunk& s) {
  const char* x = static_cast<const char*>(a.x.b[s.r]) + row * s.len * ElemSize<DT>::value;
  if (s.whole) return load_unit<DT, AL>(x, s.c0 + (int)(threadIdx.x % 64) * kU);
  Cut u;
  Unit<DT> t{};
  if (lane_cut<AL>(s, &u)) t = load_cut<DT, AL>(x, 0, u);
  return t;
}

// A unit's values; -inf where they do not count.
template <int DT, bool AL>
__device__ __forceinline__ void values(float* x, const Unit<DT>& t, const Chunk& s, int valid) {
#pragma unroll
  for (int i = 0; i < kU; ++i) x[i] = unit_get<DT>(t, i);
  if (s.whole) return;
  Cut u;
  const bool in = lane_cut<AL>(s, &u);
#pragma unroll
  for (int i = 0; i < kU; ++i) x[i] = in && counts<AL>(s, u, valid, i) ? x[i] : -INFINITY;
}

template <int DT, bool AL, int N>
__device__ __forceinline__ void fetch_all(Unit<DT>* u, const XentArgs& a, int64_t row, int q0, int step, int end) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (q0 + k * step < end) u[k] = fetch<DT, AL>(a, row, chunk(a, q0 + k * step));
}

// Joins the N chunks q0, q0 + step, ... that the wave holds.
template <int DT, bool AL, int N>
__device__ __forceinline__ void take(Part& t, const Unit<DT>* u, const XentArgs& a, int q0, int step, int end) {
  float m = t.m;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (q0 + k * step < end) {
      float x[kU];
      values<DT, AL>(x, u[k], chunk(a, q0 + k * step), a.valid);
#pragma unroll
      for (int i = 0; i < kU; ++i) m = __builtin_fmaxf(m, x[i]);
    }
  }
  const float at = anchor(m);
  float z = t.z * exp_of(t.m - at);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (q0 + k * step < end) {
      float x[kU];
      values<DT, AL>(x, u[k], chunk(a, q0 + k * step), a.valid);
#pragma unroll
      for (int i = 0; i < kU; ++i) z += exp_of(x[i] - at);
    }
  }
  t = {m, z};
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// One token: its target, and what its gradient is scaled with.
constexpr int kNoLoss = -1, kNoColumn = -2;
struct Token {
  int y;        // the target's column, or one of the above
  float c;
};
__device__ __forceinline__ Token token(const XentArgs& a, int64_t row) {
  const int64_t y = a.target64 ? static_cast<const int64_t*>(a.target)[row]
                               : (int64_t)static_cast<const int32_t*>(a.target)[row];
  Token t;
  t.y = y < 0 ? kNoLoss : y < a.valid ? (int)y : kNoColumn;
  t.c = a.grad_scale * (a.dloss ? a.dloss[row] : 1.0f);
  if (t.y == kNoColumn) t.c = __uint_as_float(0x7fc00000u);
  return t;
}

// The target's logit; not read where there is none.
template <int DT>
__device__ __forceinline__ float logit(const XentArgs& a, int64_t row, int y) {
  if (y < 0) return 0.0f;
  const int r = piece_of(a.cut, y);
  const typename Elem<DT>::S* x = static_cast<const typename Elem<DT>::S*>(a.x.b[r]);
  const int64_t at = row * piece_len(a.cut, r) + (y - piece_lo(a.cut, r));
  if constexpr (DT == 1) return __uint_as_float(x[at]);
  else return Elem<DT>::to_w(x[at]);
}

// The loss is ln z + (m - x_y), which keeps ln z where lse = m + ln z loses it in
// a large m.  A target that is no column gives NaN; a token whose columns are all
// -inf, +inf.
__device__ __forceinline__ void write_loss(const XentArgs& a, int64_t row, int y, float xy, Part t) {
  if (a.lse) a.lse[row] = empty(t) ? -INFINITY : t.m + ln_of(t.z);
  if (a.loss) {
    float loss = ln_of(t.z) + (t.m - xy);
    if (empty(t)) loss = INFINITY;
    if (y == kNoLoss) loss = 0.0f;
    if (y == kNoColumn) loss = __uint_as_float(0x7fc00000u);
    a.loss[row] = loss;
  }
}

// What a row's gradient is made with; a token without a loss, or whose columns
// are all -inf, gets zeros whatever else its row holds.
struct Grad {
  float at, cz;   // the maximum, c / z
  bool zero;
};
__device__ __forceinline__ Grad grad_of(const Token& t, Part sum) {
  Grad g;
  g.zero = t.y == kNoLoss || (t.y >= 0 && empty(sum));
  g.at = anchor(sum.m);
  g.cz = t.c / sum.z;
  return g;
}

// The gradient of a wave's chunk, zero past the valid columns.  One chunk of the
// row has the target's column.
template <int DT, bool AL>
__device__ __forceinline__ void write_grad(const Unit<DT>& t, const Chunk& s, const XentArgs& a, int64_t row,
                                           const Token& tok, const Grad& g) {
  float d[kU];
  values<DT, AL>(d, t, s, a.valid);
#pragma unroll
  for (int i = 0; i < kU; ++i) d[i] = exp_of(d[i] - g.at) * g.cz;
  char* dx = static_cast<char*>(a.dx.b[s.r]) + row * s.len * ElemSize<DT>::value;
  Cut u = {s.c0 + (int)(threadIdx.x % 64) * kU, 0, kU};
  bool in = true;
  if (!s.whole) in = lane_cut<AL>(s, &u);
  const int col = s.col0 - s.c0 + u.c;
  if (tok.y >= s.col0 && tok.y < s.col0 + kChunk) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i == tok.y) d[i] -= tok.c;
  }
  if (s.whole) {
    store_unit<DT, AL>(dx, u.c, unit_make<DT>(d));
  } else if (in) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i >= a.valid) d[i] = 0.0f;
    store_cut<DT, AL>(dx, 0, u, unit_make<DT>(d));
  }
}

template <int DT, bool AL>
__device__ __forceinline__ void write_zero(const Chunk& s, const XentArgs& a, int64_t row) {
  char* dx = static_cast<char*>(a.dx.b[s.r]) + row * s.len * ElemSize<DT>::value;
  Cut u;
  if (lane_cut<AL>(s, &u)) store_cut<DT, AL>(dx, 0, u, Unit<DT>{});
}

// A workgroup of G threads takes a row.  GRAD: each wave keeps its first K chunks
// in registers and reads the rest again for the gradient.  A gradient may take the
// logits' place: an element is only written by the lane that read it, after the
// barrier that every read of the first pass comes before.  (Units that are moved
// back from the end of a piece read elements of their neighbour's, and ignore
// them.)
constexpr int kMore = 4;

template <int DT, int G, int K, bool GRAD, bool AL>
__global__ __launch_bounds__(G) void k_xent(XentArgs a) {
  constexpr int kWaves = G / 64;
  __shared__ Part lds[16];
  const int64_t row = a.row0 + blockIdx.x;
  const int w = wave_id(), end = a.chunks * a.p;
  Unit<DT> u[K];
  fetch_all<DT, AL, K>(u, a, row, w, kWaves, end);
  const Token t = token(a, row);
  const float xy = logit<DT>(a, row, t.y);
  Part sum = {-INFINITY, 0.0f};
  take<DT, AL, K>(sum, u, a, w, kWaves, end);
  for (int q = w + K * kWaves; q < end; q += kMore * kWaves) {
    Unit<DT> v[kMore];
    fetch_all<DT, AL, kMore>(v, a, row, q, kWaves, end);
    take<DT, AL, kMore>(sum, v, a, q, kWaves, end);
  }
  sum = block_join<kWaves>(sum, lds);
  if (threadIdx.x == 0) write_loss(a, row, t.y, xy, sum);
  if constexpr (GRAD) {
    const Grad g = grad_of(t, sum);
    if (g.zero) {
      for (int q = w; q < end; q += kWaves) write_zero<DT, AL>(chunk(a, q), a, row);
      return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int q = w + k * kWaves;
      if (q < end) write_grad<DT, AL>(u[k], chunk(a, q), a, row, t, g);
    }
    for (int q0 = w + K * kWaves; q0 < end; q0 += kMore * kWaves) {
      Unit<DT> v[kMore];
      fetch_all<DT, AL, kMore>(v, a, row, q0, kWaves, end);
#pragma unroll
      for (int k = 0; k < kMore; ++k) {
        const int q = q0 + k * kWaves;
        if (q < end) write_grad<DT, AL>(v[k], chunk(a, q), a, row, t, g);
      }
    }
  }
}

constexpr int kSplitThreads = 256, kSplitWaves = kSplitThreads / 64;

// The chunks of one of a row's `splits` workgroups: [lo, hi).
__device__ __forceinline__ void split_range(const XentArgs& a, int part, int* lo, int* hi) {
  const int end = a.chunks * a.p, per = (end + a.splits - 1) / a.splits;
  *lo = min(end, part * per);
  *hi = min(end, *lo + per);
}

// Few tokens: `splits` workgroups share a row, each joining its part; the second
// launch joins the parts, and where a gradient is wanted a third reads the logits
// again.
template <int DT, bool AL>
__global__ __launch_bounds__(kSplitThreads) void k_xent_part(XentArgs a) {
  __shared__ Part lds[16];
  const int64_t row = blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  int lo, hi;
  split_range(a, part, &lo, &hi);
  Part sum = {-INFINITY, 0.0f};
  for (int q = lo + wave_id(); q < hi; q += kMore * kSplitWaves) {
    Unit<DT> v[kMore];
    fetch_all<DT, AL, kMore>(v, a, row, q, kSplitWaves, hi);
    take<DT, AL, kMore>(sum, v, a, q, kSplitWaves, hi);
  }
  sum = block_join<kSplitWaves>(sum, lds);
  if (threadIdx.x == 0) {
    float* to = a.part + (row * a.splits + part) * 2;
    to[0] = sum.m;
    to[1] = sum.z;
  }
}

// The row's parts (at most 64), joined the same way by every wave.
__device__ __forceinline__ Part all_parts(const XentArgs& a, int64_t row) {
  const int i = threadIdx.x % 64;
  Part sum = {-INFINITY, 0.0f};
  if (i < a.splits) {
    const float* from = a.part + (row * a.splits + i) * 2;
    sum = {from[0], from[1]};
  }
  return wave_join(sum);
}

template <int DT>
__global__ __launch_bounds__(256) void k_xent_join(XentArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (row >= a.tokens) return;
  const Token t = token(a, row);
  const float xy = logit<DT>(a, row, t.y);
  const Part sum = all_parts(a, row);
  if (threadIdx.x % 64 == 0) write_loss(a, row, t.y, xy, sum);
}

// The gradient alone: from the parts that k_xent_part left, or from the caller's lse.
template <int DT, bool FROM_LSE, bool AL>
__global__ __launch_bounds__(kSplitThreads) void k_xent_grad(XentArgs a) {
  const int64_t row = a.row0 + blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  int lo, hi;
  split_range(a, part, &lo, &hi);
  const Token t = token(a, row);
  Part sum;
  if constexpr (FROM_LSE) {
    const float lse = a.lse_in[row];
    sum = {lse, lse == -INFINITY ? 0.0f : 1.0f};
  } else {
    sum = all_parts(a, row);
  }
  const Grad g = grad_of(t, sum);
  for (int q0 = lo + wave_id(); q0 < hi; q0 += kMore * kSplitWaves) {
    if (g.zero) {
#pragma unroll
      for (int k = 0; k < kMore; ++k)
        if (q0 + k * kSplitWaves < hi) write_zero<DT, AL>(chunk(a, q0 + k * kSplitWaves), a, row);
      continue;
    }
    Unit<DT> v[kMore];
    fetch_all<DT, AL, kMore>(v, a, row, q0, kSplitWaves, hi);
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      const int q = q0 + k * kSplitWaves;
      if (q < hi) write_grad<DT, AL>(v[k], chunk(a, q), a, row, t, g);
    }
  }
}

template <int DT, int G, int K, bool GRAD>
hipError_t row_go(const XentArgs& args, bool al, hipStream_t s) {
  constexpr int64_t kMost = 0xFFFFFFFFll / G;
  XentArgs a = args;
  for (; a.row0 < a.tokens; a.row0 += kMost) {
    const unsigned grid = (unsigned)std::min(kMost, a.tokens - a.row0);
    if (al) k_xent<DT, G, K, GRAD, true><<<grid, G, 0, s>>>(a);
    else k_xent<DT, G, K, GRAD, false><<<grid, G, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, bool FROM_LSE>
hipError_t grad_go(const XentArgs& args, bool al, hipStream_t s) {
  XentArgs a = args;
  const int64_t most = 0xFFFFFFFFll / kSplitThreads / a.splits;
  for (; a.row0 < a.tokens; a.row0 += most) {
    const unsigned grid = (unsigned)(std::min(most, a.tokens - a.row0) * a.splits);
    if (al) k_xent_grad<DT, FROM_LSE, true><<<grid, kSplitThreads, 0, s>>>(a);
    else k_xent_grad<DT, FROM_LSE, false><<<grid, kSplitThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t xent_go(const XentArgs& a, bool grad, bool al, hipStream_t s) {
  if (a.splits > 1) {
    const unsigned grid = (unsigned)(a.tokens * a.splits);
    if (al) k_xent_part<DT, true><<<grid, kSplitThreads, 0, s>>>(a);
    else k_xent_part<DT, false><<<grid, kSplitThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_xent_join<DT><<<(unsigned)((a.tokens + 3) / 4), 256, 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess || !grad) return e;
    return grad_go<DT, false>(a, al, s);
  }
  const int chunks = a.chunks * a.p;
  if (!grad) return chunks <= 8 ? row_go<DT, 128, 4, false>(a, al, s) : row_go<DT, 512, 4, false>(a, al, s);
  if (chunks <= 8) return row_go<DT, 128, 4, true>(a, al, s);
  if (chunks <= 32) return row_go<DT, 512, 4, true>(a, al, s);
  if (chunks <= 64) return row_go<DT, 512, 8, true>(a, al, s);
  if constexpr (DT != 1)
    if (chunks > 128) return row_go<DT, 1024, 16, true>(a, al, s);
  return row_go<DT, 1024, 8, true>(a, al, s);
}

}  // namespace

int xent_chunks(int vocab, int p) { return (vocab / p + (vocab % p != 0) + kChunk - 1) / kChunk; }

int xent_splits(int64_t tokens, int vocab, int p) {
  // To be shared, a row needs two chunks for each wave of its workgroups.
  const int64_t most = std::min<int64_t>(64, (int64_t)p * xent_chunks(vocab, p) / (2 * kSplitWaves));
  if (tokens >= 512 || most < 2) return 1;
  return (int)std::min<int64_t>(most, (1024 + tokens - 1) / tokens);
}

hipError_t launch_xent(const XentArgs& a, int dtype, bool grad, bool al, hipStream_t s) {
  if (dtype == 1) return xent_go<1>(a, grad, al, s);
  if (dtype == 2) return xent_go<2>(a, grad, al, s);
  return xent_go<3>(a, grad, al, s);
}

hipError_t launch_xent_bwd(const XentArgs& a, int dtype, bool al, hipStream_t s) {
  if (dtype == 1) return grad_go<1, true>(a, al, s);
  if (dtype == 2) return grad_go<2, true>(a, al, s);
  return grad_go<3, true>(a, al, s);
}

}  // namespace ra
