// ra_xent.hip -- softmax cross entropy over logits whose vocabulary is cut over
// the ranks, with its gradient.
//
//   m = max_j x_j,  z = sum_j exp(x_j - m),  lse = m + ln z,  loss = lse - x_y
//   dx_j = k (exp(x_j - m) / z - [j = y]),   k = grad_scale * dloss
//
// Maxima, sums and exponentials are float32; dx is rounded once.
//
// The exponentials are taken as 2^(x log2 e - c) with one fused multiply-add and
// the hardware's exponential, which is within 1 ulp.  c stands for m log2 e, but z,
// the loss and the gradient are all relative to 2^c, so any c near it gives the
// same results: c is m log2 e rounded, and m itself may be a little off the
// largest logit.  Partial sums keep the c they are relative to, and two of them
// join as z = z1 2^(c1 - c) + z2 2^(c2 - c) with exact differences.
//
// That holds as long as z stays inside float32's range.  A row where it does not --
// every column -inf or masked with the type's lowest value, a NaN or +inf, logits
// beyond 10^9 or so -- is done again with the largest logit subtracted first.
//
// The pass is bound by memory: reading the logits once and writing the gradient
// once is all it cannot avoid, so a workgroup keeps as much of its row in
// registers as they hold and only what is beyond that is read a second time.  Next
// comes arithmetic, two exponentials for each logit above all, which is why the
// other operations on a logit are kept to a handful.  Measured on MI355X, where a
// copy of 8 GiB runs at 6.55 TB/s:
//   8192 x 131072 bfloat16, 8 ranks, with gradient   832 us, 5.2 TB/s
//   ... the loss alone                               352 us, 6.1 TB/s
//   ... the gradient alone, from lse                 760 us, 5.6 TB/s
//   1003 x 50017 float32, 9 ranks, with gradient      97 us, 4.1 TB/s
//   4 x 128000 bfloat16, the loss alone              7.0 us in two launches
// The first reads 1.002 times the logits' bytes and writes the gradient's once (HBM
// counters).  It took 847 us with the arithmetic left out, the same with the logits in
// one buffer, and 4% more with half of each row read twice; 2^30 logits in rows of 4096
// to 65536 columns take 768 to 806 us.  So neither bytes nor arithmetic are what is
// left; which part of the memory system is, no counter has shown.  The float32 kernels
// with eight units a lane fill the registers (two of 128 go to scratch), and with long
// rows stay at 4.5-4.7 TB/s.
#include "ra_vocab.h"

namespace ra {
namespace {

// A sum z of exponentials relative to 2^c.  An empty one is (kNone, 0).
struct Part {
  float c, z;
};
constexpr float kNone = -1e38f;

__device__ __forceinline__ Part wave_join(Part a) {
  const float c = wave_max(a.c);
  return {c, wave_sum(a.z * exp2_of(a.c - c))};
}

// Over the workgroup of at most 16 waves; every lane gets it.
__device__ __forceinline__ Part block_join(Part a, Part* lds, int waves) {
  a = wave_join(a);
  const int lane = threadIdx.x % 64;
  if (lane == 0) lds[threadIdx.x / 64] = a;
  __syncthreads();
  // every wave joins the waves' parts itself, in the same order, 16 lanes alike
  Part b = lane % 16 < waves ? lds[lane % 16] : Part{kNone, 0.0f};
  const float c = row_max(b.c);
  return {lane_value(c, 0), lane_value(row_sum(b.z * exp2_of(b.c - c)), 0)};
}

// About the largest of N units' values, from kNone up.
//
// The 16-bit types compare two values at a time as float16.  For bfloat16 that is
// right as well: both types order like sign and magnitude of their bits.  Only
// magnitudes from 2^121 up are NaN as float16 and are passed over; if they matter,
// z overflows or stays 0.
template <int DT, int N>
__device__ __forceinline__ float top_of(const Unit<DT>* u) {
  if constexpr (DT == 1) {
    float m = kNone;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < kU; ++i) m = __builtin_fmaxf(m, unit_get<DT>(u[k], i));
    return m;
  } else {
    uint32_t m = 0xfc00fc00u;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < kU / 2; ++i) asm("v_pk_max_f16 %0, %1, %2" : "=v"(m) : "v"(m), "v"(u[k].v[0][i]));
    const float lo = Elem<DT>::to_w((uint16_t)(m & 0xffffu)), hi = Elem<DT>::to_w((uint16_t)(m >> 16));
    return __builtin_fmaxf(kNone, __builtin_fmaxf(lo, hi));
  }
}

// Joins N units, one after the other as their loads arrive.
template <int DT, int N>
__device__ __forceinline__ void take(Part& t, Unit<DT>* u) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    forget<DT>(&u[k]);
    const float c = __builtin_fmaxf(t.c, top_of<DT, 1>(&u[k]) * kLog2e);
    float e[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) e[i] = exp2_of(__builtin_fmaf(unit_get<DT>(u[k], i), kLog2e, -c));
    const float z = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    t.z = __builtin_fmaf(t.z, exp2_of(t.c - c), z);
    t.c = c;
    forget<DT>(&u[k]);
  }
}

// One token: its target, and what its gradient is scaled with.
constexpr int kNoLoss = -1, kNoColumn = -2;
struct Token {
  int y;        // the target's column, or one of the above
  float k;
};
__device__ __forceinline__ Token token(const XentArgs& a, int64_t row) {
  const int64_t y = a.target64 ? static_cast<const int64_t*>(a.target)[row]
                               : (int64_t)static_cast<const int32_t*>(a.target)[row];
  Token t;
  t.y = y < 0 ? kNoLoss : y < a.valid ? (int)y : kNoColumn;
  t.k = a.grad_scale * (a.dloss ? a.dloss[row] : 1.0f);
  if (t.y == kNoColumn) t.k = __uint_as_float(0x7fc00000u);
  return t;
}

// A row's sum: relative to 2^c, or (plain) to e^c with c the largest logit.
struct Sum {
  float c, z;
  bool plain;
};

// The sum of a row with its largest logit subtracted first, by one wave; all
// lanes get it.  For the rows that need it.
template <int DT, int MODE>
__device__ __forceinline__ Part plain_part(const XentArgs& a, int64_t row) {
  const int end = a.total;
  float m = -INFINITY;
  for (int q = 0; q < end; ++q) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, 1, end);
#pragma unroll
    for (int i = 0; i < kU; ++i) m = __builtin_fmaxf(m, unit_get<DT>(u[0], i));
  }
  m = wave_max(m);
  const float at = m == -INFINITY ? 0.0f : m;
  float z = 0.0f;
  for (int q = 0; q < end; ++q) {
    Unit<DT> u[1];
    fetch_all<DT, MODE, 1>(u, a, row, q, 1, end);
#pragma unroll
    for (int i = 0; i < kU; ++i) z += exp_of(unit_get<DT>(u[0], i) - at);
  }
  return {m, wave_sum(z)};
}

// Whether z is well inside float32's range; NaN is not.
__device__ __forceinline__ bool usable(Part t) { return t.z > 0x1p-100f && t.z < 0x1p120f; }
__device__ __forceinline__ bool empty(const Sum& t) { return t.plain && t.c == -INFINITY && t.z == 0.0f; }

// The loss is taken from z and c - x_y log2 e, and not from lse, which loses z in a
// large m.  A target that no column is, gives NaN; a token whose columns are all
// -inf, +inf.
__device__ __forceinline__ void write_loss(const XentArgs& a, int64_t row, int y, float xy, const Sum& t) {
  const float l2 = log2_of(t.z);
  if (a.lse) a.lse[row] = empty(t) ? -INFINITY : t.plain ? t.c + l2 * kLn2 : (t.c + l2) * kLn2;
  if (a.loss) {
    float loss = t.plain ? l2 * kLn2 + (t.c - xy) : (l2 + __builtin_fmaf(-xy, kLog2e, t.c)) * kLn2;
    if (!t.plain && __builtin_fabsf(xy) > 0x1p100f) loss = t.c * kLn2 - xy;   // the product overflows
    if (empty(t)) loss = INFINITY;
    if (y == kNoLoss) loss = 0.0f;
    if (y == kNoColumn) loss = __uint_as_float(0x7fc00000u);
    a.loss[row] = loss;
  }
}

// What a row's gradient is made with; a token without a loss, or whose columns
// are all -inf, gets zeros whatever else its row holds.
struct Grad {
  float c, kz;    // kz = k / z
  bool plain, zero;
};
__device__ __forceinline__ Grad grad_of(const Token& t, const Sum& sum) {
  return {empty(sum) ? 0.0f : sum.c, t.k / sum.z, sum.plain, t.y == kNoLoss || (t.y >= 0 && empty(sum))};
}

// The gradient of a wave's chunk.  WHOLE: one of the first a.full.  One chunk of
// the row has the target's column.
template <int DT, int MODE, bool WHOLE, bool PLAIN>
__device__ __forceinline__ void write_grad(const Unit<DT>& t, const Chunk& s, const XentArgs& a, int64_t row,
                                           const Token& tok, const Grad& g) {
  float d[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const float x = unit_get<DT>(t, i);
    d[i] = (PLAIN ? exp_of(x - g.c) : exp2_of(__builtin_fmaf(x, kLog2e, -g.c))) * g.kz;
  }
  Lane l = lane_of<MODE>(s);
  if (WHOLE) l.c = l.from;
  const int col = s.col0 - s.c0 + l.c;
  if (tok.y >= s.col0 && tok.y < s.col0 + kChunk) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i == tok.y) d[i] -= tok.k;
  }
  if (!WHOLE) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (col + i >= a.valid) d[i] = 0.0f;       // padding's gradient is zero, whatever k is
  }
  put<DT, MODE, WHOLE>(a, row, s, l, unit_make<DT>(d));
}

template <int DT, int MODE>
__device__ __forceinline__ void write_zero(const Chunk& s, const XentArgs& a, int64_t row) {
  put<DT, MODE, false>(a, row, s, lane_of<MODE>(s), Unit<DT>{});
}

// The rows that write_grad's registers do not serve, chunk by chunk: zeros, and
// sums that are plain.  True: done.  w, step: the chunks of this wave.
template <int DT, int MODE>
__device__ __forceinline__ bool other_grad(const XentArgs& a, int64_t row, int w, int step, int end, const Token& t,
                                           const Grad& g) {
  if (!g.zero && !g.plain) return false;
  for (int q = w; q < end; q += step) {
    if (g.zero) {
      write_zero<DT, MODE>(chunk(a, q), a, row);
    } else {
      Unit<DT> u[1];
      fetch_all<DT, MODE, 1>(u, a, row, q, step, end);
      write_grad<DT, MODE, false, true>(u[0], chunk(a, q), a, row, t, g);
    }
  }
  return true;
}

constexpr int kMore = 4;

// Joins the chunks from q0 on that are a wave's.
template <int DT, int MODE>
__device__ __forceinline__ void take_rest(Part& part, const XentArgs& a, int64_t row, int q0, int step, int end) {
  for (int q = q0; q < end; q += kMore * step) {
    Unit<DT> v[kMore];
    fetch_all<DT, MODE, kMore>(v, a, row, q, step, end);
    take<DT, kMore>(part, v);
  }
}

// Writes the gradient of those chunks, reading them again.
template <int DT, int MODE, bool PLAIN>
__device__ __forceinline__ void grad_rest(const XentArgs& a, int64_t row, int q0, int step, int end, const Token& t,
                                          const Grad& g) {
  for (; q0 < end; q0 += kMore * step) {
    Unit<DT> v[kMore];
    fetch_all<DT, MODE, kMore>(v, a, row, q0, step, end);
#pragma unroll
    for (int k = 0; k < kMore; ++k) {
      const int q = q0 + k * step;
      if (q >= end) continue;
      if (q < a.full) write_grad<DT, MODE, true, PLAIN>(v[k], chunk(a, q), a, row, t, g);
      else write_grad<DT, MODE, false, PLAIN>(v[k], chunk(a, q), a, row, t, g);
    }
  }
}

// The row's sum from the waves' parts; every wave has read the whole row then.
template <int DT, int MODE>
__device__ __forceinline__ Sum sum_of(Part part, Part* lds, int waves, const XentArgs& a, int64_t row) {
  part = block_join(part, lds, waves);
  if (usable(part)) return {part.c, part.z, false};      // the same in all waves
  part = plain_part<DT, MODE>(a, row);
  __syncthreads();
  return {part.c, part.z, true};
}

// The loss alone: a workgroup of G threads to a row.
template <int DT, int G, int MODE>
__global__ __launch_bounds__(G) void k_xent_loss(XentArgs a) {
  __shared__ Part lds[G / 64];
  const int64_t row = a.row0 + blockIdx.x;
  const int w = wave_id(), end = a.total;
  Part part = {kNone, 0.0f};
  take_rest<DT, MODE>(part, a, row, w, G / 64, end);
  const Token t = token(a, row);
  const float xy = logit<DT>(a, row, t.y);
  const Sum sum = sum_of<DT, MODE>(part, lds, G / 64, a, row);
  if (threadIdx.x == 0) write_loss(a, row, t.y, xy, sum);
}

// The loss and the gradient: a workgroup to a row, or to rows in a stride.  Each wave keeps its
// first K whole chunks of a row in registers, and one more of any kind (what is
// left of a piece, in general); any others it reads again for the gradient.  As
// soon as a unit's gradient is made, its registers take the next row's unit, and
// the sums are joined as units arrive: so loads are under way at all times but in
// the exchange between the waves.
//
// A gradient may take the logits' place: an element is only written by the lane
// that owns it, after the barrier that every read of the row comes before.  (What
// units read besides their own, they ignore.)
template <int DT, int K, int MODE>
__global__ __launch_bounds__(1024) void k_xent(XentArgs a) {
  __shared__ Part lds[2][16];
  const int w = wave_id(), waves = blockDim.x / 64, end = a.total;
  const int held = min(a.full, K * waves);
  // the wave's first chunk from `held` on, and the ones behind it
  const int more = w + (max(held - w, 0) + waves - 1) / waves * waves, rest = more + waves;
  const int last = max(held - 1, 0);     // in place of chunks that are not there
  Unit<DT> u[K], v[1];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int k = 0; k < K; ++k) u[k] = fetch<DT, MODE>(a, row, chunk(a, min(w + k * waves, last)));
  v[0] = fetch<DT, MODE>(a, row, chunk(a, min(more, end - 1)));
  // two buffers in turn: a wave may be a row ahead of another's last look
  for (int turn = 0;; turn ^= 1) {
    const Token t = token(a, row);
    const float xy = logit<DT>(a, row, t.y);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (w + k * waves >= held) mask_all<DT>(&u[k]);
    Part part = {kNone, 0.0f};
    take<DT, K>(part, u);
    if (more < end) {
      mask<DT, MODE>(&v[0], a, more, chunk(a, more));
      take<DT, 1>(part, v);
      take_rest<DT, MODE>(part, a, row, rest, waves, end);
    }
    const Sum sum = sum_of<DT, MODE>(part, lds[turn], waves, a, row);
    if (threadIdx.x == 0) write_loss(a, row, t.y, xy, sum);
    const Grad g = grad_of(t, sum);
    const int64_t next = row + gridDim.x;
    const int64_t then = min(next, a.tokens - 1);
    if (other_grad<DT, MODE>(a, row, w, waves, end, t, g)) {
      if (next >= a.tokens) return;
#pragma unroll
      for (int k = 0; k < K; ++k) u[k] = fetch<DT, MODE>(a, next, chunk(a, min(w + k * waves, last)));
      v[0] = fetch<DT, MODE>(a, next, chunk(a, min(more, end - 1)));
    } else {
      if (next < a.tokens) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int q = w + k * waves;
          if (q < held) write_grad<DT, MODE, true, false>(u[k], chunk(a, q), a, row, t, g);
          u[k] = fetch<DT, MODE>(a, then, chunk(a, min(q, last)));
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int q = w + k * waves;
          if (q < held) write_grad<DT, MODE, true, false>(u[k], chunk(a, q), a, row, t, g);
        }
      }
      if (more < end) {
        write_grad<DT, MODE, false, false>(v[0], chunk(a, more), a, row, t, g);
        grad_rest<DT, MODE, false>(a, row, rest, waves, end, t, g);
      }
      if (next >= a.tokens) return;
      v[0] = fetch<DT, MODE>(a, next, chunk(a, min(more, end - 1)));
    }
    row = next;
  }
}

constexpr int kSplitThreads = 256, kSplitWaves = kSplitThreads / 64;

// The chunks of one of a row's `splits` workgroups: [lo, hi).
__device__ __forceinline__ void split_range(const XentArgs& a, int part, int* lo, int* hi) {
  const int end = a.total, per = (end + a.splits - 1) / a.splits;
  *lo = min(end, part * per);
  *hi = min(end, *lo + per);
}

// Few tokens: `splits` workgroups share a row, each joining its part; the second
// launch joins the parts, and where a gradient is wanted a third reads the logits
// again.  A row's workspace: its sum (c, z, plain), then the parts.
constexpr int kRowSum = 4;
__device__ __forceinline__ float* row_space(const XentArgs& a, int64_t row) {
  return a.part + row * (kRowSum + 2 * a.splits);
}

template <int DT, int MODE>
__global__ __launch_bounds__(kSplitThreads) void k_xent_part(XentArgs a) {
  __shared__ Part lds[16];
  const int64_t row = blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  int lo, hi;
  split_range(a, part, &lo, &hi);
  Part sum = {kNone, 0.0f};
  take_rest<DT, MODE>(sum, a, row, lo + wave_id(), kSplitWaves, hi);
  sum = block_join(sum, lds, kSplitWaves);
  if (threadIdx.x == 0) {
    float* to = row_space(a, row) + kRowSum + 2 * part;
    to[0] = sum.c;
    to[1] = sum.z;
  }
}

// A wave to a row.  Before the gradient is written: it may take the logits' place.
template <int DT, int MODE>
__global__ __launch_bounds__(256) void k_xent_join(XentArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (row >= a.tokens) return;
  const Token t = token(a, row);
  const float xy = logit<DT>(a, row, t.y);
  const int i = threadIdx.x % 64;                 // at most 64 parts
  float* space = row_space(a, row);
  Part part = {kNone, 0.0f};
  if (i < a.splits) part = {space[kRowSum + 2 * i], space[kRowSum + 2 * i + 1]};
  part = wave_join(part);
  Sum sum = {part.c, part.z, false};
  if (!usable(part)) {
    part = plain_part<DT, MODE>(a, row);
    sum = {part.c, part.z, true};
  }
  if (i == 0) {
    write_loss(a, row, t.y, xy, sum);
    space[0] = sum.c;
    space[1] = sum.z;
    space[2] = sum.plain ? 1.0f : 0.0f;
  }
}

// The gradient alone: from the sums that k_xent_join left, or from the caller's lse.
template <int DT, bool FROM_LSE, int MODE>
__global__ __launch_bounds__(kSplitThreads) void k_xent_grad(XentArgs a) {
  const int64_t row = a.row0 + blockIdx.x / a.splits;
  const int part = blockIdx.x % a.splits;
  int lo, hi;
  split_range(a, part, &lo, &hi);
  const Token t = token(a, row);
  Sum sum;
  if constexpr (FROM_LSE) {
    // e^lse is the sum.  x - lse is taken first: a product lse log2 e would be
    // rounded once more, and nothing here makes up for that.
    const float lse = a.lse_in[row];
    sum = {lse, lse == -INFINITY ? 0.0f : 1.0f, lse == -INFINITY};
  } else {
    const float* space = row_space(a, row);
    sum = {space[0], space[1], space[2] != 0.0f};
  }
  const Grad g = grad_of(t, sum);
  const int w = lo + wave_id();
  if (other_grad<DT, MODE>(a, row, w, kSplitWaves, hi, t, g)) return;
  grad_rest<DT, MODE, FROM_LSE>(a, row, w, kSplitWaves, hi, t, g);
}

template <int DT, int G, int MODE>
hipError_t loss_go(const XentArgs& args, hipStream_t s) {
  constexpr int64_t kMost = 0xFFFFFFFFll / G;
  XentArgs a = args;
  for (; a.row0 < a.tokens; a.row0 += kMost) {
    k_xent_loss<DT, G, MODE><<<(unsigned)std::min(kMost, a.tokens - a.row0), G, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The GPUs of a machine are alike: asked once.
int compute_units() {
  static const int n = [] {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
    return cus;
  }();
  return n;
}

// Workgroups that leave room for no other on a compute unit stay and take rows in a
// stride; smaller ones take a row each, and the next one's loads cover this one's
// arithmetic (2^30 bfloat16 logits, us, a row each / staying: 4096 columns 779 / 927,
// 16384 796 / 848, 65536 781 / 826, 131072 841 / 832).
template <int DT, int K, int MODE>
hipError_t row_go(const XentArgs& a, int waves, hipStream_t s) {
  const int64_t most = waves > 8 ? compute_units() : 0xFFFFFFFFll / (waves * 64);
  k_xent<DT, K, MODE><<<(unsigned)std::min(most, a.tokens), waves * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, bool FROM_LSE, int MODE>
hipError_t grad_go(const XentArgs& args, hipStream_t s) {
  XentArgs a = args;
  const int64_t most = 0xFFFFFFFFll / kSplitThreads / a.splits;
  for (; a.row0 < a.tokens; a.row0 += most) {
    const unsigned grid = (unsigned)(std::min(most, a.tokens - a.row0) * a.splits);
    k_xent_grad<DT, FROM_LSE, MODE><<<grid, kSplitThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int MODE>
hipError_t split_go(const XentArgs& a, bool grad, hipStream_t s) {
  k_xent_part<DT, MODE><<<(unsigned)(a.tokens * a.splits), kSplitThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_xent_join<DT, MODE><<<(unsigned)((a.tokens + 3) / 4), 256, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess || !grad) return e;
  return grad_go<DT, false, MODE>(a, s);
}

template <int DT, int MODE>
hipError_t xent_size(const XentArgs& a, bool grad, hipStream_t s) {
  const int chunks = a.total;
  if (a.splits > 1) return split_go<DT, MODE>(a, grad, s);
  if (!grad) return chunks <= 8 ? loss_go<DT, 128, MODE>(a, s) : loss_go<DT, 512, MODE>(a, s);
  // waves: as few as hold the row
  constexpr int kMost = DT == 1 ? 8 : 16;
  if (a.full <= 8) return row_go<DT, 4, MODE>(a, std::max(1, (a.full + 3) / 4), s);
  return row_go<DT, kMost, MODE>(a, std::min(16, (a.full + kMost - 1) / kMost), s);
}

template <int DT>
hipError_t xent_go(const XentArgs& a, bool grad, bool al, hipStream_t s) {
  if (a.cut.base < kU) return grad ? row_go<DT, 4, kTiny>(a, 1, s) : loss_go<DT, 128, kTiny>(a, s);
  return al ? xent_size<DT, kAligned>(a, grad, s) : xent_size<DT, kOdd>(a, grad, s);
}

template <int DT>
hipError_t bwd_go(const XentArgs& a, bool al, hipStream_t s) {
  if (a.cut.base < kU) return grad_go<DT, true, kTiny>(a, s);
  return al ? grad_go<DT, true, kAligned>(a, s) : grad_go<DT, true, kOdd>(a, s);
}

}  // namespace

// The chunks of a cut vocabulary.
int vocab_chunks(int vocab, int p) { return vocab / p / kChunk * p + (vocab % (p * kChunk) != 0 ? p : 0); }

void vocab_geometry(VocabArgs* a) {
  a->whole = a->cut.base / kChunk;
  a->total = vocab_chunks(a->vocab, a->p);
  a->magic = a->whole > 0 ? (uint32_t)(((1ull << 32) + a->whole - 1) / a->whole) : 0;
  // chunks come in the order of their columns: the first ones end before `valid`
  a->full = 0;
  for (int r = 0; r < a->p && a->whole > 0; ++r) {
    const int lo = r * a->cut.base + std::min(r, a->cut.extra);
    const int n = std::max(0, std::min(a->whole, (a->valid - lo) / kChunk));
    a->full += a->valid > lo ? n : 0;
    if (n < a->whole) break;
  }
}

int64_t xent_words(int64_t tokens, int splits) { return splits > 1 ? tokens * (kRowSum + 2 * splits) : 0; }

// Sharing a row costs a second launch, and a third and another look at the logits
// for the gradient.  Measured (8 ranks, bfloat16, us; shared / a workgroup to a row):
//   loss      128000 columns: 1 token 5.6 / 12.7, 128 11.9 / 13.5, 192 15.7 / 13.5
//              64000: 1 token 5.5 / 8.1, 64 8.9 / 8.5;  32000: 1 token 5.4 / 5.3
//   gradient  128000: 1 token 9.4 / 20.6, 128 25.4 / 24.8;  32000: 64 11.8 / 13.6, 128 16.6 / 14.6
//               8192: 1 token 8.1 / 9.3, 192 9.9 / 10.0
int xent_splits(int64_t tokens, int vocab, int p, bool grad) {
  const int chunks = vocab_chunks(vocab, p);
  if (tokens < 1) return 1;      // the workspace of an empty batch is asked for, too
  if (vocab / p < kU || (grad ? tokens > 96 : chunks <= 64 || tokens > chunks / 2)) return 1;
  // two chunks at least for each wave of a row's workgroups
  const int64_t most = std::min<int64_t>(64, chunks / (2 * kSplitWaves));
  return most < 2 ? 1 : (int)std::min<int64_t>(most, (1024 + tokens - 1) / tokens);
}

hipError_t launch_xent(const XentArgs& a, int dtype, bool grad, bool al, hipStream_t s) {
  if (dtype == 1) return xent_go<1>(a, grad, al, s);
  if (dtype == 2) return xent_go<2>(a, grad, al, s);
  return xent_go<3>(a, grad, al, s);
}

hipError_t launch_xent_bwd(const XentArgs& a, int dtype, bool al, hipStream_t s) {
  if (dtype == 1) return bwd_go<1>(a, al, s);
  if (dtype == 2) return bwd_go<2>(a, al, s);
  return bwd_go<3>(a, al, s);
}

}  // namespace ra
