// ra_norm.hip -- RMS norm over the sum of the ranks' partials, and its gradient.
//
//   forward    h = sum_r x_r + res,  rstd = 1 / sqrt(mean(h^2) + eps),  y = (h rstd) w
//   8 bits     scale = max(max |y|, 2^-110) / 448 for each token or group of columns,
//              q = e4m3(y / scale)
//   backward   g = sum_r dy_r,  xhat = h rstd,
//              dh = dh_in + rstd (w g - xhat mean(w g xhat)),  dw = sum over tokens of g xhat
//
// Everything between the loads and the final rounding is float32: the ranks'
// sum (in rank order), the mean of squares, the normalised values.  The norm is
// taken of the unrounded h, so y carries one rounding; the residual stream keeps
// h rounded to its own type, and the backward pass works from that.
//
// Both passes stream: each input is read once and each output written once, and
// the sum of a row stays in registers between its statistic and its output.  A
// workgroup takes a row (a wave where a row is at most 64 units), because the
// statistic then needs one exchange through LDS and no second launch.  A thread
// has one unit of the row where 1024 threads hold it: more threads with one unit
// each beat fewer with more (forward, 256 threads with four units 193 us against
// 186 with 1024; gradient, 512 with two 147 against 143).
//
// What bounds them is memory, and in particular how many streams at the same
// offset of different buffers it serves (8 ranks read, 8 written and the residual
// both ways).  Measured on MI355X, where a copy of 8 GiB runs at 6.55 TB/s:
//   4096 x 8192 bfloat16, 8 ranks, 8-bit outputs to all   168 us, 5.6 TB/s
//   its gradient                                          142 us, 5.7 TB/s
//   16384 x 8192 bfloat16, one rank, a residual both ways 172 us, 6.2 TB/s
//   1003 x 5001 float16, 9 ranks, rows on odd addresses    25 us, 5.4 TB/s
//   1 x 4096 bfloat16, 8 ranks                            3.8 us
// Asking for 64 registers, to have twice the waves, changed the first two by less
// than 1% and cost the kernels with a float32 residual 3-7%.
#include "ra_rows.h"

namespace ra {
namespace {

constexpr float kF8Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-110f;

// Eight float32 values in e4m3, to nearest even.
__device__ __forceinline__ u32x2 unit_f8(const float* x) {
  u32x2 q;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k], x[4 * k + 1], 0, false);
    q[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2], x[4 * k + 3], w, true);
  }
  return q;
}

template <int AC>
__device__ __forceinline__ void store_f8(void* p, int64_t row, const Cut& u, u32x2 q) {
  uint8_t* d = static_cast<uint8_t*>(p) + row + u.c;
  if (AC != 0 || u.hi - u.lo == kU) {
    if constexpr (AC == kStreamRows) __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(d));
    else if constexpr (AC != 0) *reinterpret_cast<u32x2*>(d) = q;
    else *reinterpret_cast<u32x2_by1*>(d) = q;
  } else {
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (owns<AC>(u, k)) d[k] = (uint8_t)(q[k / 4] >> (k % 4 * 8));
  }
}

// The scale of values whose largest magnitude has these bits.  Magnitudes are
// compared as integers: infinity is above every finite value and NaN above
// infinity, so neither is lost.
__device__ __forceinline__ float f8_amax(uint32_t bits) {
  return bits < __float_as_uint(kAmaxFloor) ? kAmaxFloor : __uint_as_float(bits);
}

// ONE: a wave to a row, four rows to a workgroup; else a workgroup to a row.  K units
// to a thread.  DT: the partials' type; RT: the residual's (0: none); F8: 8-bit output.
template <int DT, int RT, bool ONE, int K, bool F8, int AC>
__global__ __launch_bounds__(ONE ? 256 : 1024) void k_norm(NormArgs a) {
  const int G = ONE ? 64 : blockDim.x;
  __shared__ float lds_sum[16];
  __shared__ uint32_t lds_max[16];
  const int64_t row = a.row0 + (ONE ? (int64_t)blockIdx.x * 4 + threadIdx.x / 64 : (int64_t)blockIdx.x);
  const int tid = ONE ? threadIdx.x % 64 : threadIdx.x;
  if (row >= a.tokens) return;      // whole waves; only where there is no barrier
  const int hidden = a.hidden;
  const int64_t at = row * hidden;

  float h[K][kU];
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int j = tid + k * G;
    if (j * kU < hidden) {
      const Cut u = unit_cut<AC>(j, hidden);
      Unit<RT == 0 ? DT : RT> res{};
      if constexpr (RT != 0)
        if (a.res) res = load_cut<RT, AC>(a.res, at, u);
      fold_ranks<DT, AC>(h[k], a.in, a.p, at, u);
      if constexpr (RT != 0) {
#pragma unroll
        for (int i = 0; i < kU; ++i) h[k][i] += owns<AC>(u, i) ? unit_get<RT>(res, i) : 0.0f;
        if (a.res_out) store_cut<RT, AC>(a.res_out, at, u, unit_make<RT>(h[k]));
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) ss = __builtin_fmaf(h[k][i], h[k][i], ss);
    }
  }
  ss = ONE ? wave_sum(ss) : block_sum(ss, lds_sum, G / 64);
  const float rstd = 1.0f / __builtin_sqrtf(ss * a.inv_h + a.eps);
  if (tid == 0 && a.rstd) a.rstd[row] = rstd;

  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int j = tid + k * G;
    const bool in = j * kU < hidden;
    const Cut u = unit_cut<AC>(j, hidden);
    uint32_t here = 0;
    if (in) {
      const Unit<DT> w = load_cut<DT, AC != 0>(a.weight, 0, u);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        h[k][i] = owns<AC>(u, i) ? h[k][i] * rstd * unit_get<DT>(w, i) : 0.0f;
        const uint32_t m = __float_as_uint(h[k][i]) & 0x7fffffffu;
        here = here > m ? here : m;
      }
      if constexpr (!F8) {
        const Unit<DT> y = unit_make<DT>(h[k]);
        for (int r = 0; r < a.n_out; ++r) store_cut<DT, AC>(a.out.b[r], at, u, y);
      }
    }
    if constexpr (F8) {
      if (a.group) {
        // a group is 4, 8 or 16 neighbouring lanes; lanes past the row hold 0
        here = max_u32(here, dpp<kDppNeighbour>(here));
        here = max_u32(here, dpp<kDppPair>(here));
        if (a.group > 32) here = max_u32(here, dpp<kDppFour>(here));
        if (a.group > 64) here = max_u32(here, dpp<kDppEight>(here));
        const float amax = f8_amax(here), inv = kF8Max / amax;
        if (in) {
#pragma unroll
          for (int i = 0; i < kU; ++i) h[k][i] *= inv;
          const u32x2 y = unit_f8(h[k]);
          const int groups = (hidden + a.group - 1) / a.group;
          for (int r = 0; r < a.n_out; ++r) {
            store_f8<AC>(a.out.b[r], at, u, y);
            if (j * kU % a.group == 0)
              static_cast<float*>(a.scale.b[r])[row * groups + j * kU / a.group] = amax / kF8Max;
          }
        }
      } else {
        top = top > here ? top : here;
      }
    }
  }
  if constexpr (F8) {
    if (a.group) return;
    const float amax = f8_amax(ONE ? wave_max_u32(top) : block_max_u32(top, lds_max, G / 64)), inv = kF8Max / amax;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int j = tid + k * G;
      if (j * kU < hidden) {
        const Cut u = unit_cut<AC>(j, hidden);
#pragma unroll
        for (int i = 0; i < kU; ++i) h[k][i] *= inv;
        const u32x2 y = unit_f8(h[k]);
        for (int r = 0; r < a.n_out; ++r) store_f8<AC>(a.out.b[r], at, u, y);
      }
    }
    // lanes of one wave: a row has at least 64 threads, and at most 64 ranks
    if (tid < a.n_out) static_cast<float*>(a.scale.b[tid])[row] = amax / kF8Max;
  }
}

// ---------------------------------------------------------------- backward

// Workgroups take the rows in a stride and keep their columns' sums for dw in
// registers over all of them.
template <int DT, int RT, int K, int AC>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormBwdArgs a) {
  const int G = blockDim.x;
  // Four units a thread leave no registers for h: it is read again, from the cache.
  // All but two of those kernels put 6 to 21 of their 128 registers into scratch even so
  // (2048 x 32768 bfloat16, one rank: 124 us, where its bytes at a copy's rate take 62).
  constexpr bool kKeep = K <= 2;
  __shared__ float lds_sum[2][16];
  const int tid = threadIdx.x, hidden = a.hidden;
  float dw[K][kU];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < kU; ++i) dw[k][i] = 0.0f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.tokens; row += gridDim.x, turn ^= 1) {
    const int64_t at = row * hidden;
    const float rstd = a.rstd[row];
    float g[K][kU];
    Unit<RT> hu[kKeep ? K : 1];
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int j = tid + k * G;
      if (j * kU < hidden) {
        const Cut u = unit_cut<AC>(j, hidden);
        Unit<RT>& hk = hu[kKeep ? k : 0];
        hk = load_cut<RT, AC>(a.h, at, u);
        const Unit<DT> w = load_cut<DT, AC != 0>(a.weight, 0, u);
        fold_ranks<DT, AC>(g[k], a.in, a.p, at, u);
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          const float x = owns<AC>(u, i) ? unit_get<RT>(hk, i) * rstd : 0.0f;
          dw[k][i] = __builtin_fmaf(g[k][i], x, dw[k][i]);
          g[k][i] *= unit_get<DT>(w, i);
          dot = __builtin_fmaf(g[k][i], x, dot);
        }
      }
    }
    // two buffers in turn: a wave may be a row ahead of another's last read
    dot = block_sum(dot, lds_sum[turn], G / 64) * a.inv_h;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int j = tid + k * G;
      if (j * kU < hidden) {
        const Cut u = unit_cut<AC>(j, hidden);
        Unit<RT>& hk = hu[kKeep ? k : 0];
        if constexpr (!kKeep) hk = load_cut<RT, AC>(a.h, at, u);
        Unit<RT> d{};
        if (a.dh_in) d = load_cut<RT, AC>(a.dh_in, at, u);
        float y[kU];
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          const float x = unit_get<RT>(hk, i) * rstd;
          y[i] = unit_get<RT>(d, i) + rstd * (g[k][i] - x * dot);
        }
        store_cut<RT, AC>(a.dh, at, u, unit_make<RT>(y));
        const Unit<DT> t = unit_make<DT>(y);
        for (int r = 0; r < a.n_dx; ++r) store_cut<DT, AC>(a.dx.b[r], at, u, t);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int j = tid + k * G;
      if (j * kU < hidden)
        store_cut<1, AC != 0>(a.part, (int64_t)blockIdx.x * hidden, unit_cut<AC>(j, hidden), unit_make<1>(dw[k]));
    }
  }
}

// dw[c] = sum over the workgroups of part[b][c], in a fixed order: 16 rows of
// workgroups side by side, then their 16 sums.
__global__ __launch_bounds__(1024) void k_norm_dweight(const float* part, float* dw, int blocks, int hidden) {
  __shared__ float lds[16][64];
  const int col = threadIdx.x % 64, lane = threadIdx.x / 64;
  const int64_t c = (int64_t)blockIdx.x * 64 + col;
  float s = 0.0f;
  if (c < hidden) {
#pragma unroll 8
    for (int b = lane; b < blocks; b += 16) s += part[(int64_t)b * hidden + c];
  }
  lds[lane][col] = s;
  __syncthreads();
  if (lane == 0 && c < hidden) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += lds[i][col];
    dw[c] = t;
  }
}

// ---------------------------------------------------------------- launches

// Threads that hold `units` units, K to a thread.
int threads_for(int units, int K) { return (units + 64 * K - 1) / (64 * K) * 64; }

// One launch, or several where the rows pass what one dispatch counts.
template <int DT, int RT, bool ONE, int K, bool F8>
hipError_t norm_go(const NormArgs& args, int units, int access, hipStream_t s) {
  const int64_t per = ONE ? 4 : 1, threads = ONE ? 256 : threads_for(units, K);
  const int64_t most = 0xFFFFFFFFll / threads;
  NormArgs a = args;
  for (; a.row0 < a.tokens; a.row0 += most * per) {
    const dim3 grid((unsigned)std::min(most, (a.tokens - a.row0 + per - 1) / per)), block((unsigned)threads);
    if (access == kStreamRows) k_norm<DT, RT, ONE, K, F8, kStreamRows><<<grid, block, 0, s>>>(a);
    else if (access == kAlignedRows) k_norm<DT, RT, ONE, K, F8, kAlignedRows><<<grid, block, 0, s>>>(a);
    else k_norm<DT, RT, ONE, K, F8, kOddRows><<<grid, block, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int RT, bool F8>
hipError_t norm_size(const NormArgs& a, int access, hipStream_t s) {
  const int units = (a.hidden + kU - 1) / kU;
  if (units <= 64) return norm_go<DT, RT, true, 1, F8>(a, units, access, s);
  if (units <= 1024) return norm_go<DT, RT, false, 1, F8>(a, units, access, s);
  if (units <= 2048) return norm_go<DT, RT, false, 2, F8>(a, units, access, s);
  return norm_go<DT, RT, false, 4, F8>(a, units, access, s);
}

template <int DT, int RT>
hipError_t norm_out(const NormArgs& a, bool f8, int access, hipStream_t s) {
  return f8 ? norm_size<DT, RT, true>(a, access, s) : norm_size<DT, RT, false>(a, access, s);
}

template <int DT>
hipError_t norm_res(const NormArgs& a, int res_dtype, bool f8, int access, hipStream_t s) {
  if (!a.res && !a.res_out) return norm_out<DT, 0>(a, f8, access, s);
  if (DT != 1 && res_dtype == 1) return norm_out<DT, 1>(a, f8, access, s);
  return norm_out<DT, DT>(a, f8, access, s);
}

template <int DT, int RT, int K>
hipError_t bwd_go(const NormBwdArgs& a, int units, int access, int grid, hipStream_t s) {
  const int threads = threads_for(units, K);
  if (access == kStreamRows) k_norm_bwd<DT, RT, K, kStreamRows><<<grid, threads, 0, s>>>(a);
  else if (access == kAlignedRows) k_norm_bwd<DT, RT, K, kAlignedRows><<<grid, threads, 0, s>>>(a);
  else k_norm_bwd<DT, RT, K, kOddRows><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT, int RT>
hipError_t bwd_size(const NormBwdArgs& a, int access, int grid, hipStream_t s) {
  const int units = (a.hidden + kU - 1) / kU;
  if (units <= 1024) return bwd_go<DT, RT, 1>(a, units, access, grid, s);
  if (units <= 2048) return bwd_go<DT, RT, 2>(a, units, access, grid, s);
  return bwd_go<DT, RT, 4>(a, units, access, grid, s);
}

template <int DT>
hipError_t bwd_res(const NormBwdArgs& a, int h_dtype, int access, int grid, hipStream_t s) {
  if (DT != 1 && h_dtype == 1) return bwd_size<DT, 1>(a, access, grid, s);
  return bwd_size<DT, DT>(a, access, grid, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, int res_dtype, bool f8, int access, hipStream_t s) {
  if (dtype == 1) return norm_res<1>(a, res_dtype, f8, access, s);
  if (dtype == 2) return norm_res<2>(a, res_dtype, f8, access, s);
  return norm_res<3>(a, res_dtype, f8, access, s);
}

int norm_bwd_blocks(int64_t tokens) { return (int)std::min<int64_t>(tokens, kNormBwdBlocks); }

hipError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int h_dtype, float* dweight, int access, hipStream_t s) {
  const int grid = norm_bwd_blocks(a.tokens);
  if (grid > 0) {
    hipError_t e = dtype == 1   ? bwd_res<1>(a, h_dtype, access, grid, s)
                   : dtype == 2 ? bwd_res<2>(a, h_dtype, access, grid, s)
                                : bwd_res<3>(a, h_dtype, access, grid, s);
    if (e != hipSuccess) return e;
  }
  if (dweight) {   // no rows: zeros
    k_norm_dweight<<<(a.hidden + 63) / 64, 1024, 0, s>>>(a.part, dweight, grid, a.hidden);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace ra
