// Root-mean-square norm of the sum of W contributions and a residual, and its gradient.
//
// Forward, one row per workgroup at a time: h = ((x_0 + x_1) + ...) + residual in binary32 (the
// ordered sum of plr_reduce with the residual as one more source), r = 1 / sqrt(mean(h^2) +
// eps), y = h r gamma. Each thread keeps its vectors of h, so every input byte is read once and
// every output byte written once; the row needs one workgroup sum (and one maximum more for the
// 8-bit output). Bound by HBM: (W + 2) e + o bytes per element against about W + 5 operations. 8 x
// [8192, 7168] bf16 and a residual to 8-bit rows: 205 us (6.0 TB/s); one such row 4.6 us.
// Workgroups of up to 1024 threads leave 128 registers a thread. One vector a thread fits them
// (from 9 sources on up to 4 spill), and so do two of up to 8 sources. Two vectors of 9 to 16
// sources spill 28-44 registers into scratch (16 x [8192, 7168] bf16: 543 us, 4.1 TB/s), four of
// 5 to 8 sources (binary32: 2 to 8) 10-34 (8 x [2048, 32768] bf16: 328 us, 4.5 TB/s; 4 sources,
// which spill nothing: 164 us, 5.7 TB/s), four of 9 to 16 sources 108-128 (799 us, 3.2 TB/s).
//
// Gradient: with xh = h r and g = dy gamma,
//   dx = r (g - xh mean(g xh)) + dsum,   dgamma = sum over rows of dy xh.
// A workgroup walks rows b, b + B, ... and keeps its columns' dgamma sums in registers;
// its partial sums go to the workspace and a second kernel adds the B of them in order, so
// the result does not depend on which workgroup ends first. [8191, 7168] bf16 with dsum: 79 us
// (5.9 TB/s) and 4.9 us for the second kernel. Rows of more than 2048 vectors (four a thread) spill
// 73 registers in bf16, 106 in fp16 and 5 in binary32: [2048, 32768] 266 and 315 us (2.0 and 1.7
// TB/s), [2048, 16384] binary32 110 us (4.9 TB/s).
#include <algorithm>

#include "device_common.h"
#include "moe.h"
#include "wave.h"

namespace plr {

namespace {

__device__ __forceinline__ u32x4 row_load(const char* base, uint64_t pitch, int64_t row, uint32_t vec) {
  return ld16(reinterpret_cast<const u32x4*>(base + (uint64_t)row * pitch) + vec);
}
__device__ __forceinline__ void row_store(char* base, uint64_t pitch, int64_t row, uint32_t vec, u32x4 v) {
  st16(reinterpret_cast<u32x4*>(base + (uint64_t)row * pitch) + vec, v);
}

// V vectors per thread: vector t + v * threads of the row. WMAX: sources whose loads are
// in flight together (world <= WMAX).
template <int DT, int WMAX, int V, bool F8>
__global__ __launch_bounds__(kNormMaxThreads) void k_norm(const NormArgs a) {
  constexpr int N = Elems<DT>::N;
  // two sets in turn: a wave may be at the next row's sum while another reads this row's
  __shared__ uint32_t s_sum[2][16], s_max[2][16];
  const uint32_t threads = blockDim.x;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    float h[V][N];
    float sq = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = threadIdx.x + v * threads;
      if (i < a.nvec) {
        u32x4 x[WMAX], res;
#pragma unroll
        for (int w = 0; w < WMAX; ++w)
          if (w < (int)a.world) x[w] = row_load(a.src[w], a.src_pitch, row, i);
        if (a.residual) res = row_load(a.residual, a.residual_pitch, row, i);
        Elems<DT>::widen(x[0], h[v]);
#pragma unroll
        for (int w = 1; w < WMAX; ++w)
          if (w < (int)a.world) {
            float t[N];
            Elems<DT>::widen(x[w], t);
#pragma unroll
            for (int j = 0; j < N; ++j) h[v][j] += t[j];
          }
        if (a.residual) {
          float t[N];
          Elems<DT>::widen(res, t);
#pragma unroll
          for (int j = 0; j < N; ++j) h[v][j] += t[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) h[v][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) sq = __builtin_fmaf(h[v][j], h[v][j], sq);
    }
    // the stored sum is rounded once; the norm goes on with the sum as it is
    if (a.sum_out) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t i = threadIdx.x + v * threads;
        if (i < a.nvec) row_store(a.sum_out, a.sum_pitch, row, i, Elems<DT>::narrow(h[v]));
      }
    }
    sq = __uint_as_float(block_reduce(__float_as_uint(sq), AddF32(), s_sum[turn]));
    const float r = 1.0f / sqrtf(__builtin_fmaf(sq, a.inv_cols, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = threadIdx.x + v * threads;
      if (i >= a.nvec) continue;
      float gm[N];
      Elems<DT>::widen(reinterpret_cast<const u32x4*>(a.gamma)[i], gm);
#pragma unroll
      for (int j = 0; j < N; ++j) h[v][j] = h[v][j] * r * gm[j];
      if constexpr (F8) {
        // magnitudes compared as integers: the same order, and a NaN is the largest
#pragma unroll
        for (int j = 0; j < N; ++j) top = max(top, __float_as_uint(h[v][j]) & 0x7FFFFFFFu);
      } else {
        row_store(a.out, a.out_pitch, row, i, Elems<DT>::narrow(h[v]));
      }
    }
    if constexpr (F8) {
      top = max(block_reduce(top, MaxU32(), s_max[turn]), __float_as_uint(kF8Floor));
      const float m = __uint_as_float(top);
      const float inv = kF8Max / m;
      if (threadIdx.x == 0) a.out_scale[row] = m / kF8Max;
      typedef uint32_t Packed __attribute__((ext_vector_type(N / 4)));
      Packed* o = reinterpret_cast<Packed*>(a.out + (uint64_t)row * a.out_pitch);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t i = threadIdx.x + v * threads;
        if (i >= a.nvec) continue;
        Packed w;
#pragma unroll
        for (int q = 0; q < N / 4; ++q)
          w[q] = f8_quad(h[v][4 * q] * inv, h[v][4 * q + 1] * inv, h[v][4 * q + 2] * inv, h[v][4 * q + 3] * inv);
        __builtin_nontemporal_store(w, o + i);
      }
    }
  }
}

template <int DT, int V>
__global__ __launch_bounds__(kNormMaxThreads) void k_norm_back(const NormBackArgs a) {
  constexpr int N = Elems<DT>::N;
  __shared__ uint32_t s_dot[2][16];
  const uint32_t threads = blockDim.x;
  float gm[V][N], dg[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t i = threadIdx.x + v * threads;
    u32x4 g = {0, 0, 0, 0};
    if (i < a.nvec) g = reinterpret_cast<const u32x4*>(a.gamma)[i];
    Elems<DT>::widen(g, gm[v]);
#pragma unroll
    for (int j = 0; j < N; ++j) dg[v][j] = 0.f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const float r = a.rstd[row];
    float xh[V][N], d[V][N];
    u32x4 ds[V];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = threadIdx.x + v * threads;
      u32x4 hv = {0, 0, 0, 0}, dv = {0, 0, 0, 0};
      if (i < a.nvec) {
        hv = row_load(a.h, a.h_pitch, row, i);
        dv = row_load(a.dout, a.dout_pitch, row, i);
        if (a.dsum) ds[v] = row_load(a.dsum, a.dsum_pitch, row, i);
      }
      Elems<DT>::widen(hv, xh[v]);
      Elems<DT>::widen(dv, d[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        xh[v][j] *= r;
        dg[v][j] = __builtin_fmaf(d[v][j], xh[v][j], dg[v][j]);
        d[v][j] *= gm[v][j];
        dot = __builtin_fmaf(d[v][j], xh[v][j], dot);
      }
    // two arrays in turn: a wave may be at the next row's sum while another reads this one's
    dot = __uint_as_float(block_reduce(__float_as_uint(dot), AddF32(), s_dot[turn])) * a.inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = threadIdx.x + v * threads;
      if (i >= a.nvec) continue;
      float t[N];
#pragma unroll
      for (int j = 0; j < N; ++j) d[v][j] = r * (d[v][j] - xh[v][j] * dot);
      if (a.dsum) {
        Elems<DT>::widen(ds[v], t);
#pragma unroll
        for (int j = 0; j < N; ++j) d[v][j] += t[j];
      }
      row_store(a.dx, a.dx_pitch, row, i, Elems<DT>::narrow(d[v]));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t i = threadIdx.x + v * threads;
    if (i >= a.nvec) continue;
    float* p = a.partial + (uint64_t)blockIdx.x * a.nvec * N + (uint64_t)i * N;
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const u32x4 w = {__float_as_uint(dg[v][4 * q]), __float_as_uint(dg[v][4 * q + 1]),
                       __float_as_uint(dg[v][4 * q + 2]), __float_as_uint(dg[v][4 * q + 3])};
      reinterpret_cast<u32x4*>(p)[q] = w;
    }
  }
}

// dgamma[c] = sum over the partial rows: 32 columns and 16 runs of rows per workgroup, 8 rows'
// loads in flight, the runs then added in order.
constexpr int kSumRuns = 16;
__global__ __launch_bounds__(32 * kSumRuns) void k_norm_back_sum(const float* partial, float* dgamma, int64_t blocks,
                                                                 uint32_t cols) {
  __shared__ float s[kSumRuns][32];
  const uint32_t c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  const int64_t per = (blocks + kSumRuns - 1) / kSumRuns, lo = min(run * per, blocks), hi = min(lo + per, blocks);
  float sum = 0.f;
  if (c < cols) {
    int64_t b = lo;
    for (; b + 8 <= hi; b += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = partial[(uint64_t)(b + i) * cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
    for (; b < hi; ++b) sum += partial[(uint64_t)b * cols + c];
  }
  s[run][threadIdx.x & 31] = sum;
  __syncthreads();
  if (run == 0 && c < cols) {
#pragma unroll
    for (int q = 1; q < kSumRuns; ++q) sum += s[q][threadIdx.x];
    dgamma[c] = sum;
  }
}

// Vectors per thread and threads of a row of nvec vectors. Few rows (no more than compute
// units): one vector per thread where 1024 threads allow it, the shortest way through a row. More:
// two, so that more workgroups share a compute unit and one's loads overlap another's sums
// (8192 rows of 7168 bf16, 8 sources, 8-bit output: 205 against 230 us; four: 299 us). No more
// waves than the row fills.
struct RowShape {
  int v;
  uint32_t threads;
};
RowShape row_shape(uint32_t nvec, int64_t rows) {
  int v = rows > 256 && nvec > 128 ? 2 : 1;
  while ((uint32_t)v * kNormMaxThreads < nvec) v *= 2;
  const uint32_t per = (nvec + v - 1) / v;
  return {v, (per + 63) / 64 * 64};
}

template <int DT, int WMAX, bool F8>
void launch_norm_v(const NormArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.nvec, a.rows);
  const dim3 g((uint32_t)std::min<int64_t>(a.rows, kNormMaxBlocks)), b(r.threads);
  if (r.v == 1)
    launch_dp(k_norm<DT, WMAX, 1, F8>, g, b, 0, s, true, true, a);
  else if (r.v == 2)
    launch_dp(k_norm<DT, WMAX, 2, F8>, g, b, 0, s, true, true, a);
  else
    launch_dp(k_norm<DT, WMAX, 4, F8>, g, b, 0, s, true, true, a);
}

template <int DT, bool F8>
void launch_norm_w(const NormArgs& a, hipStream_t s) {
  if (a.world == 1)
    launch_norm_v<DT, 1, F8>(a, s);
  else if (a.world <= 4)
    launch_norm_v<DT, 4, F8>(a, s);
  else if (a.world <= 8)
    launch_norm_v<DT, 8, F8>(a, s);
  else
    launch_norm_v<DT, 16, F8>(a, s);
}

template <int DT>
void launch_norm_dt(const NormArgs& a, int out_dtype, hipStream_t s) {
  if (out_dtype == PLR_F8)
    launch_norm_w<DT, true>(a, s);
  else
    launch_norm_w<DT, false>(a, s);
}

template <int DT>
void launch_norm_back_dt(const NormBackArgs& a, int64_t blocks, hipStream_t s, bool last) {
  const RowShape r = row_shape(a.nvec, a.rows);
  const dim3 g((uint32_t)blocks), b(r.threads);
  if (r.v == 1)
    launch_dp(k_norm_back<DT, 1>, g, b, 0, s, true, last, a);
  else if (r.v == 2)
    launch_dp(k_norm_back<DT, 2>, g, b, 0, s, true, last, a);
  else
    launch_dp(k_norm_back<DT, 4>, g, b, 0, s, true, last, a);
}

}  // namespace

int64_t norm_back_blocks(int64_t rows) {
  // Two workgroups to a compute unit where two fit: more only add partial rows (8191 rows of
  // 7168 bf16: 84.5 us; with one 97.8, three 91.7, four 88.8 us).
  // (of no rows too: that one workgroup writes dgamma's zeros)
  return std::max<int64_t>(1, std::min<int64_t>(rows, kNormBackMaxBlocks));
}

hipError_t launch_norm(const NormArgs& a, int dtype, int out_dtype, hipStream_t s) {
  if (dtype == PLR_BF16)
    launch_norm_dt<PLR_BF16>(a, out_dtype, s);
  else if (dtype == PLR_F16)
    launch_norm_dt<PLR_F16>(a, out_dtype, s);
  else
    launch_norm_dt<PLR_F32>(a, out_dtype, s);
  return hipGetLastError();
}

hipError_t launch_norm_back(const NormBackArgs& a, int dtype, int64_t blocks, float* dgamma, hipStream_t s) {
  const bool one = blocks == 1;  // its partial row is the result
  if (dtype == PLR_BF16)
    launch_norm_back_dt<PLR_BF16>(a, blocks, s, one);
  else if (dtype == PLR_F16)
    launch_norm_back_dt<PLR_F16>(a, blocks, s, one);
  else
    launch_norm_back_dt<PLR_F32>(a, blocks, s, one);
  if (!one) {
    const uint32_t cols = a.nvec * (dtype == PLR_F32 ? 4 : 8);
    launch_dp(k_norm_back_sum, dim3((cols + 31) / 32), dim3(32 * kSumRuns), 0, s, false, true, (const float*)a.partial,
              dgamma, blocks, cols);
  }
  return hipGetLastError();
}

}  // namespace plr
