// The router: the k largest logits of every token, their softmax, and the plan that
// orders (token, slot) pairs by expert and then by token; and its gradient.
//
// Choice. LANES lanes hold one token's logits, R consecutive experts each, as integers
// in the values' order (0: an expert that cannot be chosen). A round takes the maximum over
// the lanes (lane permutations, no LDS) and its holder gives it up. 16-bit values carry their
// expert below them; of binary32 ones the lowest lane that holds the maximum and its lowest
// register are taken: ties fall to the lowest expert either way, and values are compared
// as they are. 32768 tokens of 256 bf16 logits, k = 8, take 14.1 us (their bytes about 3), the
// plan's two kernels 4.0 and 5.6 us, the gradient 7.9 us. Of the choice's instructions, for a
// wave's 4 tokens, a round is 53 of the vector and 23 of the scalar unit; making the keys before it
// is about 220 and 140 (a pair of branches for each of a lane's 16 logits), half as much as all
// eight rounds, and the second of a lane's two loads is issued after the first one's keys.
//
// Plan. A workgroup takes 64 tokens; each chosen expert gets a 64-bit mask in LDS with a
// bit per token (an atomic or, whose order does not matter), so a pair's rank among the
// workgroup's pairs of that expert is the number of lower bits set. Pairs of at most 64
// tokens are planned by the same workgroup in the same launch. Otherwise the workgroups'
// counts go to the workspace, a second kernel turns them into prefix sums over the
// workgroups, and a third adds the experts' offsets.
#include "device_common.h"
#include "moe.h"
#include "wave.h"

namespace plr {

namespace {

constexpr int kThreads = 256;
// 64 tokens at once for up to 256 experts: 32768 x 256 tokens are 8 waves a SIMD
constexpr int kChoiceThreads = 1024;

// Integers in the order of the values; NaN and -infinity are 0, which is never chosen.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (!(x > -__builtin_inff())) return 0;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 becomes +0: equal values, equal integers
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

// 16-bit values: the value's order above 0xFFFF - expert, so that one maximum gives the
// value and the lowest expert that has it, and no two keys are equal.
template <int DT>
__device__ __forceinline__ uint32_t packed(uint32_t bits, uint32_t expert) {
  constexpr uint32_t INF = DT == PLR_BF16 ? 0x7F80 : 0x7C00;
  if ((bits & 0x7FFF) > INF || bits == (INF | 0x8000)) return 0;
  if (bits == 0x8000) bits = 0;  // -0 and +0 are equal
  return (((bits & 0x8000) ? bits ^ 0xFFFF : bits | 0x8000) << 16) | (0xFFFF - expert);
}
template <int DT>
__device__ __forceinline__ float unpacked(uint32_t key) {
  const uint32_t o = key >> 16, bits = (o & 0x8000) ? o & 0x7FFF : o ^ 0xFFFF;
  if constexpr (DT == PLR_BF16) return __uint_as_float(bits << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

template <int DT>
__device__ __forceinline__ uint32_t choice_key(uint32_t bits, uint32_t expert) {
  if constexpr (DT == PLR_F32)
    return ordered(__uint_as_float(bits));
  else
    return packed<DT>(bits, expert);
}

template <int LANES, typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, F f) {
  return LANES == 16 ? row16(v, f) : wave64(v, f);
}

// Exclusive prefix of the experts' counts in LDS (cnt -> base), by the first wave; lane
// l takes the consecutive experts [l * per, l * per + per). Returns the total.
__device__ __forceinline__ int scan_experts(const int* cnt, int* base, int experts) {
  const int lane = threadIdx.x, per = (experts + 63) / 64;
  int sum = 0;
  for (int e = lane * per; e < min(experts, (lane + 1) * per); ++e) sum += cnt[e];
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int t = __shfl_up(upto, d);
    if (lane >= d) upto += t;
  }
  int run = upto - sum;
  for (int e = lane * per; e < min(experts, (lane + 1) * per); ++e) {
    base[e] = run;
    run += cnt[e];
  }
  return __shfl(upto, 63);
}

// ONE: the whole call is this workgroup's 64 tokens. VECTORS: rows are whole aligned 16-byte
// vectors.
template <int DT, int LANES, int R, bool ONE, bool VECTORS>
__global__ __launch_bounds__(kChoiceThreads) void k_route(const RouteArgs a) {
  constexpr int PER = kChoiceThreads / LANES;  // tokens at a time
  __shared__ unsigned long long mask[kRouteMaxExperts];
  __shared__ int16_t chosen[kRouteTokens][kRouteMaxK];
  __shared__ int cnt[ONE ? kRouteMaxExperts : 1], base[ONE ? kRouteMaxExperts : 1];
  __shared__ int s_total;
  const uint32_t E = a.experts, k = a.k;
  for (uint32_t e = threadIdx.x; e < E; e += kChoiceThreads) mask[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int wave_lane = threadIdx.x & 63, first_lane = wave_lane - lane;
  const int64_t token0 = (int64_t)blockIdx.x * kRouteTokens;
  const int here = (int)min<int64_t>(kRouteTokens, a.tokens - token0);
  for (int t0 = 0; t0 < here; t0 += PER) {
    const int t = t0 + group;
    const bool live = t < here;
    const char* row = a.logits + (uint64_t)(token0 + (live ? t : 0)) * a.pitch;
    uint32_t key[R];
    constexpr int N = Elems<DT>::N;
    if (VECTORS) {
#pragma unroll
      for (int v = 0; v < R / N; ++v) {
        const uint32_t e = lane * R + v * N;
        u32x4 x = {0, 0, 0, 0};
        const bool in = live && e < E;
        if (in) x = reinterpret_cast<const u32x4*>(row)[e / N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t bits = N == 4 ? x[i % 4] : (x[i / 2 % 4] >> (16 * (i & 1))) & 0xFFFF;
          key[v * N + i] = in ? choice_key<DT>(bits, e + i) : 0;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t e = lane * R + i;
        key[i] = 0;
        if (live && e < E) {
          if constexpr (DT == PLR_F32)
            key[i] = choice_key<DT>(reinterpret_cast<const uint32_t*>(row)[e], e);
          else
            key[i] = choice_key<DT>(reinterpret_cast<const uint16_t*>(row)[e], e);
        }
      }
    }
    float mine = -__builtin_inff();  // the value of choice `lane`, kept by that lane
    int id = -1;
    for (uint32_t j = 0; j < k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < R; ++i) best = max(best, key[i]);
      const uint32_t top = over_lanes<LANES>(best, MaxU32());
      int expert;
      if constexpr (DT == PLR_F32) {
        // the lowest lane of this token that holds the maximum, its lowest register
        uint64_t holders = __ballot(best == top) >> first_lane;
        if (LANES < 64) holders &= (1ull << (LANES & 63)) - 1;
        const int winner = __builtin_ctzll(holders);
        int at = 0;
#pragma unroll
        for (int i = R - 1; i > 0; --i) at = key[i] == top ? i : at;
        at = key[0] == top ? 0 : at;
        expert = __shfl(lane * R + at, first_lane + winner);
        if (lane != winner) at = -1;
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = i == at ? 0 : key[i];
      } else {
        expert = 0xFFFF - (int)(top & 0xFFFF);
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = key[i] == top ? 0 : key[i];
      }
      if (lane == (int)j && top != 0) {
        if constexpr (DT == PLR_F32)
          mine = unordered(top);
        else
          mine = unpacked<DT>(top);
        id = expert;
      }
    }
    // softmax over the chosen, the first of which is the largest; the sum is taken over
    // the lanes in a fixed order
    const float most = __shfl(mine, first_lane);
    const float p = id >= 0 ? expf(mine - most) : 0.f;
    const float sum = __uint_as_float(over_lanes<LANES>(__float_as_uint(p), AddF32()));
    if (live && lane < (int)k) {
      const int64_t o = (token0 + t) * k + lane;
      a.ids[o] = id;
      a.weights[o] = id >= 0 ? p / sum : 0.f;
      chosen[t][lane] = (int16_t)id;
      if (id >= 0) atomicOr(&mask[id], 1ull << t);
    }
  }
  __syncthreads();
  if constexpr (!ONE) {
    for (uint32_t e = threadIdx.x; e < E; e += kChoiceThreads)
      a.counts[(uint64_t)blockIdx.x * E + e] = __builtin_popcountll(mask[e]);
    // the rank inside the workgroup, for the third kernel to complete
    for (uint32_t i = threadIdx.x; i < here * k; i += kChoiceThreads) {
      const int t = i / k, id = chosen[t][i % k];
      a.positions[token0 * k + i] = id < 0 ? -1 : __builtin_popcountll(mask[id] & ((1ull << t) - 1));
    }
  } else {
    for (uint32_t e = threadIdx.x; e < E; e += kChoiceThreads) cnt[e] = __builtin_popcountll(mask[e]);
    __syncthreads();
    if (threadIdx.x < 64) {
      const int total = scan_experts(cnt, base, (int)E);
      if (threadIdx.x == 0) {
        s_total = total;
        a.offsets[E] = total;
      }
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < E; e += kChoiceThreads) a.offsets[e] = base[e];
    for (uint32_t i = threadIdx.x; i < here * k; i += kChoiceThreads) {
      const int t = i / k, id = chosen[t][i % k];
      const int p = id < 0 ? -1 : base[id] + __builtin_popcountll(mask[id] & ((1ull << t) - 1));
      a.positions[i] = p;
      if (p >= 0) a.row_token[p] = t;
      if ((int)i >= s_total) a.row_token[i] = -1;
    }
  }
}

// Prefix sums over the workgroups, per expert: 16 experts and 64 runs of workgroups (a
// thread each) per workgroup here. A thread keeps up to 8 counts of its run in registers, so
// that up to 512 workgroups (32768 tokens) are read once.
constexpr int kScanExperts = 16, kScanRuns = 64, kScanKept = 8;
__global__ __launch_bounds__(kScanExperts* kScanRuns) void k_route_scan(const RouteArgs a) {
  __shared__ int sums[kScanRuns][kScanExperts];
  const uint32_t lane = threadIdx.x % kScanExperts, r = threadIdx.x / kScanExperts;
  const uint32_t e = blockIdx.x * kScanExperts + lane;
  const uint32_t per = (a.blocks + kScanRuns - 1) / kScanRuns;
  const uint32_t lo = min(r * per, a.blocks), hi = e < a.experts ? min(lo + per, a.blocks) : lo;
  int* const c = a.counts + e;
  int kept[kScanKept];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kScanKept; ++i) {
    kept[i] = lo + i < hi ? c[(uint64_t)(lo + i) * a.experts] : 0;
    sum += kept[i];
  }
  for (uint32_t b = lo + kScanKept; b < hi; ++b) sum += c[(uint64_t)b * a.experts];
  sums[r][lane] = sum;
  __syncthreads();
  int run = 0;
  for (uint32_t w = 0; w < r; ++w) run += sums[w][lane];
#pragma unroll
  for (int i = 0; i < kScanKept; ++i)
    if (lo + i < hi) {
      c[(uint64_t)(lo + i) * a.experts] = run;
      run += kept[i];
    }
  for (uint32_t b = lo + kScanKept; b < hi; ++b) {
    const int n = c[(uint64_t)b * a.experts];
    c[(uint64_t)b * a.experts] = run;
    run += n;
  }
  if (r == kScanRuns - 1 && e < a.experts) a.totals[e] = run;
}

__global__ __launch_bounds__(kThreads) void k_route_place(const RouteArgs a) {
  __shared__ int cnt[kRouteMaxExperts], base[kRouteMaxExperts];
  __shared__ int s_total;
  const uint32_t E = a.experts, k = a.k;
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) cnt[e] = a.totals[e];
  __syncthreads();
  if (threadIdx.x < 64) {
    const int total = scan_experts(cnt, base, (int)E);
    if (threadIdx.x == 0) s_total = total;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (uint32_t e = threadIdx.x; e < E; e += kThreads) a.offsets[e] = base[e];
    if (threadIdx.x == 0) a.offsets[E] = s_total;
  }
  const int64_t token0 = (int64_t)blockIdx.x * kRouteTokens;
  const int here = (int)min<int64_t>(kRouteTokens, a.tokens - token0);
  for (uint32_t i = threadIdx.x; i < here * k; i += kThreads) {
    const int64_t o = token0 * k + i;
    const int id = a.ids[o];
    if (id >= 0) {
      const int p = base[id] + a.counts[(uint64_t)blockIdx.x * E + id] + a.positions[o];
      a.positions[o] = p;
      a.row_token[p] = (int32_t)(token0 + i / k);
    }
    if (o >= s_total) a.row_token[o] = -1;
  }
}

// f(id, d) of every slot, lane S of a 16-lane row holding slot S and handing it to its row.
template <int S = 0, typename F>
__device__ __forceinline__ void for_slots(int id, float d, uint32_t k, F f) {
  if constexpr (S < kRouteMaxK) {
    if (S >= k) return;
    const int sid = __builtin_amdgcn_mov_dpp(id, 0x150 + S, 0xF, 0xF, true);  // lane S of the row
    const int sd = __builtin_amdgcn_mov_dpp((int)__float_as_uint(d), 0x150 + S, 0xF, 0xF, true);
    f(sid, __uint_as_float((uint32_t)sd));
    for_slots<S + 1>(id, d, k, f);
  }
}

// dl[t][id_j] = w_j (dw_j - sum_i w_i dw_i), 0 for the experts that were not chosen. 16
// lanes per token: lane j holds slot j, then the lanes walk the row.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_route_back(const RouteBackArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16;
  const bool live = t < a.tokens;
  int id = -1;
  float w = 0.f, dw = 0.f;
  if (live && lane < (int)a.k) {
    const int64_t o = t * a.k + lane;
    id = a.ids[o];
    if (id >= 0) {  // an empty slot's gradient is not looked at
      w = a.weights[o];
      dw = a.dweights[o];
    }
  }
  const float pull = __uint_as_float(row16(__float_as_uint(w * dw), AddF32()));
  const float d = w * (dw - pull);
  constexpr int N = Elems<DT>::N;
  char* row = a.dlogits + (uint64_t)(live ? t : 0) * a.pitch;
  for (uint32_t e0 = 0; e0 < a.experts; e0 += 16 * N) {
    const uint32_t e = e0 + lane * N;
    float g[N];
#pragma unroll
    for (int j = 0; j < N; ++j) g[j] = 0.f;
    for_slots(id, d, a.k, [&](int sid, float sd) {
#pragma unroll
      for (int j = 0; j < N; ++j) g[j] = sid == (int)(e + j) ? sd : g[j];
    });
    if (live && e < a.experts) {
      if (e + N <= a.experts && (a.pitch & 15) == 0) {
        st16(reinterpret_cast<u32x4*>(row) + e / N, Elems<DT>::narrow(g));
      } else {
        const u32x4 v = Elems<DT>::narrow(g);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (e + j < a.experts) {
            if constexpr (DT == PLR_F32)
              reinterpret_cast<uint32_t*>(row)[e + j] = v[j];
            else
              reinterpret_cast<uint16_t*>(row)[e + j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
          }
      }
    }
  }
}

template <int DT, bool ONE, bool VECTORS>
void launch_choice(const RouteArgs& a, hipStream_t s) {
  const dim3 g(a.blocks), b(kChoiceThreads);
  constexpr int FEW = DT == PLR_F32 ? 4 : 8;  // registers for up to 64 (128) experts: a vector
  if (a.experts <= 16 * FEW)
    launch_dp(k_route<DT, 16, FEW, ONE, VECTORS>, g, b, 0, s, true, ONE, a);
  else if (a.experts <= 256)
    launch_dp(k_route<DT, 16, 16, ONE, VECTORS>, g, b, 0, s, true, ONE, a);
  else
    launch_dp(k_route<DT, 64, 16, ONE, VECTORS>, g, b, 0, s, true, ONE, a);
}

template <int DT, bool ONE>
void launch_choice(const RouteArgs& a, hipStream_t s) {
  const uint64_t bytes = a.experts * (DT == PLR_F32 ? 4 : 2);
  if (((uintptr_t)a.logits | a.pitch | bytes) % 16 == 0)
    launch_choice<DT, ONE, true>(a, s);
  else
    launch_choice<DT, ONE, false>(a, s);
}

template <int DT>
void launch_route_dt(const RouteArgs& a, hipStream_t s) {
  if (a.blocks == 1) {
    launch_choice<DT, true>(a, s);
    return;
  }
  launch_choice<DT, false>(a, s);
  launch_dp(k_route_scan, dim3((a.experts + kScanExperts - 1) / kScanExperts), dim3(kScanExperts * kScanRuns), 0, s, false, false, a);
  launch_dp(k_route_place, dim3(a.blocks), dim3(kThreads), 0, s, false, true, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
  if (dtype == PLR_BF16)
    launch_route_dt<PLR_BF16>(a, s);
  else if (dtype == PLR_F16)
    launch_route_dt<PLR_F16>(a, s);
  else
    launch_route_dt<PLR_F32>(a, s);
  return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs& a, int dtype, hipStream_t s) {
  const dim3 g((uint32_t)((a.tokens + kThreads / 16 - 1) / (kThreads / 16))), b(kThreads);
  if (dtype == PLR_BF16)
    launch_dp(k_route_back<PLR_BF16>, g, b, 0, s, true, true, a);
  else if (dtype == PLR_F16)
    launch_dp(k_route_back<PLR_F16>, g, b, 0, s, true, true, a);
  else
    launch_dp(k_route_back<PLR_F32>, g, b, 0, s, true, true, a);
  return hipGetLastError();
}

}  // namespace plr
