// moe_route_rows (include/moe_rows.h): biased sigmoid top-k of any number of
// tokens, and the routes grouped by expert.
//
// The picks are route_device.h's, one wave per token; the grouping is
// rows_group.h's. Up to 32 tokens one workgroup does all of it (one launch). Beyond, two or
// three: picks and counts per (chunk, expert), the running sums over the chunks
// where there are many, and the places. The bound is instructions, not memory:
// 16,384 tokens x 256 experts are 16 MB of logits (4 us), but some 370 vector
// instructions a token, 12 of the first launch's 18 us; the other two take 4.7
// and 4.3 us. One token: 4.5 us, all of it latency.
#include <hip/hip_runtime.h>

#include "rows_group.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// A bound that at least k of the wave's values reach, at most the k-th
// largest: the largest such value found bit by bit below the leading bits that
// all values share, ended as soon as exactly k reach it.
__device__ __forceinline__ uint32_t kth_bound(uint32_t v, int k) {
  const uint32_t hi = uniform(wave_max_u32(v)), d = hi ^ uniform(wave_min_u32(v));
  if (d == 0) return hi;
  int b = 31 - __builtin_clz(d), n_ge = -1;
  uint32_t T = b == 31 ? 0u : (hi & ~((2u << b) - 1u));
  for (; b >= 0 && n_ge != k; --b) {
    const uint32_t c = T | (1u << b);
    const int n = __popcll(__ballot(v >= c));
    if (n >= k) {
      T = c;
      n_ge = n;
    }
  }
  return T;
}

// One wave: the picks of a token by way of candidates. The exact keys (FP32
// sigmoids rounded from FP64) are needed for the few experts only that can be
// among the k largest. A key from the hardware's exp2 and reciprocal differs
// from the exact one by at most
//   2^-22 (the sigmoid: its slope times the errors of the product with log2 e,
//   the exponential and the reciprocal; |z| s (1 - s) < 0.23) + 2^-23 |key|
//   (the roundings of the two additions of the bias),
// both sides of which grow with the key, so an expert whose approximate key is
// more than 2^-20 + 2^-21 |T| below a bound T that k of them reach has k
// experts above it. The candidates, in expert order, one per lane, get their
// exact keys and are ranked by them. Returns false, having written nothing,
// where a key is NaN or infinity, fewer than k are finite, or the candidates do not fit the wave (equal
// scores of many experts): then every expert gets its exact key.
//
// Measured (route_pick_kernel): 16,384 tokens x 256 experts, top-8, 22.7 us with
// the exact key of every expert and 18.2 so; 4,095 x 896, top-16, BF16, 25.4
// and 15.8. Candidates gathered through LDS instead of lane permutations: 19.0
// and 17.1.
template <int kPer>
__device__ __forceinline__ bool pick_candidates(const float (&z)[kPer], const float (&bias)[kPer], int E, int k, int lane,
                                                int& id, float& s_mine, float& total) {
  float key[kPer];
  uint32_t top = 0u;  // 0: no expert (fewer than 64 of them, but k at least)
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float e = __builtin_amdgcn_exp2f(z[j] * -1.44269504088896341f);
    key[j] = __builtin_amdgcn_rcpf(1.f + e) + bias[j];
    odd |= !(key[j] < __builtin_inff());  // a bias of minus infinity: never among the k, see T
    top = max(top, lane + kWave * j < E ? ordered_key(key[j]) : 0u);
  }
  if (__ballot(odd)) return false;
  const uint32_t t = kth_bound(top, k);
  const float T = __uint_as_float((t & 0x80000000u) ? t ^ 0x80000000u : ~t);
  if (!(fabsf(T) < __builtin_inff())) return false;  // fewer than k finite keys
  const float low = T - (0x1p-20f + 0x1p-21f * fabsf(T));
  uint64_t sel[kPer];
  int n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    sel[j] = __ballot(lane + kWave * j < E && key[j] >= low);
    n += __popcll(sel[j]);
  }
  if (n >= kWave) return false;  // lane 63 takes the pushes of lanes without a candidate

  float cz = 0.f, cb = 0.f;
  int ce = 0, base = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint64_t m = sel[j];
    if (m != 0) {
      const int cnt = __popcll(m);
      const int below = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
      const int to = (((m >> lane) & 1ull) ? base + below : kWave - 1) * 4;
      const float rz = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(z[j])));
      const float rb = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(bias[j])));
      const int re = __builtin_amdgcn_ds_permute(to, lane + kWave * j);
      const bool here = lane >= base && lane < base + cnt;
      cz = here ? rz : cz;
      cb = here ? rb : cb;
      ce = here ? re : ce;
      base += cnt;
    }
  }
  const float score = sigmoid_f32(cz);
  const uint32_t mine = lane < n ? ordered_key(score + cb) : 0u;
  int rank = 0;
#pragma unroll 1  // unrolled, the compiler compares with all 64 lanes
  for (int q0 = 0; q0 < n; q0 += 8) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {  // lanes past n: the key 0, below every candidate's
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, q0 + q);
      rank += other > mine || (other == mine && q0 + q < lane) ? 1 : 0;
    }
  }
  const int to = (lane < n && rank < k ? rank : kWave - 1) * 4;
  id = __builtin_amdgcn_ds_permute(to, ce);
  s_mine = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(score)));
  total = 0.f;
  for (int r0 = 0; r0 < k; r0 += 8) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s_mine), r0 + q));
#pragma unroll
    for (int q = 0; q < 8; ++q) total = r0 + q < k ? total + v[q] : total;
  }
  return true;
}

// The workgroup's chunk of n tokens from t0 on, a token per wave at a time (the
// next one's logits on their way): ids and weights written, the picks also to
// `picks` (LDS, [n * k] local experts, -1 where not local, or nullptr), and
// mask[e] (LDS, [local_experts]) = the chunk's tokens that picked local expert
// e. Barriers inside, one behind the last write.
template <int kPer>
__device__ __forceinline__ void route_chunk(const moe_route_args& a, int t0, int n, int* picks, unsigned long long* mask) {
  const int lane = threadIdx.x & (kWave - 1);
  const bool bf16 = a.logits_dtype == MOE_DTYPE_BF16;
  int at[kPer];
  float bias[kPer], next[kPer];
  const auto request = [&](int i) {
    const size_t row = (size_t)(t0 + i) * a.E;
    load_logits<kPer>(bf16 ? (const void*)((const uint16_t*)a.logits + row) : (const void*)((const uint32_t*)a.logits + row),
                      bf16, at, next);
  };
#pragma unroll
  for (int j = 0; j < kPer; ++j) at[j] = min(lane + kWave * j, a.E - 1);
  int i = threadIdx.x / kWave;
  if (i < n) request(i);
#pragma unroll
  for (int j = 0; j < kPer; ++j) bias[j] = a.bias[at[j]];
  for (int e = threadIdx.x; e < a.local_experts; e += kRouteThreads) mask[e] = 0ull;
  __syncthreads();
  for (; i < n; i += kRouteWaves) {
    float z[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) z[j] = next[j];
    if (i + kRouteWaves < n) request(i + kRouteWaves);
    int id;
    float s, total;
    if (!pick_candidates<kPer>(z, bias, a.E, a.k, lane, id, s, total)) {
      float score[kPer];
      uint32_t key[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        score[j] = sigmoid_f32(z[j]);
        key[j] = ordered_key(score[j] + bias[j]);
      }
      pick_top_k<kPer>(key, score, a.E, a.k, lane, id, s, total);
    }
    if (lane < a.k) {
      const size_t r = (size_t)(t0 + i) * a.k + lane;
      a.ids[r] = id;
      a.weights[r] = pick_weight(s, total, a.routed_scale);
      const int e = id - a.local_begin;
      const bool local = e >= 0 && e < a.local_experts;
      if (local) atomicOr(&mask[e], 1ull << i);
      if (picks) picks[i * a.k + lane] = local ? e : -1;
    }
  }
  __syncthreads();
}

template <int kPer>
__global__ __launch_bounds__(kRouteThreads) void route_one_kernel(moe_route_args a) {
  __shared__ RouteShared sm;
  route_chunk<kPer>(a, 0, a.T, sm.picks, sm.mask);
  group_one(a, sm);
}

// Two workgroups a CU where the logits of a lane leave registers for them (20.3
// us with one, 18.2 with two, for 256 experts).
template <int kPer>
__global__ __launch_bounds__(kRouteThreads, kPer <= 4 ? 8 : 4) void route_pick_kernel(moe_route_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  const int chunk = chunk_tokens(a.T), t0 = blockIdx.x * chunk, n = min(chunk, a.T - t0);
  route_chunk<kPer>(a, t0, n, nullptr, mask);
  write_counts(a, mask);
}

template <int kPer>
void launch_route(const moe_route_args& a, hipStream_t stream) {
  launch_grouping(a, route_one_kernel<kPer>, route_pick_kernel<kPer>, a, stream);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_route_rows_workspace(int32_t T, int32_t local_experts) {
  using namespace moe;
  if (T <= kOneLaunch || local_experts <= 0) return 0;
  const size_t chunk = chunk_tokens(T), chunks = ((size_t)T + chunk - 1) / chunk;
  return (chunks + 1) * (size_t)local_experts * sizeof(int);
}

int moe_route_rows(const moe_route_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_route_args& a = *args;
  const int rc = check_route(a, true);
  if (rc != MOE_DECODE_OK) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int per = (a.E + kWave - 1) / kWave;
  if (a.T == 0)
    hipLaunchKernelGGL(route_none_kernel, dim3(1), dim3(kRouteThreads), 0, s, a.offsets, a.local_experts + 1);
  else if (per <= 1)
    launch_route<1>(a, s);
  else if (per <= 2)
    launch_route<2>(a, s);
  else if (per <= 4)
    launch_route<4>(a, s);
  else if (per <= 8)
    launch_route<8>(a, s);
  else
    launch_route<16>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}

}  // extern "C"
