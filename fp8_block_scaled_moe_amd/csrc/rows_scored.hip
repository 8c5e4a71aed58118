// moe_route_rows_scored (include/moe_block.h): top-k of any number of tokens by
// sigmoid or softmax scores, limited to the best groups of experts, and the routes
// grouped by expert.
//
// One wave per token: lane l holds experts l + 64 j. Every expert's score comes from
// FP64 and every key is exact, so the picks are those of the definition; the groups'
// two largest keys are found through LDS, where a group's experts lie side by side;
// the picks are route_device.h's, with keys of 0 (below every expert's) where the
// group takes no part. The grouping of the routes is rows_group.h's.
#include <hip/hip_runtime.h>

#include "../../include/moe_block.h"
#include "rows_device.h"
#include "rows_group.h"

namespace moe {
namespace {

// FP32 scores of a token's logits, rounded from FP64.
template <int kPer>
__device__ __forceinline__ void scores_of(const float (&z)[kPer], bool softmax, int E, int lane, float (&s)[kPer]) {
  if (!softmax) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j] = sigmoid_f32(z[j]);
    return;
  }
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) top = max(top, lane + kWave * j < E ? ordered_key(z[j]) : 0u);
  top = wave_max_u32(top);
  const float m = __uint_as_float((top & 0x80000000u) ? top ^ 0x80000000u : ~top);
  const double from = m == -__builtin_inff() ? 0.0 : (double)m;
  double e[kPer], sum = 0.0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    e[j] = lane + kWave * j < E ? exp((double)z[j] - from) : 0.0;
    sum += e[j];
  }
  sum = wave_sum_f64(sum);
  const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
  for (int j = 0; j < kPer; ++j) s[j] = (float)(e[j] * inv);
}

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }

// Clears the keys of experts outside the top_groups groups. at[j]: the first lane of
// the group of expert lane + 64 j (a group has `lanes` lanes, a power of two).
// `keys`: LDS of the wave's own.
template <int kPer>
__device__ __forceinline__ void limit_groups(const moe_route_scored_args& a, int lanes, const int (&at)[kPer], uint32_t* keys, int lane,
                                             uint32_t (&kv)[kPer]) {
  const int G = a.groups, size = a.route.E / G, g = lane / lanes;
#pragma unroll
  for (int j = 0; j < kPer; ++j) keys[lane + kWave * j] = kv[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  uint32_t b1 = 0u, b2 = 0u;  // the group's largest keys
  if (g < G)
    for (int i = lane & (lanes - 1); i < size; i += lanes) {
      const uint32_t v = keys[g * size + i];
      b2 = max(b2, min(b1, v));
      b1 = max(b1, v);
    }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int o = 1; o < lanes; o <<= 1) {
    const uint32_t c1 = __shfl_xor(b1, o, kWave), c2 = __shfl_xor(b2, o, kWave);
    b2 = max(max(b2, c2), min(b1, c1));
    b1 = max(b1, c1);
  }
  const uint32_t mine = ordered_key(a.group_best == 2 ? key_value(b1) + key_value(b2) : key_value(b1));
  int rank = 0;
  for (int q = 0; q < G; ++q) {
    const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, q * lanes);
    rank += other > mine || (other == mine && q < g) ? 1 : 0;
  }
  const uint64_t in = __ballot(g < G && rank < a.top_groups);
#pragma unroll
  for (int j = 0; j < kPer; ++j) kv[j] = (in >> at[j]) & 1ull ? kv[j] : 0u;
}

// As rows_route.hip's route_chunk, by scores and groups. `keys`: LDS, kPer * 64
// values a wave, where there are groups.
template <int kPer, bool kGroups>
__device__ __forceinline__ void scored_chunk(const moe_route_scored_args& sa, int t0, int n, int* picks, unsigned long long* mask,
                                             uint32_t* keys) {
  const moe_route_args& a = sa.route;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const bool bf16 = a.logits_dtype == MOE_DTYPE_BF16;
  int at[kPer], group[kPer];
  float bias[kPer], next[kPer];
  const auto request = [&](int i) {
    const size_t row = (size_t)(t0 + i) * a.E;
    load_logits<kPer>(bf16 ? (const void*)((const uint16_t*)a.logits + row) : (const void*)((const uint32_t*)a.logits + row),
                      bf16, at, next);
  };
#pragma unroll
  for (int j = 0; j < kPer; ++j) at[j] = min(lane + kWave * j, a.E - 1);
  int i = wave;
  if (i < n) request(i);
#pragma unroll
  for (int j = 0; j < kPer; ++j) bias[j] = a.bias ? a.bias[at[j]] : 0.f;
  int lanes = kWave;
  if (kGroups) {
    while (lanes * sa.groups > kWave) lanes >>= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) group[j] = at[j] / (a.E / sa.groups) * lanes;
  }
  for (int e = threadIdx.x; e < a.local_experts; e += kRouteThreads) mask[e] = 0ull;
  __syncthreads();
  for (; i < n; i += kRouteWaves) {
    float z[kPer], score[kPer];
    uint32_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) z[j] = next[j];
    if (i + kRouteWaves < n) request(i + kRouteWaves);
    scores_of<kPer>(z, sa.scores == MOE_SCORES_SOFTMAX, a.E, lane, score);
#pragma unroll
    for (int j = 0; j < kPer; ++j)  // a NaN with every bit set would have the key 0
      key[j] = lane + kWave * j < a.E ? max(ordered_key(a.bias ? score[j] + bias[j] : score[j]), 1u) : 0u;
    if (kGroups) limit_groups<kPer>(sa, lanes, group, keys + wave * kPer * kWave, lane, key);
    int id;
    float s, total;
    pick_top_k<kPer>(key, score, a.E, a.k, lane, id, s, total);
    if (lane < a.k) {
      const size_t r = (size_t)(t0 + i) * a.k + lane;
      a.ids[r] = id;
      a.weights[r] = !sa.renormalise ? s * a.routed_scale : total == 0.f ? 0.f : pick_weight(s, total, a.routed_scale);
      const int e = id - a.local_begin;
      const bool local = e >= 0 && e < a.local_experts;
      if (local) atomicOr(&mask[e], 1ull << i);
      if (picks) picks[i * a.k + lane] = local ? e : -1;
    }
  }
  __syncthreads();
}

template <int kPer, bool kGroups>
__global__ __launch_bounds__(kRouteThreads) void scored_one_kernel(moe_route_scored_args a) {
  __shared__ RouteShared sm;
  __shared__ uint32_t keys[kGroups ? kRouteWaves * kPer * kWave : 1];
  scored_chunk<kPer, kGroups>(a, 0, a.route.T, sm.picks, sm.mask, keys);
  group_one(a.route, sm);
}

template <int kPer, bool kGroups>
__global__ __launch_bounds__(kRouteThreads) void scored_pick_kernel(moe_route_scored_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  __shared__ uint32_t keys[kGroups ? kRouteWaves * kPer * kWave : 1];
  const int chunk = chunk_tokens(a.route.T), t0 = blockIdx.x * chunk, n = min(chunk, a.route.T - t0);
  scored_chunk<kPer, kGroups>(a, t0, n, nullptr, mask, keys);
  write_counts(a.route, mask);
}

template <int kPer>
void launch_scored(const moe_route_scored_args& a, hipStream_t stream) {
  if (a.top_groups < a.groups)  // else every group takes part
    launch_grouping(a.route, scored_one_kernel<kPer, true>, scored_pick_kernel<kPer, true>, a, stream);
  else
    launch_grouping(a.route, scored_one_kernel<kPer, false>, scored_pick_kernel<kPer, false>, a, stream);
}

}  // namespace
}  // namespace moe

extern "C" int moe_route_rows_scored(const moe_route_scored_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_route_scored_args& a = *args;
  const int rc = check_route(a.route, false);
  if (rc != MOE_DECODE_OK) return rc;
  if (a.groups < 1 || a.top_groups < 1 || a.top_groups > a.groups || a.renormalise < 0 || a.renormalise > 1)
    return MOE_DECODE_ERR_INVALID_ARG;
  if (a.scores < MOE_SCORES_SIGMOID || a.scores > MOE_SCORES_SOFTMAX || a.groups > MOE_ROUTE_MAX_GROUPS || a.route.E % a.groups)
    return MOE_DECODE_ERR_UNSUPPORTED;
  const int size = a.route.E / a.groups;
  if (a.group_best < 1 || a.group_best > 2 || a.group_best > size || a.route.k > a.top_groups * size)
    return MOE_DECODE_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int per = (a.route.E + kWave - 1) / kWave;
  if (a.route.T == 0)
    hipLaunchKernelGGL(route_none_kernel, dim3(1), dim3(kRouteThreads), 0, s, a.route.offsets, a.route.local_experts + 1);
  else if (per <= 1)
    launch_scored<1>(a, s);
  else if (per <= 2)
    launch_scored<2>(a, s);
  else if (per <= 4)
    launch_scored<4>(a, s);
  else if (per <= 8)
    launch_scored<8>(a, s);
  else
    launch_scored<16>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP;
}
