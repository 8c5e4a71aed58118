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

// Approximate keys of a token's experts from the hardware's exp2 and reciprocal, which
// differ from the exact ones by at most
//   2^-22 (the sigmoid: its slope times the errors of the product with log2 e,
//   the exponential and the reciprocal; |z| s (1 - s) < 0.23) + 2^-23 |key|
//   (the roundings of the two additions of the bias);
// then the picks by way of candidates (rows_group.h).
//
// Measured (route_pick_kernel): 16,384 tokens x 256 experts, top-8, 22.7 us with
// the exact key of every expert and 18.2 so; 4,095 x 896, top-16, BF16, 25.4
// and 15.8. Candidates gathered through LDS instead of lane permutations: 19.0
// and 17.1.
template <int kPer>
__device__ __forceinline__ bool pick_candidates(const float (&z)[kPer], const float (&bias)[kPer], int E, int k, int lane,
                                                int& id, float& s_mine, float& total) {
  float key[kPer];
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float e = __builtin_amdgcn_exp2f(z[j] * -1.44269504088896341f);
    key[j] = __builtin_amdgcn_rcpf(1.f + e) + bias[j];
    odd |= !(key[j] < __builtin_inff());  // a bias of minus infinity: never among the k, see T
  }
  if (__ballot(odd)) return false;
  const auto any = [&](int j) { return lane + kWave * j < E; };
  return pick_near<kPer>(key, z, bias, any, k, lane, [](float v) { return sigmoid_f32(v); }, id, s_mine, total);
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
