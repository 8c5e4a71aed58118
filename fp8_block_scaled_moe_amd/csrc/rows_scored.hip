// moe_route_rows_scored (include/moe_block.h): top-k of any number of tokens by
// sigmoid or softmax scores, limited to the best groups of experts, and the routes
// grouped by expert.
//
// One wave per token: lane l holds experts l + 64 j. The picks are those of the exact
// keys, FP32 roundings of FP64 scores. Softmax scores are exact for all experts, since
// the sum needs every exponential in FP64 anyway; sigmoid scores are the hardware's
// first, which choose groups (where the least of the chosen and the best of the others
// lie further apart than their errors) and candidates, and only the candidates get
// exact ones. The groups' largest keys are found through LDS, where a group's experts
// lie side by side. The grouping of the routes is rows_group.h's.
//
// Bound by its instructions and by a wave's chain of them: 16,384 tokens x 256 experts in
// 8 groups, some 535 vector instructions a token, 32 us in a graph (21 of them the picks, the
// two launches of the grouping 10; the logits alone would take 4); without groups 26, by
// softmax 35. 4,095 x 896 by softmax 27: every wave has one token, its loads, maximum,
// exponentials, sum, bound and candidates follow each other, and the waves wait for 58% of
// their cycles; the exponentials in FP64 are 2.5 of it (measured against FP32 ones). One
// token: 6 us.
#include <hip/hip_runtime.h>

#include "../../include/moe_block.h"
#include "rows_device.h"
#include "rows_group.h"

namespace moe {
namespace {

// exp(x) for x <= 0: 2^(n / 32) by table, where n is the nearest integer to 32 x / ln 2,
// and six terms for what is left (at most ln 2 / 64; the seventh is 2^-58). The 32 values
// of the table are the LDS's 64 banks, so lanes that differ in entry differ in bank.
// Thirteen FP64 instructions, where the library's exponential has twice as many.
constexpr int kExpParts = 32;
__device__ __forceinline__ double exp_below_0(double x, const double* table) {
  x = fmax(x, -800.0);  // 0 as FP32, and far below any sum's last bit
  const double n = rint(x * (kExpParts * 1.4426950408889634));
  double r = fma(n, -0x1.62e42fee00000p-6, x);  // ln 2 / 32 in two parts
  r = fma(n, -0x1.a39ef35793c76p-38, r);
  const double p = fma(r, fma(r, fma(r, fma(r, fma(r, fma(r, 1.0 / 720.0, 1.0 / 120.0), 1.0 / 24.0), 1.0 / 6.0), 0.5), 1.0), 1.0);
  const int i = (int)n;
  return ldexp(table[i & (kExpParts - 1)] * p, i >> 5);
}

// 1 / (1 + exp(-z)) in FP64, rounded to FP32; a NaN stays one.
__device__ __forceinline__ float sigmoid_of(float z, const double* table) {
  const double e = exp_below_0(-fabs((double)z), table);
  return z != z ? z : (float)((z < 0.f ? e : 1.0) / (1.0 + e));
}

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }

// The softmax of a token's logits, FP32 roundings of FP64 values. With a NaN or plus
// infinity among them every exponential counts as 0, and so all are 0 times infinity.
constexpr uint32_t kNan = 0xFFFFFFFFu;  // the key of a NaN of either sign
template <int kPer>
__device__ __forceinline__ void softmax_of(const float (&z)[kPer], int E, int lane, const double* table, float (&s)[kPer]) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) top = max(top, lane + kWave * j >= E ? 0u : z[j] != z[j] ? kNan : ordered_key(z[j]));
  const float m = key_value(wave_max_u32(top));
  const double from = m == -__builtin_inff() ? 0.0 : (double)m;
  double e[kPer], sum = 0.0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    e[j] = lane + kWave * j < E ? exp_below_0((double)z[j] - from, table) : 0.0;
    sum += e[j];
    if (j % 2) __builtin_amdgcn_sched_barrier(0);  // all at once, they would take the registers of the logits
  }
  sum = wave_sum_f64(sum);
  // of minus infinities alone the sum is 0 too: their scores are 0
  const double inv = m == -__builtin_inff() ? 0.0 : 1.0 / sum;
#pragma unroll
  for (int j = 0; j < kPer; ++j) s[j] = (float)(e[j] * inv);
}

// A group's two largest keys (b1 >= b2) with those of other lanes.
__device__ __forceinline__ void merge(float& b1, float& b2, float c1, float c2) {
  b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
  b1 = fmaxf(b1, c1);
}
template <int kControl>
__device__ __forceinline__ void merge_dpp(float& b1, float& b2) {  // by a permutation inside rows of 16
  const int c1 = __builtin_amdgcn_mov_dpp(__float_as_int(b1), kControl, 0xF, 0xF, false);
  const int c2 = __builtin_amdgcn_mov_dpp(__float_as_int(b2), kControl, 0xF, 0xF, false);
  merge(b1, b2, __int_as_float(c1), __int_as_float(c2));
}

// The groups that take part, as a mask of their first lanes (a group has `lanes` lanes,
// a power of two), by the keys. `near`: the keys are up to 2^-22 + 2^-23 |key| off;
// false where that leaves it open whether some group takes part. Without, equal groups
// go by their index. `keys`: LDS of the wave's own, 16-byte aligned.
template <int kPer>
__device__ __forceinline__ bool best_groups(const moe_route_scored_args& a, int lanes, const float (&key)[kPer], bool near, float* keys, int lane,
                                            uint64_t& in) {
  // opaque, so that nothing that follows from these is kept for the next token: where it was, it went
  // to scratch memory (16,384 tokens x 256 experts in 8 groups, 25.0 us with it and 21 without)
  int G = a.groups, size = a.route.E / a.groups;
  asm volatile("" : "+s"(G), "+s"(size), "+s"(lanes), "+v"(lane));
  const int g = lane >> (31 - __builtin_clz(lanes)), sub = lane & (lanes - 1);
#pragma unroll
  for (int j = 0; j < kPer; ++j) keys[lane + kWave * j] = key[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  float b1 = -__builtin_inff(), b2 = b1;  // the group's largest keys
  const float* const of_group = keys + min(g, G - 1) * size;
  if (size % (4 * lanes) == 0) {
#pragma unroll 1
    for (int i = 4 * sub; i < size; i += 4 * lanes) {
      const float4_t v = *reinterpret_cast<const float4_t*>(of_group + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        b2 = __builtin_amdgcn_fmed3f(b1, b2, v[q]);
        b1 = fmaxf(b1, v[q]);
      }
    }
  } else {
#pragma unroll 1
    for (int i = sub; i < size; i += 4 * lanes) {
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = of_group[min(i + q * lanes, size - 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float u = i + q * lanes < size ? v[q] : -__builtin_inff();
        b2 = __builtin_amdgcn_fmed3f(b1, b2, u);
        b1 = fmaxf(b1, u);
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (lanes > 1) merge_dpp<0xB1>(b1, b2);   // swap neighbours
  if (lanes > 2) merge_dpp<0x4E>(b1, b2);   // swap pairs
  if (lanes > 4) merge_dpp<0x141>(b1, b2);  // half-row mirror
  if (lanes > 8) merge_dpp<0x140>(b1, b2);  // row mirror
#pragma unroll 1
  for (int o = 16; o < lanes; o <<= 1) merge(b1, b2, __shfl_xor(b1, o, kWave), __shfl_xor(b2, o, kWave));
  const float value = a.group_best == 2 ? b1 + b2 : b1;
  // near: a group's exact value lies between `low` and `high`. Its error follows the keys that are added, which may be
  // far larger than their sum: 2^-21 + 2^-23 (|b1| + |b2|) of theirs and both sums' roundings, half of `off` (an
  // infinite value, of experts kept out or of a sum past the range, is what it is). Eight times the error sent some
  // tokens of 4,095 x 896 in 8 groups the exact way: 28.3 us and not 26.
  float low = value, high = value;
  if (near && fabsf(value) < __builtin_inff()) {
    const float off = fmaf(0x1p-21f, a.group_best == 2 ? fabsf(b1) + fabsf(b2) : fabsf(b1), 0x1p-20f);
    low = value - off;
    high = value + off;
  }
  // groups surely ahead of the lane's own, and those that may be (itself among the latter)
  const auto ahead = [&](float other_low, int q) { return other_low > high || (!near && other_low == high && q < g); };
  const auto maybe = [&](float other_low, float other_high, int q) { return near ? other_high >= low : ahead(other_low, q) || q == g; };
  int sure = 0, may = 0;
  if (G <= lanes) {  // a group's lanes compare it with one other each
    const float other = __shfl(low, sub * lanes, kWave), over = near ? __shfl(high, sub * lanes, kWave) : other;
    const bool there = sub < G;
    const uint64_t s = __ballot(there && ahead(other, sub)), m = __ballot(there && maybe(other, over, sub));
    const uint64_t field = lanes == kWave ? ~0ull : (1ull << lanes) - 1ull;
    const int first = lane & ~(lanes - 1);
    sure = __popcll((s >> first) & field);
    may = __popcll((m >> first) & field);
  } else {
#pragma unroll 1
    for (int q = 0; q < G; ++q) {
      const float other = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(low), q * lanes));
      const float over = near ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(high), q * lanes)) : other;
      sure += ahead(other, q) ? 1 : 0;
      may += maybe(other, over, q) ? 1 : 0;
    }
  }
  in = __ballot(g < G && may <= a.top_groups);
  return __ballot(g < G && may > a.top_groups && sure < a.top_groups) == 0;
}

struct Pick {
  int id;
  float s, total;
};

// The picks of token t by the exact keys of all experts: for keys that are NaN or
// infinite, groups or candidates too close to tell apart. A NaN among the keys shows in
// all of the token's weights, whether its expert is picked or not.
template <int kPer, bool kGroups, bool kSoftmax>
__device__ __forceinline__ Pick pick_exactly(const moe_route_scored_args& sa, int t, int lanes, float* keys, const double* table) {
  const moe_route_args& a = sa.route;
  int lane = threadIdx.x & (kWave - 1);
  asm volatile("" : "+v"(lane), "+s"(t));  // as in best_groups
  const bool bf16 = a.logits_dtype == MOE_DTYPE_BF16;
  const size_t row = (size_t)t * a.E;
  int at[kPer];
  float z[kPer], score[kPer], key[kPer];
  uint32_t kv[kPer];
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) at[j] = min(lane + kWave * j, a.E - 1);
  load_logits<kPer>(bf16 ? (const void*)((const uint16_t*)a.logits + row) : (const void*)((const uint32_t*)a.logits + row), bf16, at, z);
  if (kSoftmax) softmax_of<kPer>(z, a.E, lane, table, score);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (!kSoftmax) score[j] = sigmoid_of(z[j], table);
    key[j] = a.bias ? score[j] + a.bias[at[j]] : score[j];
    kv[j] = lane + kWave * j >= a.E ? 0u : key[j] != key[j] ? kNan : ordered_key(key[j]);
    nan |= key[j] != key[j];  // lanes past E have the last expert's
    __builtin_amdgcn_sched_barrier(0);
  }
  if (kGroups) {
    uint64_t in;
    best_groups<kPer>(sa, lanes, key, false, keys, lane, in);
#pragma unroll
    for (int j = 0; j < kPer; ++j) kv[j] = (in >> (at[j] / (a.E / sa.groups) * lanes)) & 1ull ? kv[j] : 0u;
  }
  Pick p;
  pick_top_k<kPer>(kv, score, a.E, a.k, lane, p.id, p.s, p.total);
  if (__ballot(nan) != 0) p.s = p.total = __builtin_nanf("");
  return p;
}

// As rows_route.hip's route_chunk, by scores and groups. `keys`: LDS, kPer * 64
// values a wave, where there are groups; `table`: LDS.
template <int kPer, bool kGroups, bool kSoftmax>
__device__ __forceinline__ void scored_chunk(const moe_route_scored_args& sa, int t0, int n, int* picks, unsigned long long* mask,
                                             float* keys, double* table) {
  const moe_route_args& a = sa.route;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const bool bf16 = a.logits_dtype == MOE_DTYPE_BF16;
  constexpr bool kAhead = kPer < 16;  // the next token's logits on their way: 16 a lane leave no registers for it
  const auto expert = [&](int j) { return min(lane + kWave * j, a.E - 1); };
  float bias[kPer], next[kPer];
  const auto request = [&](int i) {
    const size_t row = (size_t)(t0 + i) * a.E;
    int at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) at[j] = expert(j);
    load_logits<kPer>(bf16 ? (const void*)((const uint16_t*)a.logits + row) : (const void*)((const uint32_t*)a.logits + row),
                      bf16, at, next);
  };
  int i = __builtin_amdgcn_readfirstlane(wave);
  if (i < n) request(i);
#pragma unroll
  for (int j = 0; j < kPer; ++j) bias[j] = a.bias ? a.bias[expert(j)] : 0.f;
  int lanes = kWave;
  uint32_t group[(kPer + 3) / 4] = {};  // the first lanes of the experts' groups, a byte each
  if (kGroups) {
    while (lanes * sa.groups > kWave) lanes >>= 1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) group[j / 4] |= (uint32_t)(expert(j) / (a.E / sa.groups) * lanes) << (8 * (j % 4));
  }
  for (int e = threadIdx.x; e < a.local_experts; e += kRouteThreads) mask[e] = 0ull;
  if (threadIdx.x < kExpParts) table[threadIdx.x] = exp2((double)threadIdx.x / kExpParts);
  __syncthreads();
  const auto write = [&](int i, int id, float s, float total) {
    if (lane < a.k) {
      const size_t r = (size_t)(t0 + i) * a.k + lane;
      a.ids[r] = id;
      a.weights[r] = !sa.renormalise ? s * a.routed_scale : total == 0.f ? 0.f : pick_weight(s, total, a.routed_scale);
      const int e = id - a.local_begin;
      const bool local = e >= 0 && e < a.local_experts;
      if (local) atomicOr(&mask[e], 1ull << i);
      if (picks) picks[i * a.k + lane] = local ? e : -1;
    }
  };
  uint64_t left = 0;  // tokens of this wave that the candidates do not settle
  for (; i < n; i += kRouteWaves) {
    float z[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) z[j] = next[j];
    if (kAhead && i + kRouteWaves < n) request(i + kRouteWaves);
    int id;
    float s, total;
    uint64_t in_groups = ~0ull;
    const auto takes_part = [&](int j) { return ((in_groups >> (group[j / 4] >> (8 * (j % 4)) & 0xFFu)) & 1ull) != 0; };
    const auto in = [&](int j) { return lane + kWave * j < a.E; };
    const auto leave_out = [&](float (&key)[kPer]) {  // minus infinity: never among the candidates
#pragma unroll
      for (int j = 0; j < (kPer + 3) / 4; ++j) asm volatile("" : "+v"(group[j]));  // as in best_groups
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] = takes_part(j) ? key[j] : -__builtin_inff();
    };
    float key[kPer];
    bool done = false, odd = false;
    if (kSoftmax) softmax_of<kPer>(z, a.E, lane, table, z);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      key[j] = (kSoftmax ? z[j] : __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z[j] * -1.44269504088896341f))) + bias[j];
      odd |= !(key[j] < __builtin_inff());
    }
    if (__ballot(odd) == 0) {
      bool sure = true;
      if (kGroups) {
        sure = best_groups<kPer>(sa, lanes, key, !kSoftmax, keys + wave * kPer * kWave, lane, in_groups);
        leave_out(key);
      }
      const auto exact = [&](float v) { return kSoftmax ? v : sigmoid_of(v, table); };
      if (sure) done = pick_near<kPer>(key, z, bias, in, a.k, lane, exact, id, s, total);
    }
    if (done)
      write(i, id, s, total);
    else
      left |= 1ull << i;
    if (!kAhead && i + kRouteWaves < n) request(i + kRouteWaves);
  }
  for (; left != 0; left &= left - 1) {  // apart, so that it takes no registers from the usual way
    const int at = __builtin_ctzll(left);
    const Pick p = pick_exactly<kPer, kGroups, kSoftmax>(sa, t0 + at, lanes, keys + wave * kPer * kWave, table);
    write(at, p.id, p.s, p.total);
  }
  __syncthreads();
}

template <int kPer, bool kGroups, bool kSoftmax>
__global__ __launch_bounds__(kRouteThreads) void scored_one_kernel(moe_route_scored_args a) {
  __shared__ RouteShared sm;
  __shared__ alignas(16) float keys[kGroups ? kRouteWaves * kPer * kWave : 1];
  __shared__ double table[kExpParts];
  scored_chunk<kPer, kGroups, kSoftmax>(a, 0, a.route.T, sm.picks, sm.mask, keys, table);
  group_one(a.route, sm);
}

template <int kPer, bool kGroups, bool kSoftmax>
__global__ __launch_bounds__(kRouteThreads, kPer <= 4 ? 8 : 4) void scored_pick_kernel(moe_route_scored_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  __shared__ alignas(16) float keys[kGroups ? kRouteWaves * kPer * kWave : 1];
  __shared__ double table[kExpParts];
  const int chunk = chunk_tokens(a.route.T), t0 = blockIdx.x * chunk, n = min(chunk, a.route.T - t0);
  scored_chunk<kPer, kGroups, kSoftmax>(a, t0, n, nullptr, mask, keys, table);
  write_counts(a.route, mask);
}

template <int kPer, bool kGroups>
void launch_scored(const moe_route_scored_args& a, hipStream_t stream) {
  if (a.scores == MOE_SCORES_SOFTMAX)
    launch_grouping(a.route, scored_one_kernel<kPer, kGroups, true>, scored_pick_kernel<kPer, kGroups, true>, a, stream);
  else
    launch_grouping(a.route, scored_one_kernel<kPer, kGroups, false>, scored_pick_kernel<kPer, kGroups, false>, a, stream);
}

template <int kPer>
void launch_scored(const moe_route_scored_args& a, hipStream_t stream) {
  if (a.top_groups < a.groups)  // else every group takes part
    launch_scored<kPer, true>(a, stream);
  else
    launch_scored<kPer, false>(a, stream);
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
