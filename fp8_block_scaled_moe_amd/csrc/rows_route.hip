// moe_route_rows (include/moe_rows.h): biased sigmoid top-k of any number of
// tokens, and the routes grouped by expert.
//
// The picks are route_device.h's, one wave per token. The grouping is a
// counting sort by expert that is stable and has no order-dependent step: a
// token picks an expert at most once, so a chunk of 64 tokens keeps, per
// expert, a 64-bit mask of the tokens that picked it (LDS or-atomics: the
// same mask in any order), and a route's place is
//   offset of the expert + count of earlier chunks + tokens below in the mask.
// Up to 64 tokens one workgroup does all of it (one launch). Beyond, three:
// picks and counts per (chunk, expert), the running sums over the chunks,
// and the places. The bound is the FP64 sigmoid and the selection (VALU), not
// memory: 16 MB of logits for 16,384 tokens x 256 experts.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe_rows.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kChunk = 64;      // tokens per workgroup: the bits of a mask
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kScanExperts = 64;  // experts per workgroup of the chunk sums
constexpr int kScanParts = kRouteThreads / kScanExperts;

// One wave: the picks of token t; ids and weights written.
template <int kPer>
__device__ __forceinline__ void route_token(const moe_route_args& a, int t, int lane) {
  int at[kPer];
  float z[kPer], score[kPer];
  uint32_t key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) at[j] = min(lane + kWave * j, a.E - 1);
  load_logits<kPer>(a.logits_dtype == MOE_DTYPE_BF16
                        ? (const void*)((const uint16_t*)a.logits + (size_t)t * a.E)
                        : (const void*)((const uint32_t*)a.logits + (size_t)t * a.E),
                    a.logits_dtype == MOE_DTYPE_BF16, at, z);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    score[j] = sigmoid_f32(z[j]);
    key[j] = ordered_key(score[j] + a.bias[at[j]]);
  }
  int id;
  float s, total;
  pick_top_k<kPer>(key, score, a.E, a.k, lane, id, s, total);
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = id;
    a.weights[(size_t)t * a.k + lane] = pick_weight(s, total, a.routed_scale);
  }
}

// The workgroup's chunk: picks of its tokens.
template <int kPer>
__device__ __forceinline__ void route_chunk(const moe_route_args& a, int t0, int n) {
  for (int i = threadIdx.x / kWave; i < n; i += kRouteWaves) route_token<kPer>(a, t0 + i, threadIdx.x & (kWave - 1));
}

// Local expert of a route of the chunk, -1 where it is not local.
__device__ __forceinline__ int local_expert(const moe_route_args& a, int t0, int q) {
  const int e = a.ids[(size_t)t0 * a.k + q] - a.local_begin;
  return e >= 0 && e < a.local_experts ? e : -1;
}

// Masks of the chunk's tokens per local expert (mask [local_experts]). The
// ids were written by this workgroup or an earlier launch. Barriers inside.
__device__ __forceinline__ void chunk_masks(const moe_route_args& a, int t0, int n, unsigned long long* mask) {
  for (int e = threadIdx.x; e < a.local_experts; e += kRouteThreads) mask[e] = 0ull;
  __syncthreads();
  for (int q = threadIdx.x; q < n * a.k; q += kRouteThreads) {
    const int e = local_expert(a, t0, q);
    if (e >= 0) atomicOr(&mask[e], 1ull << (q / a.k));
  }
  __syncthreads();
}

// Exclusive sum over the workgroup's threads (v of thread e belongs to
// expert e); `total` is the sum of all. Barriers inside.
__device__ __forceinline__ int block_exclusive(int v, int* wave_sum, int& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int incl = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    incl += lane >= o ? up : 0;
  }
  if (lane == kWave - 1) wave_sum[wave] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) {
    before += w < wave ? wave_sum[w] : 0;
    total += wave_sum[w];
  }
  return before + incl - v;
}

// Places of the chunk's routes: base[e] = first place of the chunk's rows of
// local expert e.
__device__ __forceinline__ void place_routes(const moe_route_args& a, int t0, int n, const unsigned long long* mask,
                                             const int* base) {
  for (int q = threadIdx.x; q < n * a.k; q += kRouteThreads) {
    const int e = local_expert(a, t0, q), i = q / a.k;
    int p = -1;
    if (e >= 0) {
      p = base[e] + __popcll(mask[e] & ((1ull << i) - 1ull));
      a.rows[p] = t0 + i;
    }
    a.pos[(size_t)t0 * a.k + q] = p;
  }
}

template <int kPer>
__global__ __launch_bounds__(kRouteThreads) void route_one_kernel(moe_route_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  __shared__ int base[MOE_DECODE_MAX_EXPERTS], wave_sum[kRouteWaves];
  route_chunk<kPer>(a, 0, a.T);
  __syncthreads();  // the ids are read back by other waves of this workgroup
  chunk_masks(a, 0, a.T, mask);
  const int e = threadIdx.x;
  int total;
  const int first = block_exclusive(e < a.local_experts ? __popcll(mask[e]) : 0, wave_sum, total);
  if (e < a.local_experts) {
    base[e] = first;
    a.offsets[e] = first;
  }
  if (e == 0) a.offsets[a.local_experts] = total;
  __syncthreads();
  place_routes(a, 0, a.T, mask, base);
}

template <int kPer>
__global__ __launch_bounds__(kRouteThreads) void route_pick_kernel(moe_route_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  const int t0 = blockIdx.x * kChunk, n = min(kChunk, a.T - t0);
  route_chunk<kPer>(a, t0, n);
  __syncthreads();
  chunk_masks(a, t0, n, mask);
  int* count = static_cast<int*>(a.workspace) + a.local_experts + (size_t)blockIdx.x * a.local_experts;
  for (int e = threadIdx.x; e < a.local_experts; e += kRouteThreads) count[e] = __popcll(mask[e]);
}

// Running sums over the chunks, in place: each thread has one expert (its
// lane) and one part of the chunks. Workspace: totals [local_experts], then
// counts [chunks][local_experts].
__global__ __launch_bounds__(kRouteThreads) void route_sum_kernel(int* ws, int chunks, int experts) {
  __shared__ int part[kScanParts][kScanExperts];
  const int lane = threadIdx.x % kScanExperts, p = threadIdx.x / kScanExperts;
  const int e = blockIdx.x * kScanExperts + lane;
  const bool live = e < experts;
  const int c0 = (int)((int64_t)chunks * p / kScanParts), c1 = (int)((int64_t)chunks * (p + 1) / kScanParts);
  int* count = ws + experts + (live ? e : 0);
  int sum = 0;
  if (live)
    for (int c = c0; c < c1; ++c) sum += count[(size_t)c * experts];
  part[p][lane] = sum;
  __syncthreads();
  int run = 0;
  for (int q = 0; q < p; ++q) run += part[q][lane];
  if (!live) return;
  for (int c = c0; c < c1; ++c) {
    const int v = count[(size_t)c * experts];
    count[(size_t)c * experts] = run;
    run += v;
  }
  if (p == kScanParts - 1) ws[e] = run;
}

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(moe_route_args a) {
  __shared__ unsigned long long mask[MOE_DECODE_MAX_EXPERTS];
  __shared__ int base[MOE_DECODE_MAX_EXPERTS], wave_sum[kRouteWaves];
  const int t0 = blockIdx.x * kChunk, n = min(kChunk, a.T - t0);
  const int* ws = static_cast<const int*>(a.workspace);
  const int e = threadIdx.x;
  const bool live = e < a.local_experts;
  int total;
  const int first = block_exclusive(live ? ws[e] : 0, wave_sum, total);
  if (live) base[e] = first + ws[a.local_experts + (size_t)blockIdx.x * a.local_experts + e];
  if (blockIdx.x == 0) {
    if (live) a.offsets[e] = first;
    if (e == 0) a.offsets[a.local_experts] = total;
  }
  chunk_masks(a, t0, n, mask);
  place_routes(a, t0, n, mask, base);
}

template <int kPer>
void launch_route(const moe_route_args& a, hipStream_t stream) {
  if (a.T <= kChunk) {
    hipLaunchKernelGGL(route_one_kernel<kPer>, dim3(1), dim3(kRouteThreads), 0, stream, a);
    return;
  }
  const int chunks = (a.T + kChunk - 1) / kChunk;
  hipLaunchKernelGGL(route_pick_kernel<kPer>, dim3(chunks), dim3(kRouteThreads), 0, stream, a);
  hipLaunchKernelGGL(route_sum_kernel, dim3((a.local_experts + kScanExperts - 1) / kScanExperts), dim3(kRouteThreads), 0,
                     stream, static_cast<int*>(a.workspace), chunks, a.local_experts);
  hipLaunchKernelGGL(route_place_kernel, dim3(chunks), dim3(kRouteThreads), 0, stream, a);
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_route_rows_workspace(int32_t T, int32_t local_experts) {
  using namespace moe;
  if (T <= kChunk || local_experts <= 0) return 0;
  const size_t chunks = ((size_t)T + kChunk - 1) / kChunk;
  return (chunks + 1) * (size_t)local_experts * sizeof(int);
}

int moe_route_rows(const moe_route_args* args, void* stream) {
  using namespace moe;
  if (!args) return MOE_DECODE_ERR_INVALID_ARG;
  const moe_route_args& a = *args;
  if (a.T < 0 || a.k < 1 || a.E < 1 || a.local_begin < 0 || a.local_experts < 1 || !std::isfinite(a.routed_scale))
    return MOE_DECODE_ERR_INVALID_ARG;
  if (a.E > MOE_DECODE_MAX_EXPERTS || a.k > MOE_DECODE_MAX_TOP_K || a.k > a.E || a.T > MOE_ROWS_MAX_TOKENS ||
      (a.logits_dtype != MOE_DTYPE_F32 && a.logits_dtype != MOE_DTYPE_BF16))
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (a.local_experts > a.E || a.local_begin > a.E - a.local_experts) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a.offsets || misaligned4(a.offsets)) return MOE_DECODE_ERR_INVALID_ARG;
  if (a.T > 0) {
    if (!a.logits || !a.bias || !a.ids || !a.weights || !a.rows || !a.pos) return MOE_DECODE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a.logits) & (a.logits_dtype == MOE_DTYPE_BF16 ? 1u : 3u)) || misaligned4(a.bias) ||
        misaligned4(a.ids) || misaligned4(a.weights) || misaligned4(a.rows) || misaligned4(a.pos))
      return MOE_DECODE_ERR_INVALID_ARG;
    const size_t need = moe_route_rows_workspace(a.T, a.local_experts);
    if (need && (!a.workspace || misaligned4(a.workspace))) return MOE_DECODE_ERR_INVALID_ARG;
    if (a.workspace_bytes < need) return MOE_DECODE_ERR_SCRATCH_TOO_SMALL;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int per = (a.E + kWave - 1) / kWave;
  if (per <= 1)
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
