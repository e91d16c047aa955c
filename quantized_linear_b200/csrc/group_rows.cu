// Rows grouped by an index: the plan (order, offsets) of a grouped product, and the router of a
// mixture-of-experts layer, which makes its plan in the same call.
//
// The plan is a stable counting sort of M small keys: position(i) = #{keys below key_i} + #{i' < i with
// the same key}.  A chunk of consecutive keys belongs to one CTA and a run of it to one warp; a
// warp ranks 32 keys at once with a match mask (equal keys to the left of a lane), so no atomic
// decides a place and the result depends on the keys alone.  Up to CHUNK_ONE keys run in one launch;
// more take two: the chunks' histograms, then every CTA sums the histograms before its own chunk
// (a few hundred KB from L2) and places its keys.  Both are bound by latency: the arrays are a few MB.
// Measured, cold L2: 8192 tokens of 128 experts, k = 8, routed and planned in 16.7 us (two launches); 32 tokens of 64
// experts in 7.3 (one), most of it the call.
#include <algorithm>
#include <type_traits>

#include "ql_internal.cuh"

namespace {

constexpr int CHUNK_ONE = 4096;    // keys one CTA places in a single launch
constexpr int CHUNK_MIN = 1024;    // keys per CTA otherwise, more when that would take over CHUNKS_MAX CTAs
constexpr int CHUNKS_MAX = 256;
constexpr int ONE_TOKENS = 64;     // tokens the router handles in a single launch
constexpr int ROUTE_MIN = 32;      // tokens per CTA otherwise: one per warp while the chunks stay few
constexpr int PLACE_THREADS = 1024;
constexpr unsigned FULL = 0xffffffffu;

struct Chunks {
  int size, count;
};
Chunks chunks_of(int M) {
  int size = std::max(CHUNK_MIN, (M + CHUNKS_MAX - 1) / CHUNKS_MAX);
  size = (size + 31) / 32 * 32;
  return {size, (M + size - 1) / size};
}
Chunks token_chunks_of(int T) {   // tokens per CTA of the router
  const int size = std::max(ROUTE_MIN, (T + CHUNKS_MAX - 1) / CHUNKS_MAX);
  return {size, (T + size - 1) / size};
}

size_t scatter_smem(int G) { return (size_t)(PLACE_THREADS / 32 + 2) * G * sizeof(int) + 16; }

__device__ __forceinline__ int key_of(const int32_t *index, int i, int end, int G) {
  if (i >= end) return -1;
  const int k = __ldcg(index + i);
  return (unsigned)k < (unsigned)G ? k : -1;
}

// Places keys [s0, s1) of the M keys.  hist: [nchunks][G] histograms of all chunks (nullptr: these are
// all keys); chunk: this CTA's.
__device__ void place_chunk(const int32_t *index, int M, int G, int s0, int s1, const int *hist, int nchunks,
                            int chunk, int32_t *__restrict__ order, int32_t *__restrict__ offsets,
                            unsigned char *smem) {
  int *base = reinterpret_cast<int *>(smem);                                   // [G + 1]
  int *before = base + G + 4;                                                  // [G]
  int *wh = before + G;                                                        // [warps][G]
  const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *mine = wh + (size_t)warp * G;
  for (int i = threadIdx.x; i < nw * G; i += blockDim.x) wh[i] = 0;
  for (int g = threadIdx.x; g < G; g += blockDim.x) base[g] = before[g] = 0;
  const int run = ((s1 - s0 + nw - 1) / nw + 31) / 32 * 32;
  const int r0 = min(s1, s0 + warp * run), r1 = min(s1, r0 + run);
  __syncthreads();
  for (int i = r0; i < r1; i += 32) {
    const int key = key_of(index, i + lane, r1, G);
    const unsigned same = __match_any_sync(FULL, key);
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // per group: the runs' counts become starts within the chunk; base gets the total over all chunks, before the sum of
  // the chunks in front of this one
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < nw; ++w) {
      const int c = wh[(size_t)w * G + g];
      wh[(size_t)w * G + g] = sum;
      sum += c;
    }
    if (!hist) base[g] = sum;
  }
  if (hist) {   // threads share out (chunk, group) pairs, so that a few loads in flight per thread cover them all
    const int g32 = (G + 31) / 32 * 32, segs = max(1, (int)blockDim.x / g32);
    for (int g = threadIdx.x % g32, seg = threadIdx.x / g32; g < G && seg < segs; g += g32) {
      int all = 0, mine_before = 0;
#pragma unroll 16
      for (int c = seg; c < nchunks; c += segs) {
        const int v = __ldcg(hist + (size_t)c * G + g);
        all += v;
        if (c < chunk) mine_before += v;
      }
      atomicAdd(base + g, all);            // integer sums: the order does not matter
      atomicAdd(before + g, mine_before);
    }
  }
  __syncthreads();
  if (warp == 0) {   // exclusive sum over the groups
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int v = g < G ? base[g] : 0;
      int s = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(FULL, s, d);
        if (lane >= d) s += u;
      }
      if (g < G) base[g] = carry + s - v;
      carry += __shfl_sync(FULL, s, 31);
    }
    if (lane == 0) base[G] = carry;
  }
  __syncthreads();
  if (chunk == 0)
    for (int g = threadIdx.x; g <= G; g += blockDim.x) offsets[g] = base[g];
  const int total = base[G];
  for (int i = r0; i < r1; i += 32) {
    const int key = key_of(index, i + lane, r1, G);
    const unsigned same = __match_any_sync(FULL, key);
    int at = -1;
    if (key >= 0) at = base[key] + before[key] + mine[key] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    if (at >= 0) order[at] = i + lane;
    __syncwarp();
  }
  for (int i = max(s0, total) + threadIdx.x; i < s1; i += blockDim.x) order[i] = -1;
}

__global__ void __launch_bounds__(1024)
    group_place_kernel(const int32_t *index, int M, int G, int size, const int *hist, int nchunks, int32_t *order,
                       int32_t *offsets) {
  extern __shared__ __align__(16) unsigned char smem[];
  qld::pdl_trigger();
  qld::pdl_wait();
  const int s0 = blockIdx.x * size, s1 = min(M, s0 + size);
  place_chunk(index, M, G, s0, s1, hist, nchunks, blockIdx.x, order, offsets, smem);
}

__global__ void __launch_bounds__(256) group_hist_kernel(const int32_t *index, int M, int G, int size, int *hist) {
  extern __shared__ int count[];
  qld::pdl_trigger();
  qld::pdl_wait();
  for (int g = threadIdx.x; g < G; g += blockDim.x) count[g] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * size, s1 = min(M, s0 + size);
  for (int i = s0 + threadIdx.x; i < s1; i += blockDim.x) {
    const int key = key_of(index, i, s1, G);
    if (key >= 0) atomicAdd(count + key, 1);   // integer sums: the order does not matter
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += blockDim.x) hist[(size_t)blockIdx.x * G + g] = count[g];
}

// ------------------------------------------------------------------------------------------ router
// One warp per token: lane l holds logits l, l + 32, ... as unsigned keys whose order is the order of
// the floats (NaN largest, -0 equal to +0), and each of the k rounds takes the largest key of the warp
// (redux) and the smallest index that holds it.  Taken and masked (-inf) entries have key 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  if (v == -__int_as_float(0x7f800000)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xffffffffu) return __int_as_float(0x7fffffff);
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
  return v;
}

template <int V>
__device__ __forceinline__ void route_token(const void *logits, int ldt, int64_t t, int E, int k, int normalize,
                                            int32_t *experts, float *weights, int *count) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    key[j] = 0;
    if (e < E)
      key[j] = order_key(ldt == QL_OUT_F32 ? __ldcg(static_cast<const float *>(logits) + t * E + e)
                                           : qld::bf16_to_f32(__ldcg(static_cast<const uint16_t *>(logits) + t * E + e)));
  }
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) best = max(best, key[j]);
  const float top = key_value(__reduce_max_sync(FULL, best));
  float all = 0.f;
  if (!normalize) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] != 0) all += expf(key_value(key[j]) - top);
    all = warp_sum(all);
  }
  uint32_t my_key = 0;
  int my_expert = -1;
  for (int r = 0; r < k; ++r) {
    best = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) best = max(best, key[j]);
    const uint32_t win = __reduce_max_sync(FULL, best);
    if (win == 0) break;   // fewer than k experts left
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int j = V - 1; j >= 0; --j)
      if (key[j] == win) at = lane + 32 * j;
    at = __reduce_min_sync(FULL, at);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (at == unsigned(lane + 32 * j)) key[j] = 0;
    if (lane == r) {
      my_key = win;
      my_expert = (int)at;
    }
  }
  const float e = my_expert >= 0 ? expf(key_value(my_key) - top) : 0.f;
  const float total = normalize ? warp_sum(e) : all;
  if (lane < k) {
    experts[t * k + lane] = my_expert;
    weights[t * k + lane] = my_expert >= 0 ? __fdiv_rn(e, total) : 0.f;
    if (count && my_expert >= 0) atomicAdd(count + my_expert, 1);
  }
}

// ONE: a single CTA routes every token and then places the slots; else each CTA routes `size`
// tokens and leaves the histogram of its slots.
template <int V, bool ONE>
__global__ void __launch_bounds__(1024)
    moe_route_kernel(const void *logits, int ldt, int T, int E, int k, int normalize, int size, int32_t *experts,
                     float *weights, int *hist, int32_t *order, int32_t *offsets) {
  extern __shared__ __align__(16) unsigned char smem[];
  int *count = ONE ? nullptr : reinterpret_cast<int *>(smem);
  qld::pdl_trigger();
  qld::pdl_wait();
  if constexpr (!ONE) {
    for (int g = threadIdx.x; g < E; g += blockDim.x) count[g] = 0;
    __syncthreads();
  }
  const int t1 = min(T, (int)(blockIdx.x + 1) * size);
  for (int t = blockIdx.x * size + (threadIdx.x >> 5); t < t1; t += blockDim.x >> 5)
    route_token<V>(logits, ldt, t, E, k, normalize, experts, weights, count);
  __syncthreads();
  if constexpr (ONE)
    place_chunk(experts, T * k, E, 0, T * k, nullptr, 1, 0, order, offsets, smem);
  else
    for (int g = threadIdx.x; g < E; g += blockDim.x) hist[(size_t)blockIdx.x * E + g] = count[g];
}

template <int V>
void launch_route(const void *logits, ql_out_dtype ldt, int T, int E, int k, int normalize, int32_t *experts,
                  float *weights, int *hist, int32_t *order, int32_t *offsets, cudaStream_t s) {
  if (T <= ONE_TOKENS) {
    const size_t smem = scatter_smem(E);
    if (smem > 40 * 1024) (void)ql::set_max_smem(moe_route_kernel<V, true>, (int)smem);
    ql::launch(moe_route_kernel<V, true>, 1, PLACE_THREADS, smem, s, logits, (int)ldt, T, E, k, normalize, T, experts, weights,
               hist, order, offsets);
  } else {
    const Chunks c = token_chunks_of(T);
    ql::launch(moe_route_kernel<V, false>, c.count, 1024, E * sizeof(int), s, logits, (int)ldt, T, E, k, normalize,
               c.size, experts, weights, hist, order, offsets);
  }
}

// the second launch: places the keys of every chunk
void launch_place(const int32_t *index, int M, int G, Chunks c, const int *hist, int32_t *order, int32_t *offsets,
                  cudaStream_t s) {
  const size_t smem = scatter_smem(G);
  if (smem > 40 * 1024) (void)ql::set_max_smem(group_place_kernel, (int)smem);
  ql::launch(group_place_kernel, std::max(1, c.count), PLACE_THREADS, smem, s, index, M, G, c.size, hist, c.count, order,
             offsets);
}

}  // namespace

namespace ql {

size_t group_rows_workspace_size(int M, int G) {
  if (M <= CHUNK_ONE) return 0;
  return ((size_t)chunks_of(M).count * G * sizeof(int) + 255) / 256 * 256;
}

ql_status group_rows_launch(const int32_t *index, int M, int G, int32_t *order, int32_t *offsets, void *ws,
                            cudaStream_t s) {
  if (M <= CHUNK_ONE) {
    launch_place(index, M, G, {std::max(M, 1), 1}, nullptr, order, offsets, s);
  } else {
    const Chunks c = chunks_of(M);
    int *hist = static_cast<int *>(ws);
    launch(group_hist_kernel, c.count, 256, G * sizeof(int), s, index, M, G, c.size, hist);
    launch_place(index, M, G, c, hist, order, offsets, s);
  }
  return launch_status("group_rows");
}

size_t moe_route_workspace_size(int T, int E, int k) {
  (void)k;
  if (T <= ONE_TOKENS) return 0;
  return ((size_t)token_chunks_of(T).count * E * sizeof(int) + 255) / 256 * 256;
}

ql_status moe_route_launch(const void *logits, ql_out_dtype ldt, int T, int E, int k, bool normalize, int32_t *experts,
                           float *weights, int32_t *order, int32_t *offsets, void *ws, cudaStream_t s) {
  int *hist = T <= ONE_TOKENS ? nullptr : static_cast<int *>(ws);
  auto go = [&](auto v) {
    launch_route<decltype(v)::value>(logits, ldt, T, E, k, normalize ? 1 : 0, experts, weights, hist, order, offsets, s);
  };
  if (E <= 32) go(std::integral_constant<int, 1>{});
  else if (E <= 64) go(std::integral_constant<int, 2>{});
  else if (E <= 128) go(std::integral_constant<int, 4>{});
  else if (E <= 256) go(std::integral_constant<int, 8>{});
  else if (E <= 512) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
  if (hist) {
    const Chunks c = token_chunks_of(T);
    launch_place(experts, T * k, E, {c.size * k, c.count}, hist, order, offsets, s);
  }
  return launch_status("moe_route");
}

}  // namespace ql
