// Low-rank adapters of many requests beside a shared projection:
//   y_s[i] += scale_g B_{s,g} (A_{s,g} x[i]) for the rows i of adapter g, several layers of one x.
// Two launches: t = A x (one warp per row, layer and rank index) into the workspace, then y += B t.
#include <algorithm>

#include "ql_internal.cuh"

namespace {

constexpr int MAX_LAYERS = 4;

struct Layers {
  const uint16_t *A[MAX_LAYERS], *B[MAX_LAYERS];
  void *y[MAX_LAYERS];
  int N[MAX_LAYERS];
};

// the group of position p (offsets clamped to [0, T]), -1 for none
__device__ __forceinline__ int group_at(const int32_t *offsets, int G, int p, int T) {
  int lo = 0, hi = G;   // the last g with offsets[g] <= p
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (offsets[mid] <= p) lo = mid; else hi = mid - 1;
  }
  return lo < G && offsets[lo] <= p && p < offsets[lo + 1] ? lo : -1;
}

__global__ void __launch_bounds__(256)
    lora_shrink_plain_kernel(const Layers L, int S, const uint16_t *x, const int32_t *order,
                             const int32_t *offsets, const float *scale, int G, int T, int r,
                             int K, float *t) {
  const int lane = threadIdx.x & 31;
  qld::pdl_trigger();
  qld::pdl_wait();
  const int64_t units = (int64_t)T * S * r;
  for (int64_t u = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; u < units;
       u += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    const int p = (int)(u / (S * r)), s = (int)(u / r % S), j = (int)(u % r);
    const int g = group_at(offsets, G, p, T), row = order[p];
    if (g < 0 || (unsigned)row >= (unsigned)T) continue;
    const uint16_t *a = L.A[s] + ((int64_t)g * r + j) * K, *xr = x + (int64_t)row * K;
    float acc = 0.f;
    for (int k = lane; k < K; k += 32) acc = qld::fma_bf16(a[k], xr[k], acc);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    if (lane == 0) t[((int64_t)s * T + p) * r + j] = scale ? acc * scale[g] : acc;
  }
}

__global__ void __launch_bounds__(256)
    lora_expand_plain_kernel(const Layers L, int S, const int32_t *order, const int32_t *offsets,
                             int ydt, int G, int T, int r, const float *t) {
  qld::pdl_trigger();
  qld::pdl_wait();
  for (int s = 0; s < S; ++s) {
    const int N = L.N[s];
    const int64_t units = (int64_t)T * N;
    for (int64_t u = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; u < units; u += (int64_t)gridDim.x * blockDim.x) {
      const int p = (int)(u / N), n = (int)(u - (int64_t)p * N);
      const int g = group_at(offsets, G, p, T), row = order[p];
      if (g < 0 || (unsigned)row >= (unsigned)T) continue;
      const uint16_t *b = L.B[s] + ((int64_t)g * N + n) * r;
      const float *tp = t + ((int64_t)s * T + p) * r;
      float acc = 0.f;
      for (int j = 0; j < r; ++j) acc = fmaf(qld::bf16_to_f32(b[j]), tp[j], acc);
      if (ydt == QL_OUT_F32) {
        static_cast<float *>(L.y[s])[(int64_t)row * N + n] += acc;
      } else {
        uint16_t *q = static_cast<uint16_t *>(L.y[s]) + (int64_t)row * N + n;
        *q = qld::f32_to_bf16_rn(qld::bf16_to_f32(*q) + acc);
      }
    }
  }
}

}  // namespace

namespace ql {

size_t lora_workspace_size(int S, int T, int r) { return ((size_t)S * T * r * sizeof(float) + 255) / 256 * 256; }

ql_status lora_add_launch(const lora_layer *layers, int S, const uint16_t *x, const int32_t *order,
                          const int32_t *offsets, const float *scale, ql_out_dtype ydt, int G, int T, int r, int K,
                          void *ws, cudaStream_t s) {
  Layers L{};
  int64_t cols = 0;
  for (int i = 0; i < S; ++i) {
    L.A[i] = layers[i].A;
    L.B[i] = layers[i].B;
    L.y[i] = layers[i].y;
    L.N[i] = layers[i].N;
    cols = std::max<int64_t>(cols, layers[i].N);
  }
  float *t = static_cast<float *>(ws);
  const int64_t most = (int64_t)sm_count() * 8;
  launch(lora_shrink_plain_kernel, (int)std::min<int64_t>(((int64_t)T * S * r + 7) / 8, most), 256, 0, s, L, S, x, order,
         offsets, scale, G, T, r, K, t);
  launch(lora_expand_plain_kernel, (int)std::min<int64_t>((T * cols + 255) / 256, most), 256, 0, s, L, S, order, offsets,
         (int)ydt, G, T, r, t);
  return launch_status("lora_add");
}

}  // namespace ql
