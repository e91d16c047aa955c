// The weighted sum that ends a mixture-of-experts layer:
//   out[t] = residual[t] + sum_j weights[t][j] * y[t k + j],  j ascending, in fp32.
// Bound by memory: each row of y is read once.  A thread owns 8 columns of one token (16 bytes of
// bf16), so the k rows' loads of a thread are independent and all in flight at once; places
// without an expert are not read.
#include <algorithm>
#include <type_traits>

#include "ql_internal.cuh"

namespace {

constexpr int COLS = 8;

template <bool F32>
__device__ __forceinline__ void load8(const void *p, size_t i, float (&v)[COLS]) {
  if constexpr (F32) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = qld::bf16_to_f32(u[j] & 0xffffu);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float load1(const void *p, size_t i, bool f32) {
  return f32 ? static_cast<const float *>(p)[i] : qld::bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}

// VEC: N % 8 == 0, so that every row starts on 16 bytes; else one column per thread.
template <bool YF32, bool OF32, bool VEC>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const void *y, const int32_t *experts, const float *weights, const void *residual, void *out,
                       int64_t count, int per_row, int k, int N) {
  qld::pdl_trigger();
  qld::pdl_wait();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < count; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per_row;
    const int n = (int)(i - t * per_row) * (VEC ? COLS : 1);
    if constexpr (VEC) {
      float acc[COLS] = {};
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        if (__ldcg(experts + t * k + j) < 0) continue;
        const float w = __ldcg(weights + t * k + j);
        float v[COLS];
        load8<YF32>(y, (size_t)(t * k + j) * N + n, v);
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] = fmaf(w, v[c], acc[c]);
      }
      const size_t o = (size_t)t * N + n;
      if (residual) {
        float v[COLS];
        load8<OF32>(residual, o, v);
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] += v[c];
      }
      if constexpr (OF32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + o);
        p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      } else {
        uint32_t u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          u[c] = uint32_t(qld::f32_to_bf16_rn(acc[2 * c])) | (uint32_t(qld::f32_to_bf16_rn(acc[2 * c + 1])) << 16);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + o) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    } else {
      float acc = 0.f;
      for (int j = 0; j < k; ++j)
        if (__ldcg(experts + t * k + j) >= 0)
          acc = fmaf(__ldcg(weights + t * k + j), load1(y, (size_t)(t * k + j) * N + n, YF32), acc);
      const size_t o = (size_t)t * N + n;
      if (residual) acc += load1(residual, o, OF32);
      if (OF32)
        static_cast<float *>(out)[o] = acc;
      else
        static_cast<uint16_t *>(out)[o] = qld::f32_to_bf16_rn(acc);
    }
  }
}

}  // namespace

namespace ql {

ql_status moe_combine_launch(const void *y, ql_out_dtype ydt, const int32_t *experts, const float *weights,
                             const void *residual, void *out, ql_out_dtype odt, int T, int k, int N, cudaStream_t s) {
  auto go = [&](auto yf, auto of, auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    const int per_row = VEC ? N / COLS : N;
    const int64_t count = (int64_t)T * per_row;
    const int grid = (int)std::min<int64_t>((count + 255) / 256, (int64_t)sm_count() * 8);
    launch(moe_combine_kernel<decltype(yf)::value, decltype(of)::value, VEC>, grid, 256, 0, s, y, experts, weights,
           residual, out, count, per_row, k, N);
  };
  auto pick = [&](auto yf, auto of) {
    if (N % COLS == 0)
      go(yf, of, std::true_type{});
    else
      go(yf, of, std::false_type{});
  };
  if (ydt == QL_OUT_F32)
    odt == QL_OUT_F32 ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
  else
    odt == QL_OUT_F32 ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
  return launch_status("moe_combine");
}

}  // namespace ql
