// The weighted sum that ends a mixture-of-experts layer:
//   out[t] = residual[t] + sum_j weights[t][j] * y[t k + j],  j ascending, in fp32.
//
// Bound by memory: each row of y is read once.  Where rows start on 16 bytes (N % 8 == 0) a persistent CTA per SM
// keeps a ring of shared memory full of pieces of rows (2048 columns of up to eight rows and of the residual, one bulk
// copy each), so that some 200 KB are in flight per SM whatever the threads wait for; 256 threads own eight columns
// each and add.  4096 tokens of k = 8, N = 5120 take 74-80 us (5.3-5.7 TB/s, 88 with a cold L2); loads to registers
// took 104, as registers hold too little in flight, and at 16 tokens 12.3 us instead of 8.2 (cold).  Places without an
// expert are not read.
#include <algorithm>
#include <type_traits>

#include "ql_internal.cuh"
#include "grouped_ptx.cuh"

namespace {

using pairgemm::Waiter;

constexpr int COLS = 8;                      // columns per thread
constexpr int THREADS = 256;
constexpr int CHUNK = THREADS * COLS;        // columns of a piece
constexpr int AT = 8;                        // rows of a stage, besides the residual's
constexpr int RING_BYTES = 216 * 1024;

__device__ int g_combine_timeout = 0;

__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
}
template <bool F32>
__device__ __forceinline__ void unpack8(const uint32_t *u, float (&x)[COLS]) {
#pragma unroll
  for (int i = 0; i < COLS; ++i)
    x[i] = __uint_as_float(F32 ? u[i] : i % 2 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
}
template <bool F32>
__device__ __forceinline__ void piece8(uint32_t a, float (&x)[COLS]) {
  uint32_t v[2][4];
  lds128(a, v[0]);
  if (F32) lds128(a + 16, v[1]);
  unpack8<F32>(v[0], x);
}
template <bool F32>
__device__ __forceinline__ void store8(char *dst, const float (&acc)[COLS]) {
  if constexpr (F32) {
    reinterpret_cast<float4 *>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4 *>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = pairgemm::pack2(acc[2 * c], acc[2 * c + 1], pairgemm::OUT_BF16);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// Items: (token, chunk of columns), and of each the places in groups of AT, a stage each.
template <bool YF32, bool OF32>
__global__ void __launch_bounds__(THREADS + 32, 1)
    moe_combine_kernel(const void *y, const int32_t *experts, const float *weights, const void *residual, void *out, int k,
                       int N, unsigned chunks, unsigned items) {
  constexpr int YB = YF32 ? 4 : 2, OB = OF32 ? 4 : 2;
  constexpr int STAGE = CHUNK * (AT * YB + OB), ST = RING_BYTES / STAGE;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(8) uint64_t bars[2 * ST];
  __shared__ float wt[ST][AT];
  __shared__ unsigned on[ST];                // which rows of a stage were read
  __shared__ uint32_t abort_word;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t full = static_cast<uint32_t>(__cvta_generic_to_shared(bars)), empty = full + 8 * ST;
  const uint32_t aslot = static_cast<uint32_t>(__cvta_generic_to_shared(&abort_word));
  const Waiter wait{aslot, sm100::mapa_shared(aslot, 0)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, groups = (k + AT - 1) / AT;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      sm100::mbar_init(full + 8 * i, 1);
      sm100::mbar_init(empty + 8 * i, THREADS / 32);
    }
    abort_word = 0;
    sm100::fence_barrier_init();
  }
  qld::pdl_trigger();
  qld::pdl_wait();
  __syncthreads();
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
  if (warp == THREADS / 32) {
    // ------------------------------------------------------------ copies
    // Four stages at a time: lane 8 q + j has row j of stage q, and its place's expert and weight are read while the four
    // stages before are issued.
    const int q = lane >> 3, j8 = lane & 7;
    const unsigned units = (items - blockIdx.x + gridDim.x - 1) / gridDim.x * groups;  // gridDim.x <= items
    auto place = [&](unsigned u, unsigned &t, int &n0, int &g) {  // unit u of this CTA: token t, columns from n0, rows of group g
      const unsigned n = groups == 1 ? u : u / groups, i = blockIdx.x + n * gridDim.x;
      g = (int)(u - n * groups);
      t = i / chunks;
      n0 = (int)(i - t * chunks) * CHUNK;
    };
    auto look = [&](unsigned u, int &e, float &w) {
      e = -1;
      w = 0.f;
      unsigned t;
      int n0, g;
      place(u, t, n0, g);
      const int j = g * AT + j8;
      if (u < units && j < k) {
        const int64_t s = (int64_t)t * k + j;
        e = __ldcg(experts + s);
        w = __ldcg(weights + s);
      }
    };
    int e;
    float w;
    look(q, e, w);
    for (unsigned u = 0; u < units && ok; u += 4) {
      int e2;
      float w2;
      look(u + 4 + q, e2, w2);
      unsigned t;
      int n0, g;
      place(u + q, t, n0, g);
      const int cols = min(CHUNK, N - n0), j = g * AT + j8;
      const unsigned rows = __ballot_sync(0xffffffffu, e >= 0) >> (8 * q) & 255u;
      const bool res = g == groups - 1 && residual != nullptr;
      for (int p = 0; p < 4 && u + p < units; ++p) {
        if (!__all_sync(0xffffffffu, wait.wait(empty + 8 * st, ph ^ 1, false))) { ok = false; break; }
        if (q == p) {
          wt[st][j8] = w;
          if (j8 == 0) on[st] = rows;
        }
        __syncwarp();
        if (q == p && j8 == 0)
          sm100::mbar_arrive_expect_tx(full + 8 * st, __popc(rows) * cols * YB + (res ? cols * OB : 0));
        __syncwarp();
        const uint32_t dst = base + st * STAGE;
        if (q == p) {
          if (e >= 0)
            sm100::bulk_g2s(dst + j8 * CHUNK * YB, static_cast<const char *>(y) + (((size_t)t * k + j) * N + n0) * YB,
                            cols * YB, full + 8 * st);
          if (j8 == 0 && res)
            sm100::bulk_g2s(dst + AT * CHUNK * YB, static_cast<const char *>(residual) + ((size_t)t * N + n0) * OB, cols * OB,
                            full + 8 * st);
        }
        __syncwarp();
        if (++st == ST) {
          st = 0;
          ph ^= 1;
        }
      }
      e = e2;
      w = w2;
    }
  } else {
    // ------------------------------------------------------------ sums
    for (unsigned i = blockIdx.x; i < items && ok; i += gridDim.x) {
      const unsigned t = i / chunks;
      const int n = (int)(i - t * chunks) * CHUNK + threadIdx.x * COLS;
      float acc[COLS] = {};
      for (int g = 0; g < groups; ++g) {
        if (!__all_sync(0xffffffffu, wait.wait(full + 8 * st, ph, false))) { ok = false; break; }
        const uint32_t src = base + st * STAGE;
        const unsigned rows = on[st];
        if (n < N) {
#pragma unroll
          for (int j = 0; j < AT; ++j)
            if (rows >> j & 1) {
              const float w = wt[st][j];
              float x[COLS];
              piece8<YF32>(src + (j * CHUNK + threadIdx.x * COLS) * YB, x);
#pragma unroll
              for (int c = 0; c < COLS; ++c) acc[c] = fmaf(w, x[c], acc[c]);
            }
          if (g == groups - 1 && residual != nullptr) {
            float x[COLS];
            piece8<OF32>(src + AT * CHUNK * YB + threadIdx.x * COLS * OB, x);
#pragma unroll
            for (int c = 0; c < COLS; ++c) acc[c] += x[c];
          }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(empty + 8 * st);
        if (++st == ST) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok || n >= N) continue;
      store8<OF32>(static_cast<char *>(out) + ((size_t)t * N + n) * OB, acc);
    }
  }
  if (!ok) {
    atomicExch(&g_combine_timeout, 1);
    pairgemm::settle();
  }
}

__device__ __forceinline__ float load1(const void *p, size_t i, bool f32) {
  return f32 ? __ldcg(static_cast<const float *>(p) + i) : qld::bf16_to_f32(__ldcg(static_cast<const uint16_t *>(p) + i));
}

// Any N: rows that no bulk copy can start at.  Single columns, THREADS apart, so that a thread still has eight loads in
// flight per row (4096 tokens, N = 5119: 143 us; four rows ahead at 72 registers took twice that).
template <bool YF32, bool OF32>
__global__ void __launch_bounds__(THREADS)
    moe_combine_odd_kernel(const void *y, const int32_t *experts, const float *weights, const void *residual, void *out,
                           int k, int N, unsigned chunks) {
  qld::pdl_trigger();
  qld::pdl_wait();
  const unsigned t = blockIdx.x / chunks;
  const int n0 = (blockIdx.x - t * chunks) * CHUNK + threadIdx.x;
  float acc[COLS] = {};
#pragma unroll 2
  for (int j = 0; j < k; ++j) {
    const size_t s = (size_t)t * k + j;
    if (__ldcg(experts + s) < 0) continue;
    const float w = __ldcg(weights + s);
    float v[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) v[c] = n0 + c * THREADS < N ? load1(y, s * N + n0 + c * THREADS, YF32) : 0.f;
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[c] = fmaf(w, v[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const int n = n0 + c * THREADS;
    if (n >= N) break;
    const size_t o = (size_t)t * N + n;
    const float r = residual ? acc[c] + load1(residual, o, OF32) : acc[c];
    if (OF32)
      static_cast<float *>(out)[o] = r;
    else
      static_cast<uint16_t *>(out)[o] = qld::f32_to_bf16_rn(r);
  }
}

}  // namespace

namespace ql {

ql_status moe_combine_launch(const void *y, ql_out_dtype ydt, const int32_t *experts, const float *weights,
                             const void *residual, void *out, ql_out_dtype odt, int T, int k, int N, cudaStream_t s) {
  const int64_t items = (int64_t)T * ((N + CHUNK - 1) / CHUNK);
  if (items >= ((int64_t)1 << 31)) return fail(QL_ERR_UNSUPPORTED, "moe_combine: T * N is too large");
  auto pick = [&](auto yf, auto of) {
    constexpr bool YF = decltype(yf)::value, OF = decltype(of)::value;
    const unsigned chunks = (N + CHUNK - 1) / CHUNK;
    if (N % COLS == 0) {
      constexpr int stage = CHUNK * (AT * (YF ? 4 : 2) + (OF ? 4 : 2)), smem = RING_BYTES / stage * stage;
      if (set_max_smem(moe_combine_kernel<YF, OF>, smem) != cudaSuccess) return false;
      launch(moe_combine_kernel<YF, OF>, (int)std::min<int64_t>(items, sm_count()), THREADS + 32, smem, s, y, experts, weights,
             residual, out, k, N, chunks, (unsigned)items);
    } else {
      launch(moe_combine_odd_kernel<YF, OF>, (int)items, THREADS, 0, s, y, experts, weights, residual, out, k, N, chunks);
    }
    return true;
  };
  const bool yf = ydt == QL_OUT_F32, of = odt == QL_OUT_F32;
  if (!(yf ? (of ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{}))
           : (of ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{}))))
    return fail(QL_ERR_CUDA, "moe_combine: cannot reserve shared memory");
  return launch_status("moe_combine");
}

ql_status moe_combine_read_timeout(int *flag) {
  int zero = 0;
  if (cudaMemcpyFromSymbol(flag, g_combine_timeout, sizeof(int)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_combine_timeout, &zero, sizeof(int)) != cudaSuccess)
    return fail(QL_ERR_CUDA, "ql_check: cannot read the device timeout flag");
  return QL_OK;
}

}  // namespace ql
