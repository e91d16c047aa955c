// BenQ products grouped by an index, on the tensor cores: y[yr(i)] = W_g x[xr(i)] for the positions i of
// group g, and the gated pair h = silu(x G_g^T) * (x U_g^T), at every size from one position to many.
//
// The product is taken transposed: the MMA's M side is W (decoded), its N side the positions of one
// group, so a group of c positions costs ceil(c / 16) * 16 columns and no padding to a 128-row tile.  The
// work unit is a CTA pair (two SMs) and a tile of 2 x 128 rows of W by up to 384 positions.
//
// What bounds such a kernel is the shared-memory port (128 bytes per clock and SM): a table lookup moves 2
// of the 4 bytes of each bank, the X tile is written once by TMA and read by the tensor core.  Hence:
//   * decoded W never touches shared memory: a decoder thread owns one row of W, looks its codes up and
//     writes the bf16 pairs to tensor memory (tcgen05.st), from where the MMA takes A;
//   * each lane has the table of its row in a column of its own (word c * 32 + lane), so that 32 lanes
//     with 32 different tables never meet in a bank, and a lookup is a shift, an AND|OR and a load;
//   * the pair halves the X traffic: each SM loads and feeds half of the positions (cta_group::2).
// Per 64-wide K block and SM that is 256 + 48 wavefronts of lookups and codes, 48 of code writes and
// n/2 + n/2 of X for n positions, against 2 n clocks of MMA.
//
// Roles (512 threads per CTA): warp 0 loads X (rows gathered by x_rows, or tiles); warp 1 issues the MMAs
// (even CTA) or relays decoded blocks (odd CTA); warp 2 loads codes and tables; warps 4-7 drain the
// accumulators; warps 8-15, two warpgroups on alternate K blocks, decode.  Accumulators are two slots of
// 192 columns, so one tile's epilogue overlaps the next tile's MMAs.
//
// The gated form gives each warp of lanes 16 gate rows and the same features' 16 up rows: silu(g) * u then needs
// one exchange between the halves of a warp.
//
// The tensor core adds to its fp32 accumulator with truncation, about K * 1e-9 of the result after K
// inputs.  That is far below a bf16 rounding; for fp32 outputs each run of `seg` K blocks (512 inputs, more only
// above K = 12288) goes to an accumulator of its own and the epilogue adds the runs in fp32.
#include <cuda.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "ql_internal.cuh"
#include "pair_gemm.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace pairgemm;

constexpr int RW = 128;                        // rows of W per CTA and tile
constexpr int NS = 192;                        // positions per accumulator slot (the MMA's N)
constexpr int NT = 2 * NS;                     // positions per tile
constexpr int XR = NT / 2;                     // positions whose x rows one CTA loads
constexpr int SX = 4, SA = 4, SC = 3;          // stages: x, decoded W, codes
constexpr int X_BYTES = XR * 128;              // 24 KB: 64 bf16 per row
constexpr int X_BOX = 32;                      // rows per copy when rows are not gathered
constexpr int CKB = 3;                         // K blocks per code stage: rows of 144 bytes, a 16-byte load of 8
constexpr int C_ROW = CKB * 48;                // rows is free of bank conflicts
constexpr int C_BYTES = RW * C_ROW;            // 18 KB
constexpr int LUT_BYTES = RW * 128;            // 16 KB
constexpr int TBL_BYTES = 4 * 8192;            // lane-private tables: 4 warps of rows x [64][32] words
constexpr int NDW = 8;                         // decoder warps (two warpgroups)
constexpr int THREADS = 512;
constexpr int D_COL = 0, A_COL = NT;           // tensor memory columns: accumulators, then SA stages of 32
constexpr int MAX_SEG = NT / 16;               // runs of K blocks with an accumulator each (fp32 outputs)
constexpr int SEG_KB = 8;
constexpr int OFF_X = TBL_BYTES;
constexpr int OFF_C = OFF_X + SX * X_BYTES;
constexpr int OFF_LUT = OFF_C + SC * C_BYTES;
constexpr int OFF_BAR = OFF_LUT + LUT_BYTES;
constexpr int NBAR = 2 * SX + 3 * SA + 2 * SC + 2 + 4 + 8;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tensor-memory address, abort flag
constexpr int OFF_GRP = OFF_MISC + 16;         // token tiles before each group, int [G + 1]
static_assert(A_COL + 32 * SA <= 512, "tensor memory");
static_assert(OFF_X % 1024 == 0 && X_BYTES % 1024 == 0 && (XR / 2) * 128 % 1024 == 0, "swizzle atoms");
static_assert(OFF_C % 128 == 0 && C_BYTES % 128 == 0 && OFF_LUT % 128 == 0 && OFF_BAR % 8 == 0, "alignment");
constexpr size_t smem_bytes(int G) { return OFF_GRP + (size_t)(G + 1) * sizeof(int) + 8192; }
static_assert(smem_bytes(QL_MAX_GROUPS) <= 232448, "shared memory");
constexpr uint16_t PAIR = 0x3;

__device__ int g_grouped_timeout = 0;

struct Bars {
  uint32_t full_x, empty_x, dec_done, peer_a, empty_a, full_c, empty_c, lut_full, lut_empty, tbl_free, tbl_ready,
      acc_full, acc_empty;
  __device__ Bars(uint32_t b)
      : full_x(b), empty_x(full_x + 8 * SX), dec_done(empty_x + 8 * SX), peer_a(dec_done + 8 * SA),
        empty_a(peer_a + 8 * SA), full_c(empty_a + 8 * SA), empty_c(full_c + 8 * SC), lut_full(empty_c + 8 * SC),
        lut_empty(lut_full + 8), tbl_free(lut_empty + 8), tbl_ready(tbl_free + 8 * 4), acc_full(tbl_ready + 8 * 4),
        acc_empty(acc_full + 8 * 2) {}
};
static_assert(NBAR >= 2 * SX + 3 * SA + 2 * SC + 2 + 8 + 4, "barriers");

struct Args {
  const uint16_t *lut, *lut2;
  ql_groups g;
  void *y;
  int ydt, N, K, ntl, nt_max, seg, nseg;   // tiles of W rows per group, positions per tile, K blocks per run, runs
};

// One tile: W rows of index wt, positions [p0, p1) of group g; nh columns per MMA, one MMA per half.
struct Tile {
  int g, wt, p0, p1, nh, halves;
};

// Which accumulator slots a tile takes (the same sequence in the MMA issuer and the epilogue): a tile of one slot
// takes the other than the last, a tile of two takes both.  used[s] counts a slot's tiles for its barriers' phases.
struct Slots {
  int next = 0, used[2] = {0, 0};
  __device__ __forceinline__ int take(int slots) {
    const int s = slots == 2 ? 0 : next;
    next = slots == 2 ? 0 : next ^ 1;
    return s;
  }
  __device__ __forceinline__ void done(int first, int slots) {
    used[0] += (slots == 2 || first == 0);
    used[1] += (slots == 2 || first == 1);
  }
};

// (code J of a row's 64-code block) << 7: the offset of its entry in a lane-private table
template <int J>
__device__ __forceinline__ uint32_t entry_at(const uint32_t (&w)[12], uint32_t base) {
  constexpr int s = 6 * J, q = s >> 5, h = s & 31;
  uint32_t v;
  if constexpr (h < 7)
    v = w[q] << (7 - h);
  else if constexpr (h <= 26)
    v = w[q] >> (h - 7);
  else
    v = __funnelshift_r(w[q], w[q + 1], h - 7);
  return (v & 0x1F80u) | base;
}
template <int J>
struct Lookup {
  static __device__ __forceinline__ void run(const uint32_t (&w)[12], uint32_t base, uint32_t (&out)[32]) {
    Lookup<J - 2>::run(w, base, out);
    const uint32_t a = lds32(entry_at<J - 2>(w, base)), b = lds32(entry_at<J - 1>(w, base));
    out[(J - 2) / 2] = __byte_perm(a, b, 0x5410);
  }
};
template <>
struct Lookup<0> {
  static __device__ __forceinline__ void run(const uint32_t (&)[12], uint32_t, uint32_t (&)[32]) {}
};

__device__ __forceinline__ void lds128(uint32_t a, uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(a));
}

__device__ __forceinline__ void store_out(void *y, int ydt, size_t i, float v) {
  if (ydt == QL_OUT_F32)
    static_cast<float *>(y)[i] = v;
  else
    static_cast<uint16_t *>(y)[i] = qld::f32_to_bf16_rn(v);
}

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    benq_grouped_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_c,
                        const __grid_constant__ CUtensorMap map_c2, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const uint32_t sbase = (raw + 8191u) & ~8191u;   // the lookups OR the code into the table's address
  unsigned char *const sm = smem_raw + (sbase - raw);
  const Bars bar(sbase + OFF_BAR);
  const uint32_t tmem_slot = sbase + OFF_MISC;
  int *const cum = reinterpret_cast<int *>(sm + OFF_GRP);   // token tiles before each group
  const int G = a.g.G;
  const uint32_t rank = sm100::cluster_ctarank();
  const bool lead = rank == 0;
  const Waiter wt{tmem_slot + 4, sm100::mapa_shared(tmem_slot + 4, rank ^ 1u)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nkb = a.K / 64;
  bool ok = true;
  // a wait of a whole warp: no lane goes on alone when one gave up
  auto warp_wait = [&](uint32_t b, uint32_t parity, bool cluster_scope) {
    return __all_sync(0xffffffffu, wt.wait(b, parity, cluster_scope)) != 0;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < SX; ++s) {
      sm100::mbar_init(bar.full_x + 8 * s, 1);
      sm100::mbar_init(bar.empty_x + 8 * s, 1);
    }
    for (int s = 0; s < SA; ++s) {
      sm100::mbar_init(bar.dec_done + 8 * s, 4);
      sm100::mbar_init(bar.peer_a + 8 * s, 1);
      sm100::mbar_init(bar.empty_a + 8 * s, 1);
    }
    for (int s = 0; s < SC; ++s) {
      sm100::mbar_init(bar.full_c + 8 * s, 1);
      sm100::mbar_init(bar.empty_c + 8 * s, NDW);
    }
    sm100::mbar_init(bar.lut_full, 1);
    sm100::mbar_init(bar.lut_empty, NDW);
    for (int q = 0; q < 4; ++q) {
      sm100::mbar_init(bar.tbl_free + 8 * q, 2);
      sm100::mbar_init(bar.tbl_ready + 8 * q, 2);
    }
    for (int s = 0; s < 2; ++s) {
      sm100::mbar_init(bar.acc_full + 8 * s, 1);
      sm100::mbar_init(bar.acc_empty + 8 * s, 2 * 4);
    }
    sts32(tmem_slot + 4, 0);
    sm100::fence_barrier_init();
    sm100::prefetch_tensormap(&map_x);
    sm100::prefetch_tensormap(&map_c);
    if (GATED) sm100::prefetch_tensormap(&map_c2);
  }
  if (warp == 1) {
    __syncwarp();
    sm100::tmem_alloc_pair(tmem_slot, 512);
    sm100::tmem_relinquish_pair();
  }
  qld::pdl_trigger();
  qld::pdl_wait();   // the plan decides which weights are read, so every role needs it
  if (warp == 2) {   // token tiles before each group
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      int n = 0;
      if (g < G) {
        const int s0 = max(0, min(a.g.M, a.g.offsets[g])), s1 = max(0, min(a.g.M, a.g.offsets[g + 1]));
        n = s1 > s0 ? (s1 - s0 + a.nt_max - 1) / a.nt_max : 0;
      }
      int s = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
      }
      if (g < G) cum[g] = carry + s - n;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) cum[G] = carry;
  }
  sm100::tc_fence_before();
  sm100::cluster_sync();   // both CTAs' barriers initialised, tensor memory allocated, tiles counted
  sm100::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + OFF_MISC);
  const int nitems = cum[G] * a.ntl;
  auto tile_at = [&](int item) {
    Tile t;
    const int tt = item / a.ntl;
    t.wt = item - tt * a.ntl;
    int lo = 0, hi = G - 1;   // the group with cum[g] <= tt < cum[g + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid + 1] <= tt) lo = mid + 1; else hi = mid;
    }
    t.g = lo;
    const int s0 = max(0, min(a.g.M, __ldcg(a.g.offsets + lo))), s1 = max(0, min(a.g.M, __ldcg(a.g.offsets + lo + 1)));
    const int nt = cum[lo + 1] - cum[lo], per = (s1 - s0 + nt - 1) / nt;   // a group's tiles are of equal length
    t.p0 = s0 + (tt - cum[lo]) * per;
    t.p1 = min(s1, t.p0 + per);
    const int n = (per + 15) & ~15;
    t.halves = n > NS ? 2 : 1;
    t.nh = t.halves == 2 ? ((n / 2 + 15) & ~15) : n;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ x producer
    const uint32_t lead_full = sm100::mapa_shared(bar.full_x, 0);
    int it = 0;
    for (int wi = pair; wi < nitems && ok; wi += npairs) {
      const Tile t = tile_at(wi);
      const int nr = t.nh / 2;                 // rows of this CTA per half
      if (a.g.x_rows) {
        // lane l gathers rows 4 l .. 4 l + 3 of each half (nr <= 96: 24 lanes); a place past the tile or
        // a row out of range reads row 0, whose column is not stored
        const int groups = nr / 4;
        int4 r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = t.p0 + h * t.nh + (int)rank * nr + 4 * lane + e;
            int x = 0;
            if (h < t.halves && lane < groups && p < t.p1) x = __ldcg(a.g.x_rows + p) / a.g.x_div;
            v[e] = (unsigned)x < (unsigned)a.g.X ? x : 0;
          }
          r[h] = make_int4(v[0], v[1], v[2], v[3]);
        }
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % SX;
          if (it >= SX && !warp_wait(bar.empty_x + 8 * s, ((it / SX) & 1) ^ 1, true)) { ok = false; break; }
          if (lead && lane == 0) sm100::mbar_arrive_expect_tx(bar.full_x + 8 * s, 2 * t.halves * nr * 128);
          __syncwarp();
          if (lane < groups) {
            const uint32_t dst = sbase + OFF_X + s * X_BYTES + lane * 512;
            sm100::tma_gather4_pair(dst, &map_x, kb * 64, r[0], lead_full + 8 * s);
            if (t.halves == 2) sm100::tma_gather4_pair(dst + (XR / 2) * 128, &map_x, kb * 64, r[1], lead_full + 8 * s);
          }
        }
      } else if (lane == 0) {
        const int boxes = (nr + X_BOX - 1) / X_BOX;   // rows past the tile load other rows, whose columns are not stored
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int s = it % SX;
          if (it >= SX && !wt.wait(bar.empty_x + 8 * s, ((it / SX) & 1) ^ 1, true)) { ok = false; break; }
          if (lead) sm100::mbar_arrive_expect_tx(bar.full_x + 8 * s, 2 * t.halves * boxes * X_BOX * 128);
          for (int h = 0; h < t.halves; ++h)
            for (int b = 0; b < boxes; ++b)
              sm100::tma_load_2d_pair(sbase + OFF_X + s * X_BYTES + h * (XR / 2) * 128 + b * X_BOX * 128, &map_x, kb * 64,
                                      t.p0 + h * t.nh + (int)rank * nr + b * X_BOX, lead_full + 8 * s);
        }
      }
    }
  } else if (warp == 1) {
    if (lead && lane == 0) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      int it = 0;
      Slots sl;
      for (int wi = pair; wi < nitems && ok; wi += npairs) {
        const Tile t = tile_at(wi);
        const int slots = a.nseg > 1 ? 2 : t.halves, first_slot = sl.take(slots);
        for (int j = first_slot; j < first_slot + slots && ok; ++j)
          if (sl.used[j] > 0 && !wt.wait(bar.acc_empty + 8 * j, (sl.used[j] - 1) & 1, true)) ok = false;
        if (!ok) break;
        sm100::tc_fence_after();
        const uint32_t idesc = sm100::idesc_bf16_f32(256, t.nh);
        const uint32_t d0 = tmem + D_COL + first_slot * NS;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int sx = it % SX, sa = it % SA;
          if (!wt.wait(bar.full_x + 8 * sx, (it / SX) & 1, true) || !wt.wait(bar.dec_done + 8 * sa, (it / SA) & 1, false) ||
              !wt.wait(bar.peer_a + 8 * sa, (it / SA) & 1, true)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          const uint32_t at = tmem + A_COL + sa * 32, xb = sbase + OFF_X + sx * X_BYTES;
          const int run = kb / a.seg;
          const bool first = kb == run * a.seg;
          for (int h = 0; h < t.halves; ++h) {
            const uint32_t d = d0 + (a.nseg > 1 ? run * t.nh : h * NS);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              sm100::mma_f16kind_pair_ts(d, at + kk * 8, sm100::sw128_kmajor_desc(xb + h * (XR / 2) * 128 + kk * 32), idesc,
                                         (!first || kk > 0) ? 1u : 0u);
          }
          sm100::mma_commit_pair(bar.empty_x + 8 * sx, PAIR);
          sm100::mma_commit_pair(bar.empty_a + 8 * sa, PAIR);
        }
        if (!ok) break;
        for (int j = first_slot; j < first_slot + slots; ++j) sm100::mma_commit_pair(bar.acc_full + 8 * j, PAIR);
        sl.done(first_slot, slots);
      }
    } else if (!lead && lane == 0) {
      // ---------------------------------------------------------- forwarder (odd CTA)
      const uint32_t lead_peer = sm100::mapa_shared(bar.peer_a, 0);
      int it = 0;
      for (int wi = pair; wi < nitems && ok; wi += npairs)
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const int sa = it % SA;
          if (!wt.wait(bar.dec_done + 8 * sa, (it / SA) & 1, false)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          sm100::tc_fence_before();
          sm100::mbar_arrive_cluster(lead_peer + 8 * sa);
        }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ code and table producer
    if (lane == 0) {
      int ic = 0, tl = 0;
      const int ncs = (nkb + CKB - 1) / CKB;
      const int64_t rows = (int64_t)G * a.N;
      for (int wi = pair; wi < nitems && ok; wi += npairs, ++tl) {
        const Tile t = tile_at(wi);
        const int n0 = (t.wt * 2 + (int)rank) * (GATED ? RW / 2 : RW);
        const int64_t row0 = (int64_t)t.g * a.N + n0;
        if (tl > 0 && !wt.wait(bar.lut_empty, (tl - 1) & 1, false)) { ok = false; break; }
        // rows past this group's last load the next group's (or none): their results are not stored
        constexpr int per = GATED ? RW / 2 : RW;
        const int have = n0 < a.N ? (int)min((int64_t)per, rows - row0) : 0;
        if (have > 0) {
          sm100::mbar_arrive_expect_tx(bar.lut_full, (GATED ? 2 : 1) * have * 128);
          sm100::bulk_g2s(sbase + OFF_LUT, a.lut + row0 * 64, have * 128, bar.lut_full);
          if (GATED) sm100::bulk_g2s(sbase + OFF_LUT + per * 128, a.lut2 + row0 * 64, have * 128, bar.lut_full);
        } else {
          sm100::mbar_arrive(bar.lut_full);
        }
        for (int cs = 0; cs < ncs; ++cs, ++ic) {
          const int s = ic % SC;
          if (ic >= SC && !wt.wait(bar.empty_c + 8 * s, ((ic / SC) & 1) ^ 1, false)) { ok = false; break; }
          if (have > 0) {
            const uint32_t dst = sbase + OFF_C + s * C_BYTES;
            sm100::mbar_arrive_expect_tx(bar.full_c + 8 * s, C_BYTES);
            sm100::tma_load_2d(dst, &map_c, cs * C_ROW, (int)row0, bar.full_c + 8 * s);
            if (GATED) sm100::tma_load_2d(dst + C_BYTES / 2, &map_c2, cs * C_ROW, (int)row0, bar.full_c + 8 * s);
          } else {
            sm100::mbar_arrive(bar.full_c + 8 * s);
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ decoders
    const int q = warp & 3, wg = (warp >> 2) & 1;
    // the row of the staged codes and tables that this lane decodes
    const int row = GATED ? (lane < 16 ? 0 : RW / 2) + 16 * q + (lane & 15) : 32 * q + lane;
    const uint32_t tbl = sbase + q * 8192 + lane * 4;
    const uint32_t lutrow = sbase + OFF_LUT + row * 128;
    int it = 0, ic = 0, tl = 0;
    for (int wi = pair; wi < nitems && ok; wi += npairs, ++tl) {
      // the lane-private tables of this tile: each of the two warps of these rows writes half of them
      if (!warp_wait(bar.lut_full, tl & 1, false)) { ok = false; break; }
      uint32_t e[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) lds128(lutrow + wg * 64 + ((j + lane) & 3) * 16, e[4 * j], e[4 * j + 1], e[4 * j + 2], e[4 * j + 3]);
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(bar.lut_empty);
        sm100::mbar_arrive(bar.tbl_free + 8 * q);
      }
      if (!warp_wait(bar.tbl_free + 8 * q, tl & 1, false)) { ok = false; break; }   // both warps are past the last tile
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t to = tbl + (wg * 32 + ((j + lane) & 3) * 8) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sts32(to + 2 * i * 128, e[4 * j + i] & 0xffffu);
          sts32(to + (2 * i + 1) * 128, e[4 * j + i] >> 16);
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(bar.tbl_ready + 8 * q);
      if (!warp_wait(bar.tbl_ready + 8 * q, tl & 1, false)) { ok = false; break; }

      for (int kb0 = 0; kb0 < nkb && ok; kb0 += CKB, ++ic) {
        const int sc = ic % SC;
        if (!warp_wait(bar.full_c + 8 * sc, (ic / SC) & 1, false)) { ok = false; break; }
        const int kb1 = min(nkb, kb0 + CKB);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          if ((it & 1) != wg) continue;
          uint32_t w[12];
          const uint32_t cp = sbase + OFF_C + sc * C_BYTES + row * C_ROW + (kb - kb0) * 48;
#pragma unroll
          for (int j = 0; j < 3; ++j) lds128(cp + 16 * j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          uint32_t out[32];
          Lookup<64>::run(w, tbl, out);
          const int sa = it % SA;
          if (it >= SA && !warp_wait(bar.empty_a + 8 * sa, ((it / SA) & 1) ^ 1, true)) { ok = false; break; }
          sm100::tc_fence_after();
          __syncwarp();
          sm100::tmem_st_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + A_COL + sa * 32, out);
          sm100::tmem_wait_st();
          sm100::tc_fence_before();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(bar.dec_done + 8 * sa);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(bar.empty_c + 8 * sc);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t lead_empty = sm100::mapa_shared(bar.acc_empty, 0);
    Slots sl;
    for (int wi = pair; wi < nitems && ok; wi += npairs) {
      const Tile t = tile_at(wi);
      const int slots = a.nseg > 1 ? 2 : t.halves, first_slot = sl.take(slots);
      const int n = GATED ? (t.wt * 2 + (int)rank) * (RW / 2) + 16 * q + (lane & 15)
                          : (t.wt * 2 + (int)rank) * RW + 32 * q + lane;
      for (int h = 0; h < t.halves && ok; ++h) {
        const int slot = first_slot + h;
        if (!warp_wait(bar.acc_full + 8 * slot, sl.used[slot] & 1, true)) { ok = false; break; }
        if (a.nseg > 1 && !warp_wait(bar.acc_full + 8, sl.used[1] & 1, true)) { ok = false; break; }
        sm100::tc_fence_after();
        for (int c = 0; c < t.nh; c += 16) {
          const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + D_COL + slot * NS + c;
          uint32_t v[16];
          sm100::tmem_ld_32x32b_x16(at, v);
          sm100::tmem_wait_ld();
          for (int r = 1; r < a.nseg; ++r) {
            uint32_t u[16];
            sm100::tmem_ld_32x32b_x16(at + r * t.nh, u);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
          }
          // the output row of position c + (lane & 15), -1 for none
          const int p = t.p0 + h * t.nh + c + (lane & 15);
          int yr = -1;
          if (p < t.p1) {
            yr = a.g.y_rows ? __ldcg(a.g.y_rows + p) : p;
            const int xi = a.g.x_rows ? __ldcg(a.g.x_rows + p) : p;
            if ((unsigned)yr >= (unsigned)a.g.Y || xi < 0 || (a.g.x_rows ? xi / a.g.x_div : xi) >= a.g.X) yr = -1;
          }
          if constexpr (GATED) {
            // lanes 0-15 hold g, lanes 16-31 u of the same features: after the exchange the lower half has both
            // for columns 0-7 and the upper half for columns 8-15
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t mine = lane < 16 ? v[i] : v[8 + i], give = lane < 16 ? v[8 + i] : v[i];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 16);
              const float gv = __uint_as_float(lane < 16 ? mine : got), uv = __uint_as_float(lane < 16 ? got : mine);
              const int yi = __shfl_sync(0xffffffffu, yr, (lane < 16 ? 0 : 8) + i);
              if (yi >= 0 && n < a.N) store_out(a.y, a.ydt, (size_t)yi * a.N + n, qld::silu_mul(gv, uv));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int yi = __shfl_sync(0xffffffffu, yr, i);
              if (yi >= 0 && n < a.N) store_out(a.y, a.ydt, (size_t)yi * a.N + n, __uint_as_float(v[i]));
            }
          }
        }
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          sm100::mbar_arrive_cluster(lead_empty + 8 * slot);
          if (a.nseg > 1) sm100::mbar_arrive_cluster(lead_empty + 8);
        }
      }
      sl.done(first_slot, slots);
    }
  }

  if (!ok) atomicExch(&g_grouped_timeout, 1);
  // neither CTA leaves while its peer may still arrive on its barriers or use its shared or tensor memory
  sm100::tc_fence_before();
  sm100::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    sm100::tc_fence_after();
    sm100::tmem_dealloc_pair(tmem, 512);
  }
}

// CTA pairs that can be resident at once on the current device (cached per device and kernel).
template <bool GATED>
int resident_pairs() {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (ql::sm_count() / 2));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes(QL_MAX_GROUPS);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, benq_grouped_kernel<GATED>, &cfg) != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = ql::sm_count() / 2;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

}  // namespace

namespace ql {

ql_status benq_grouped_mma_launch(const uint8_t *codes, const uint16_t *lut, const uint8_t *codes2, const uint16_t *lut2,
                                  const ql_groups &g, const uint16_t *x, void *y, ql_out_dtype ydt, int N, int K,
                                  cudaStream_t s) {
  const char *who = codes2 ? "benq_grouped_gate_up" : "benq_grouped_linear";
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return fail(QL_ERR_CUDA, "%s: cuTensorMapEncodeTiled is unavailable", who);
  const int per = codes2 ? RW / 2 : RW;   // rows of each layer per CTA and tile
  CUtensorMap mx, mc, mc2;
  if (!encode_rows_sw128(enc, &mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, g.X, K, K, g.x_rows ? 1 : X_BOX))
    return fail(QL_ERR_CUDA, "%s: cannot encode the activation tensor map", who);
  auto codes_map = [&](CUtensorMap *m, const uint8_t *c) {
    const cuuint64_t rowbytes = (cuuint64_t)K * 3 / 4;
    const cuuint64_t dims[2] = {rowbytes, (cuuint64_t)g.G * N};
    const cuuint64_t strides[1] = {rowbytes};
    const cuuint32_t box[2] = {C_ROW, (cuuint32_t)per};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(c), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!codes_map(&mc, codes) || !codes_map(&mc2, codes2 ? codes2 : codes))
    return fail(QL_ERR_CUDA, "%s: cannot encode the code tensor map", who);
  Args a{lut, lut2, g, y, (int)ydt, N, K, (N + 2 * per - 1) / (2 * per), NT, K / 64, 1};
  if (ydt == QL_OUT_F32 && K / 64 > SEG_KB) {
    a.seg = std::max(SEG_KB, (K / 64 + MAX_SEG - 1) / MAX_SEG);
    a.nseg = (K / 64 + a.seg - 1) / a.seg;
    a.nt_max = std::min(NS, NT / a.nseg / 16 * 16);   // every run's accumulator fits beside the others
  }
  const size_t smem = smem_bytes(g.G);
  // the most tiles that the counts could make (each group may end inside a tile)
  const int64_t items = ((int64_t)std::min(g.G, g.M) + g.M / a.nt_max) * a.ntl;
  auto go = [&](auto gated) -> ql_status {
    constexpr bool GATED = decltype(gated)::value;
    if (set_max_smem(benq_grouped_kernel<GATED>, (int)smem_bytes(QL_MAX_GROUPS)) != cudaSuccess)
      return fail(QL_ERR_CUDA, "%s: cannot reserve shared memory", who);
    const int grid = 2 * (int)std::min<int64_t>(items, resident_pairs<GATED>());
    launch(benq_grouped_kernel<GATED>, grid, THREADS, smem, s, mx, mc, mc2, a);
    return launch_status(who);
  };
  return codes2 ? go(std::true_type{}) : go(std::false_type{});
}

ql_status benq_grouped_read_timeout(int *flag) {
  int zero = 0;
  if (cudaMemcpyFromSymbol(flag, g_grouped_timeout, sizeof(int)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_grouped_timeout, &zero, sizeof(int)) != cudaSuccess)
    return fail(QL_ERR_CUDA, "ql_check: cannot read the device timeout flag");
  return QL_OK;
}

}  // namespace ql
