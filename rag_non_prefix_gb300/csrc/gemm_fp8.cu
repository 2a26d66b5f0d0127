// Product of two e4m3 matrices with a scale per group of 128 channels of a row of A (tokens) and
// per 128 x 128 block of B (weights):
//   acc[m][n] = sum over groups g of  sa[g][m] * sb[n / 128][g] * sum_{k in g} A[m][k] B[n][k]
//
// The tensor core sums the products of one group (four tcgen05.mma kind::f8f6f4 of 32 channels)
// into tensor memory; eight warps then read that sum, multiply it by the group's two scales and
// add it to fp32 registers, while the tensor core works on the next group in the other half of
// tensor memory.  Weights sit on the tensor core's rows: a CTA pair (one CTA per SM) computes 256
// weight rows x bt tokens, bt a multiple of 16 up to 256, so that a ragged number of tokens is
// padded to 16 and not to 128, and few tokens stream the weights with little else.
//   warp 0: TMA producer of codes   warp 1: tensor-memory owner, in even CTAs the MMA issuer
//   warp 2: TMA producer of token scales   warps 4-11: scaling, sums and epilogue
// The eight warps read tensor memory as 16 lanes x 256 bits (a thread gets 2 tokens of rows i / 4
// and i / 4 + 8), so that a thread needs the scales of an eighth of the tokens only: reading 32
// lanes x 1 token it would need all of them, which costs as much shared-memory bandwidth as the
// MMAs' operands.  The sums run as packed fp32 (fma.rn.f32x2, two tokens).
//
// Two ways to the output:
//   - registers (many tokens): each warp stages 16 tokens x 32 features and stores them by TMA;
//     SwiGLU's weight rows are loaded as 8 gate, 8 up, 8 gate, ... rows, so that a thread holds
//     gate and up of the same feature, and the group's largest magnitude (128 features over both
//     CTAs) is formed by a maximum in the shared memory of both.
//   - shared memory (few tokens): a cluster of S pairs splits the channels; every CTA leaves its
//     fp32 sums in its shared memory, and each CTA of the cluster finishes 1 / (2 S) of the tokens
//     for all 256 rows, adding the S parts in a fixed order.
// Every wait is bounded: a warp that gives up records ST_WAIT_TIMEOUT and runs on without waiting
// or storing, so that the barriers it shares are still met; the cluster meets at its closing
// barrier before any CTA frees its tensor memory or leaves.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "common.cuh"
#include "internal.h"

namespace cb {

namespace f8 {

constexpr int THREADS = 384;
constexpr int ROWS = 128;                  // weight rows per CTA
constexpr int A_BYTES = ROWS * 128;        // 16 KiB: 128 weight rows x one group of channels
constexpr int MAX_STAGES = 12;
constexpr int SC_SLOTS = 8;                // token scales of a group: slots of 256 floats
constexpr int OFF_SCALES = 1024;           // after the barriers
constexpr int OFF_AMAX = OFF_SCALES + SC_SLOTS * 1024;  // SwiGLU: 2 x 256 maxima, then 256 quotients
constexpr int OFF_RING = OFF_AMAX + 3 * 1024;
constexpr int SMEM_ALLOC = 232448;         // the per-block maximum (227 KiB), 1 KiB of it aligns the base
constexpr int SMEM_USE = SMEM_ALLOC - 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr int PART_PITCH = ROWS + 4;       // floats per token of a CTA's partial sums

// Accumulators in tensor memory: as many groups' sums as fit may wait to be read.
__host__ __device__ constexpr int n_acc(int bt) { return bt <= 64 ? 8 : bt <= 128 ? 4 : 2; }

struct Params {
  Fp8Gemm g;
  int width;        // output features
  int bt;           // tokens per tile
  int tok_tiles, units;
  int split;        // pairs per cluster, each taking a part of the groups
  int groups;       // ceil(K / 128)
  int stages, stage_bytes;
  int out_off;      // staging (registers) or partial sums (shared memory), after the ring
  int interleaved;  // SwiGLU rows through one map of both matrices (else two maps, 8 rows at a time)
  int up_first;     // g.b is the up and g.b2 the gate matrix
  int add_in_place;
  int ragged;       // output rows end inside 16 bytes: a TMA store would write up to the 16th
};

// Bytes of the output area after the ring.
__host__ __device__ constexpr int out_bytes(int epilogue, int bt, bool via_smem) {
  return via_smem ? (bt * PART_PITCH * 4 + 1023) / 1024 * 1024
                  : epilogue == CB_FP8_SWIGLU_FP8 ? bt * 64 : epilogue == CB_FP8_STORE_BF16 ? 8 * 2 * 1024 : 8 * 2 * 2048;
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D, both K-major, M = 256, N = n.
__device__ __forceinline__ uint32_t idesc_pair(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
}
// D (128 lanes in each CTA of the pair) (+)= A . B^T over 32 channels; issued by the even CTA.
__device__ __forceinline__ void mma_f8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 lanes x 8 N8 fp32 columns: r[4 j .. 4 j + 3] = (row i / 4, columns 8 j + 2 (i % 4), + 1), then row i / 4 + 8.
template <int N8> __device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, uint32_t* r);
template <> __device__ __forceinline__ void tmem_ld16x256<1>(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
template <> __device__ __forceinline__ void tmem_ld16x256<2>(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
template <> __device__ __forceinline__ void tmem_ld16x256<4>(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Waits for this thread's tensor-memory reads; what was read into r may be used after it only.
template <int N> __device__ __forceinline__ void tmem_wait_ld_of(uint32_t* r, uint32_t* q) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]), "+r"(q[i]));
}

// ----------------------------------------------------------------------------- packed fp32 pairs
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
  return r;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ----------------------------------------------------------------------------- cluster exchange
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void red_max_cluster(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// mbar_wait_bounded with acquire at cluster scope (other CTAs' shared memory is read after it)
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (it == 0) t0 = global_ns();
    if ((it & 255u) == 255u && (*abort || global_ns() - t0 > 2000000000ull)) return false;
  }
}
// Arrival on another CTA's barrier that orders no memory access: what it announces is that tensor
// memory was read (tcgen05.wait::ld and the tcgen05 fence order that).  With release at cluster
// scope the same arrival took ~1200 cycles.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Whether the phase has completed, without waiting: polled ahead of the work that hides its latency.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ float silu(float x) { return x / (1.0f + __expf(-x)); }

struct Bars {
  uint64_t full[MAX_STAGES];      // codes of a stage have landed (even CTAs)
  uint64_t done[MAX_STAGES];      // its MMAs are done: the stage is free and the group's sums are readable
  uint64_t acc_empty[8];          // both CTAs' warps have read an accumulator (even CTAs)
  uint64_t sc_full[SC_SLOTS], sc_empty[SC_SLOTS];
  uint64_t part_full, part_free;  // shared-memory output: the cluster's parts are written / read
  uint64_t amax_full[2];          // SwiGLU from registers: the maxima of a tile are complete
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(Bars) <= OFF_SCALES, "barriers overrun their area");

// HB: tokens per warpgroup (half a tile).  SWIGLU: B and B2 interleaved by 8 rows.  VIA_SMEM: the
// output goes through shared memory (and the channels may be split over the cluster's pairs).
template <int HB, bool SWIGLU, bool VIA_SMEM>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmS,
                    const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr int BT = 2 * HB;
  // tokens per tensor-memory read: an even number of reads, so that two buffers alternate across groups
  constexpr int CH = HB % 64 == 0 ? 32 : HB % 32 == 0 ? 16 : 8;
  constexpr int NCH = HB / CH;
  constexpr uint32_t B_BYTES = HB * 128;
  constexpr uint32_t NACC = n_acc(BT), ACC_STRIDE = TMEM_COLS / NACC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem);
  float* sc = reinterpret_cast<float*>(smem + OFF_SCALES);
  uint32_t* amax = reinterpret_cast<uint32_t*>(smem + OFF_AMAX);  // [2][256]
  float* quot = reinterpret_cast<float*>(smem + OFF_AMAX + 2048);  // [256]
  uint8_t* ring = smem + OFF_RING;
  uint8_t* out = smem + p.out_off;
  volatile int* abort = &bars.abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(rank >> 1), h = static_cast<int>(rank & 1u);
  const uint32_t lead = rank & ~1u;
  const int cid = static_cast<int>(cluster_id_x()), NC = static_cast<int>(n_clusters_x());
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  // this pair's groups of channels
  const int g0 = static_cast<int>(static_cast<long long>(p.groups) * pair / p.split);
  const int g1 = static_cast<int>(static_cast<long long>(p.groups) * (pair + 1) / p.split);

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.done[s], 1);
    }
    for (int b = 0; b < 8; ++b) mbar_init(&bars.acc_empty[b], 16);  // eight warps of both CTAs
    for (int b = 0; b < 2; ++b) mbar_init(&bars.amax_full[b], 16);
    for (int s = 0; s < SC_SLOTS; ++s) {
      mbar_init(&bars.sc_full[s], 1);
      mbar_init(&bars.sc_empty[s], 8);
    }
    mbar_init(&bars.part_full, 16 * p.split);
    mbar_init(&bars.part_free, 16 * p.split);
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 3 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmS);
    if (!VIA_SMEM) prefetch_tmap(&tmC);
  }
  if (SWIGLU && !VIA_SMEM && warp >= 4)
    for (int i = threadIdx.x - 128; i < 512; i += 256) amax[i] = __float_as_uint(FP8_AMAX_MIN);
  if (warp == 1) {
    tmem_alloc_pair(&bars.tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers and maxima are initialised before another CTA reaches them
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  pdl_wait();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------- TMA producer of codes
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int u = cid; ok && u < p.units; u += NC) {
        const int wt = u / p.tok_tiles, tt = u - wt * p.tok_tiles;
        const int trow = tt * BT + h * HB;
        for (int g = g0; g < g1; ++g) {
          if (!mbar_wait_bounded(&bars.done[s], ph ^ 1u, abort)) {
            ok = false;
            break;
          }
          uint8_t* a = ring + s * static_cast<uint32_t>(p.stage_bytes);
          const uint32_t bar = mapa_shared(smem_u32(&bars.full[s]), lead);
          if (h == 0) mbar_arrive_expect_tx(&bars.full[s], 2u * (A_BYTES + B_BYTES));
          if (!SWIGLU) {
            tma_load_2d_pair(a, &tmW, bar, g * 128, wt * 256 + h * ROWS);
          } else if (p.interleaved) {
            tma_load_4d_pair(a, &tmW, bar, g * 128, 0, 0, (wt * 128 + h * 64) / 8);
          } else {
            for (int i = 0; i < 8; ++i) {
              tma_load_2d_pair(a + i * 2048, &tmW, bar, g * 128, wt * 128 + h * 64 + i * 8);
              tma_load_2d_pair(a + i * 2048 + 1024, &tmW2, bar, g * 128, wt * 128 + h * 64 + i * 8);
            }
          }
          tma_load_2d_pair(a + A_BYTES, &tmX, bar, g * 128, trow);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort = 1;
        set_status(p.g.status, ST_WAIT_TIMEOUT);
      }
    } else if (warp == 1 && lane == 0 && h == 0) {
      // ---------------------------------------------------------------- MMA issuer (even CTAs)
      const uint32_t idesc = idesc_pair(BT);
      const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * pair));
      const uint32_t ring_u32 = smem_u32(ring);
      uint32_t s = 0, ph = 0, sa = ring_u32, b = 0, aph = 1;
      bool ok = true, full_ready = false, acc_ready = false;  // polled during the previous group's MMAs
      for (int u = cid; ok && u < p.units; u += NC) {
        for (int g = g0; g < g1; ++g) {
          if ((!acc_ready && !mbar_wait_bounded(&bars.acc_empty[b], aph, abort)) ||
              (!full_ready && !mbar_wait_bounded(&bars.full[s], ph, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t* done = &bars.done[s];
          const uint64_t da = sw128_desc(sa), db = sw128_desc(sa + A_BYTES);
          const uint32_t tacc = tmem + b * ACC_STRIDE;
          sa += static_cast<uint32_t>(p.stage_bytes);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
            sa = ring_u32;
          }
          if (++b == NACC) {
            b = 0;
            aph ^= 1u;
          }
          full_ready = mbar_test(&bars.full[s], ph);
          acc_ready = mbar_test(&bars.acc_empty[b], aph);
          mma_f8_pair(tacc, da, db, idesc, 0u);
          mma_f8_pair(tacc, da + 2, db + 2, idesc, 1u);  // + 32 bytes along K (encoded >> 4)
          mma_f8_pair(tacc, da + 4, db + 4, idesc, 1u);
          mma_f8_pair(tacc, da + 6, db + 6, idesc, 1u);
          tc_commit_pair_mc(done, pair_mask);
        }
      }
      if (!ok) {
        *abort = 1;
        set_status(p.g.status, ST_WAIT_TIMEOUT);
      }
      // no MMA may still be running when the cluster meets at its closing barrier
      tc_commit_pair_mc(&bars.drain, static_cast<uint16_t>(1u << rank));
      mbar_wait_bounded(&bars.drain, 0u, nullptr);
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------------- TMA producer of token scales
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int u = cid; ok && u < p.units; u += NC) {
        const int tt = u % p.tok_tiles;
        for (int g = g0; g < g1; ++g) {
          if (!mbar_wait_bounded(&bars.sc_empty[s], ph ^ 1u, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars.sc_full[s], BT * 4);
          tma_load_2d(sc + s * 256, &tmS, &bars.sc_full[s], tt * BT, g);
          if (++s == SC_SLOTS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        *abort = 1;
        set_status(p.g.status, ST_WAIT_TIMEOUT);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ scaling, sums, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3, w = (warp >> 2) - 1;  // tensor-memory lanes 32 quarter .., tokens w HB ..
    const int et = threadIdx.x - 128;                    // 0 .. 255
    const int wt_t = threadIdx.x & 127;                  // thread of its warpgroup
    const int ri = lane >> 2, ci = (lane & 3) * 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t acc_empty_lead = mapa_shared(smem_u32(bars.acc_empty), lead);
    uint32_t ss = 0, sph = 0, st = 0, ph = 0, b = 0;
    bool ok = true;
    auto give_up = [&]() {
      ok = false;
      *abort = 1;
      if (lane == 0) set_status(p.g.status, ST_WAIT_TIMEOUT);
    };
    int nth = 0;  // tiles done
    for (int u = cid; u < p.units; u += NC, ++nth) {
      const int wt = u / p.tok_tiles, tt = u - wt * p.tok_tiles;
      const int t0 = tt * BT;
      // the weight block's scales of this CTA's rows (rows past the last one are zeros: any block will do)
      const int blk = SWIGLU ? wt : min(wt * 2 + h, (p.width - 1) >> 7);
      const float* sb0 = p.g.b_scale + static_cast<long long>(blk) * p.g.ld_bs;
      const float* sb1 = SWIGLU ? p.g.b2_scale + static_cast<long long>(blk) * p.g.ld_b2s : sb0;
      uint64_t acc[HB / 8][4];  // per 8 tokens: rows i/4, + 8, + 16, + 24 of the quarter, 2 tokens each
#pragma unroll
      for (int j = 0; j < HB / 8; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0;
      float nb0 = __ldg(sb0 + g0), nb1 = SWIGLU ? __ldg(sb1 + g0) : 0.f;
      // Two register buffers: the next read of tensor memory, which may be the next group's first,
      // runs under the sums of the current one.
      uint32_t lo[2][CH / 2], hi[2][CH / 2];
      bool sc_ready = false, acc_ready = false;
      // the group's sums and scales are there: start its first read
      auto begin = [&]() {
        if (ok && !((sc_ready || mbar_wait_bounded(&bars.sc_full[ss], sph, abort)) &&
                    (acc_ready || mbar_wait_bounded(&bars.done[st], ph, abort))))
          give_up();
        __syncwarp();
        tc_fence_after();
        const uint32_t tacc = tmem + b * ACC_STRIDE + lane_base + static_cast<uint32_t>(w * HB);
        tmem_ld16x256<CH / 8>(tacc, lo[0]);
        tmem_ld16x256<CH / 8>(tacc + (16u << 16), hi[0]);
      };
      begin();
#pragma unroll 1
      for (int g = g0; g < g1; ++g) {
        const uint64_t s0 = pack2(nb0, nb0), s1 = SWIGLU ? pack2(nb1, nb1) : s0;
        if (g + 1 < g1) {
          nb0 = __ldg(sb0 + g + 1);
          if (SWIGLU) nb1 = __ldg(sb1 + g + 1);
        }
        const uint32_t tacc = tmem + b * ACC_STRIDE + lane_base + static_cast<uint32_t>(w * HB);
        const float* sv = sc + ss * 256 + w * HB + ci;
        const uint32_t ss_now = ss;
        auto sums = [&](int c) {
          const int i = c & 1;
#pragma unroll
          for (int j = 0; j < CH / 8; ++j) {
            const int jj = c * (CH / 8) + j;
            const uint64_t sa = *reinterpret_cast<const uint64_t*>(sv + jj * 8);
            const uint64_t m0 = mul2(sa, s0), m1 = SWIGLU ? mul2(sa, s1) : m0;
            acc[jj][0] = fma2(pack2u(lo[i][4 * j], lo[i][4 * j + 1]), m0, acc[jj][0]);
            acc[jj][1] = fma2(pack2u(lo[i][4 * j + 2], lo[i][4 * j + 3]), m1, acc[jj][1]);
            acc[jj][2] = fma2(pack2u(hi[i][4 * j], hi[i][4 * j + 1]), m0, acc[jj][2]);
            acc[jj][3] = fma2(pack2u(hi[i][4 * j + 2], hi[i][4 * j + 3]), m1, acc[jj][3]);
          }
        };
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          tmem_wait_ld_of<CH / 2>(lo[c & 1], hi[c & 1]);
          if (c + 1 < NCH) {
            tmem_ld16x256<CH / 8>(tacc + (c + 1) * CH, lo[(c + 1) & 1]);
            tmem_ld16x256<CH / 8>(tacc + (c + 1) * CH + (16u << 16), hi[(c + 1) & 1]);
            sums(c);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_lead + b * 8);
            if (++b == NACC) b = 0;
            if (++st == stages) {
              st = 0;
              ph ^= 1u;
            }
            if (++ss == SC_SLOTS) {
              ss = 0;
              sph ^= 1u;
            }
            if (NCH % 2) sums(c);
            if (g + 1 < g1) {
              sc_ready = mbar_test(&bars.sc_full[ss], sph);
              acc_ready = mbar_test(&bars.done[st], ph);
              begin();
            }
            if (NCH % 2 == 0) sums(c);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sc_empty[ss_now]);
      }

      if constexpr (VIA_SMEM) {
        // ---------------------------------------------------------------- through shared memory
        float* part = reinterpret_cast<float*>(out);  // [BT][PART_PITCH]
        const int CS = 2 * p.split;
        const uint32_t parity = nth & 1;
        // the parts of the previous tile have been read by the whole cluster
        if (ok && !mbar_wait_cluster(&bars.part_free, parity ^ 1u, abort)) give_up();
        ok = __all_sync(0xffffffffu, ok);
#pragma unroll
        for (int j = 0; j < HB / 8; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 v = unpack2(acc[j][r]);
            float* d = part + (w * HB + j * 8 + ci) * PART_PITCH + quarter * 32 + r * 8 + ri;
            d[0] = v.x;
            d[PART_PITCH] = v.y;
          }
        __syncwarp();
        if (lane < CS) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.part_full), lane));
        if (ok && !mbar_wait_cluster(&bars.part_full, parity, abort)) give_up();
        ok = __all_sync(0xffffffffu, ok);
        // this CTA finishes tokens rank * per .. of the tile
        const int per = (BT + CS - 1) / CS;
        const int j0 = static_cast<int>(rank) * per, j1 = min(min(BT, j0 + per), p.g.M - t0);
        const uint32_t part_u32 = smem_u32(part);
        if constexpr (!SWIGLU) {
          const int f = wt * 256 + et;
          const uint32_t hh = static_cast<uint32_t>(et >> 7);
          for (int j = j0; j < j1; ++j) {
            float v = 0.f;
            for (int s = 0; s < p.split; ++s)
              v += ld_cluster_f32(mapa_shared(part_u32 + (j * PART_PITCH + (et & 127)) * 4, 2 * s + hh));
            const long long o = static_cast<long long>(t0 + j) * p.g.ldc + f;
            if (f < p.width && ok) {
              if (p.g.epilogue == CB_FP8_STORE_BF16)
                static_cast<bf16*>(p.g.c)[o] = __float2bfloat16_rn(v);
              else
                static_cast<float*>(p.g.c)[o] = p.g.epilogue == CB_FP8_ADD_F32 ? p.g.addend[o] + v : v;
            }
          }
        } else {
          // a warpgroup per token, thread x takes feature x of the tile's 128
          const uint32_t hh = static_cast<uint32_t>(wt_t >> 6);
          const int fl = wt_t & 63, row = (fl >> 3) * 16 + (fl & 7);  // its gate row; the up row is 8 further
          const int f = wt * 128 + wt_t;
          for (int j = j0; j < j1; j += 2) {
            const int jj = min(j + w, j1 - 1);  // an odd last token is finished by both warpgroups alike
            float gate = 0.f, up = 0.f;
            for (int s = 0; s < p.split; ++s) {
              const uint32_t a = mapa_shared(part_u32 + (jj * PART_PITCH + row) * 4, 2 * s + hh);
              gate += ld_cluster_f32(a);
              up += ld_cluster_f32(a + 32);
            }
            const float y = p.up_first ? silu(up) * gate : silu(gate) * up;
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(y) & 0x7fffffffu);
            if (lane == 0) amax[w * 4 + quarter] = m;
            named_bar(1 + w, 128);
            uint32_t a = __float_as_uint(FP8_AMAX_MIN);
#pragma unroll
            for (int q = 0; q < 4; ++q) a = max(a, amax[w * 4 + q]);
            named_bar(1 + w, 128);
            const float am = __uint_as_float(a);
            if (ok && f < p.width) {
              static_cast<uint8_t*>(p.g.c)[static_cast<long long>(t0 + jj) * p.g.ldc + f] =
                  __nv_cvt_float_to_fp8(y * (FP8_MAX / am), __NV_SATFINITE, __NV_E4M3);
              if (wt_t == 0) p.g.c_scale[static_cast<long long>(wt) * p.g.ld_cs + t0 + jj] = am / FP8_MAX;
            }
          }
        }
        __syncwarp();
        if (lane < CS) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.part_free), lane));
      } else if constexpr (SWIGLU) {
        // ---------------------------------------------------------------- SwiGLU from registers
        const uint32_t par = nth & 1;
        uint32_t* am = amax + par * 256;
        // y over the gate's registers: acc[j][0] rows i/4 and acc[j][2] rows i/4 of the upper 16
        uint32_t m[HB / 4];
#pragma unroll
        for (int j = 0; j < HB / 8; ++j) {
          const bool sw = p.up_first;
          const float2 ga = unpack2(sw ? acc[j][1] : acc[j][0]), ua = unpack2(sw ? acc[j][0] : acc[j][1]);
          const float2 gb = unpack2(sw ? acc[j][3] : acc[j][2]), ub = unpack2(sw ? acc[j][2] : acc[j][3]);
          const float2 ya = make_float2(silu(ga.x) * ua.x, silu(ga.y) * ua.y);
          const float2 yb = make_float2(silu(gb.x) * ub.x, silu(gb.y) * ub.y);
          acc[j][0] = pack2(ya.x, ya.y);
          acc[j][2] = pack2(yb.x, yb.y);
          m[2 * j] = max(__float_as_uint(ya.x) & 0x7fffffffu, __float_as_uint(yb.x) & 0x7fffffffu);
          m[2 * j + 1] = max(__float_as_uint(ya.y) & 0x7fffffffu, __float_as_uint(yb.y) & 0x7fffffffu);
        }
        const uint32_t am_own = smem_u32(am), am_peer = mapa_shared(am_own, rank ^ 1u);
#pragma unroll
        for (int i = 0; i < HB / 4; ++i) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
          // token column of m[i]: 8 (i / 2) + ci + i % 2; the eight lanes that share it take turns
          if (ri == (i & 7)) {
            const uint32_t off = static_cast<uint32_t>(w * HB + (i >> 1) * 8 + ci + (i & 1)) * 4;
            red_max_cluster(mapa_shared(am_own, rank) + off, m[i]);
            red_max_cluster(am_peer + off, m[i]);
          }
        }
        __syncwarp();
        if (lane < 2) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.amax_full[par]), lead + lane));
        if (ok && !mbar_wait_cluster(&bars.amax_full[par], (nth >> 1) & 1, abort)) give_up();
        ok = __all_sync(0xffffffffu, ok);
        if (wt_t < HB) {
          const int col = w * HB + wt_t;
          const float a = __uint_as_float(am[col]);
          am[col] = __float_as_uint(FP8_AMAX_MIN);
          quot[col] = FP8_MAX / a;
          if (h == 0 && ok && t0 + col < p.g.M) p.g.c_scale[static_cast<long long>(wt) * p.g.ld_cs + t0 + col] = a / FP8_MAX;
        }
        uint8_t* slab = out + w * HB * 64;  // [HB tokens][64 features], 64-byte swizzle
        if (wt_t == 0) bulk_wait_read_all();
        named_bar(1 + w, 128);
#pragma unroll
        for (int j = 0; j < HB / 8; ++j) {
          const float2 q = *reinterpret_cast<const float2*>(quot + w * HB + j * 8 + ci);
          const int tok = j * 8 + ci;  // even: the pair tok, tok + 1 shares its swizzle
          uint8_t* d = slab + tok * 64 + ((quarter ^ ((tok >> 1) & 3)) << 4) + ri;
          const float2 ya = unpack2(acc[j][0]), yb = unpack2(acc[j][2]);
          const uint32_t ca = __nv_cvt_float2_to_fp8x2(make_float2(ya.x * q.x, ya.y * q.y), __NV_SATFINITE, __NV_E4M3);
          const uint32_t cb = __nv_cvt_float2_to_fp8x2(make_float2(yb.x * q.x, yb.y * q.y), __NV_SATFINITE, __NV_E4M3);
          d[0] = static_cast<uint8_t>(ca);
          d[64] = static_cast<uint8_t>(ca >> 8);
          d[8] = static_cast<uint8_t>(cb);
          d[72] = static_cast<uint8_t>(cb >> 8);
        }
        fence_proxy_async_smem();
        named_bar(1 + w, 128);
        if (wt_t == 0 && ok && t0 + w * HB < p.g.M) {
          tma_store_2d(&tmC, slab, wt * 128 + h * 64, t0 + w * HB);
          bulk_commit();
        }
      } else {
        // ---------------------------------------------------------------- fp32 or bf16 from registers
        const bool to_bf16 = p.g.epilogue == CB_FP8_STORE_BF16;
        const bool add = p.g.epilogue == CB_FP8_ADD_F32;
        const int slab_bytes = to_bf16 ? 1024 : 2048;  // 16 tokens x 32 features
        uint8_t* mine = out + (warp - 4) * 2 * slab_bytes;
        const int f0 = wt * 256 + h * ROWS + quarter * 32;
#pragma unroll
        for (int jp = 0; jp < HB / 16; ++jp) {
          const int tok0 = t0 + w * HB + jp * 16;
          if (tok0 < p.g.M && f0 < p.width) {  // (uniform in the warp)
            uint8_t* slab = mine + (jp & 1) * slab_bytes;
            const bool tail = p.ragged && f0 + 32 > p.width;  // stored element by element
            if (add && (tail || !p.add_in_place)) {
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  float2 v = unpack2(acc[jp * 2 + jj][r]);
                  const int tok = tok0 + jj * 8 + ci, f = f0 + r * 8 + ri;
                  const float* a = p.g.addend + static_cast<long long>(tok) * p.g.ldc + f;
                  if (f < p.width && tok < p.g.M) v.x = a[0] + v.x;
                  if (f < p.width && tok + 1 < p.g.M) v.y = a[p.g.ldc] + v.y;
                  acc[jp * 2 + jj][r] = pack2(v.x, v.y);
                }
            }
            if (tail) {
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float2 v = unpack2(acc[jp * 2 + jj][r]);
                  const int tok = tok0 + jj * 8 + ci, f = f0 + r * 8 + ri;
                  const long long o = static_cast<long long>(tok) * p.g.ldc + f;
                  if (!ok || f >= p.width) continue;
                  if (to_bf16) {
                    bf16* c = static_cast<bf16*>(p.g.c) + o;
                    if (tok < p.g.M) c[0] = __float2bfloat16_rn(v.x);
                    if (tok + 1 < p.g.M) c[p.g.ldc] = __float2bfloat16_rn(v.y);
                  } else {
                    float* c = static_cast<float*>(p.g.c) + o;
                    if (tok < p.g.M) c[0] = v.x;
                    if (tok + 1 < p.g.M) c[p.g.ldc] = v.y;
                  }
                }
              continue;
            }
            if (lane == 0) bulk_wait_read_all_but_1();
            __syncwarp();
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const int j = jp * 2 + jj;
              if (to_bf16) {
                uint32_t v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float2 x = unpack2(acc[j][r]);
                  v[r] = pack_bf16x2(x.x, x.y);
                }
                // matrix r (features 8 r ..) is stored transposed: lane 8 r + t points at token t's 16 bytes
                const int tok = jj * 8 + (lane & 7);
                stmatrix_x4_trans(smem_u32(slab) + tok * 64 + (((lane >> 3) ^ ((tok >> 1) & 3)) << 4), v[0], v[1], v[2],
                                  v[3]);
              } else {
                const int tok = jj * 8 + ci;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  const float2 x = unpack2(acc[j][r]);
                  const int fb = (r * 8 + ri) * 4;
                  *reinterpret_cast<float*>(slab + tok * 128 + (fb ^ ((tok & 7) << 4))) = x.x;
                  *reinterpret_cast<float*>(slab + (tok + 1) * 128 + (fb ^ (((tok + 1) & 7) << 4))) = x.y;
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
              if (add && p.add_in_place)
                tma_reduce_add_2d(&tmC, slab, f0, tok0);
              else
                tma_store_2d(&tmC, slab, f0, tok0);
              bulk_commit();
            }
          }
        }
      }
    }
    bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  // No CTA leaves, or frees the pair's tensor memory, while another may still reach its barriers or
  // shared memory: every issuer has drained its MMAs, every producer and epilogue has finished.
  cluster_sync_all();
  // After a timeout anywhere in the cluster, copies issued for stages that were never consumed may
  // still be in flight: give them time to land before the memory is released.
  if (bars.abort || (p.g.status != nullptr && (*reinterpret_cast<volatile int32_t*>(p.g.status) & ST_WAIT_TIMEOUT))) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 200000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

}  // namespace f8

// ============================================================================= planner + launcher
namespace {

using namespace f8;

typedef void (*Kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                       const Params);

template <int HB, bool VIA_SMEM> Kernel pick(bool swiglu) {
  return swiglu ? gemm_fp8_kernel<HB, true, VIA_SMEM> : gemm_fp8_kernel<HB, false, VIA_SMEM>;
}
Kernel kernel_of(int bt, bool swiglu, bool via_smem) {
  if (via_smem) switch (bt) {
      case 16: return pick<8, true>(swiglu);
      case 32: return pick<16, true>(swiglu);
      case 64: return pick<32, true>(swiglu);
      case 128: return pick<64, true>(swiglu);
      default: return nullptr;
    }
  switch (bt) {
    case 128: return pick<64, false>(swiglu);
    case 192: return pick<96, false>(swiglu);
    case 256: return pick<128, false>(swiglu);
    default: return nullptr;
  }
}

// Clusters of `cs` CTAs that are resident at once (one CTA per SM), per device.
int resident_clusters(int cs) {
  static std::atomic<int> cache[4][64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int ci = cs == 2 ? 0 : cs == 4 ? 1 : 2;
  if (dev >= 0 && dev < 64) {
    const int v = cache[ci][dev].load();
    if (v > 0) return v;
  }
  const void* fn = reinterpret_cast<const void*>(kernel_of(16, false, true));
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC) != cudaSuccess) return 0;
  cudaLaunchConfig_t q = {};
  q.gridDim = dim3(cs * 64);
  q.blockDim = dim3(THREADS);
  q.dynamicSmemBytes = SMEM_ALLOC;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  q.attrs = attr;
  q.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &q) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) cache[ci][dev].store(n);
  return n;
}

// cb_gemm_scaled_set_plan: tokens per tile (0: the model decides) and pairs per cluster (0: output
// from registers).
std::atomic<int> g_plan{0};

struct Plan {
  int bt, split, clusters, stages, out_off;
  bool via_smem;
};

Plan plan(const Fp8Gemm& g) {
  const bool swiglu = g.epilogue == CB_FP8_SWIGLU_FP8;
  const int width = swiglu ? g.N / 2 : g.N, groups = (g.K + 127) / 128;
  const int w_tiles = swiglu ? (width + 127) / 128 : (width + 255) / 256;
  Plan best{};
  double best_us = 1e30;
  const int forced = g_plan.load();
  auto consider = [&](int bt, int split, bool via_smem) {
    if (forced && forced != bt * 8 + (via_smem ? split : 0)) return;
    split = std::min(split, groups);
    if (split == 3) split = 2;
    const int clusters = resident_clusters(2 * split);
    if (clusters <= 0) return;
    const long long tiles = (g.M + bt - 1) / bt, units = tiles * w_tiles;
    const double waves = static_cast<double>((units + clusters - 1) / clusters);
    const double kb = std::max(2.0 * bt + 40.0, 500.0);
    const double epi = via_smem ? 1500.0 + 40.0 * bt / split : swiglu ? 16.0 * bt : 12.0 * bt;
    const double us = waves * ((groups + split - 1) / split * kb + epi) / 1800.0;
    if (us < best_us) {
      const int room = SMEM_USE - OFF_RING - out_bytes(g.epilogue, bt, via_smem);
      best_us = us;
      // (a stage's barrier is read until its accumulator is: at least n_acc(bt) stages, which all have)
      best = Plan{bt, split, clusters, std::min(MAX_STAGES, room / (A_BYTES + bt * 64)), 0, via_smem};
      best.out_off = OFF_RING + best.stages * (A_BYTES + bt * 64);
    }
  };
  for (int bt : {16, 32, 64, 128})
    for (int split : {1, 2, 4}) consider(bt, split, true);
  for (int bt : {128, 192, 256}) consider(bt, 1, false);
  return best;
}

// Gate and up rows through one map: dims {K, 8 rows, first / second matrix, rows / 8}, the step
// between the matrices being their distance in memory (g.b is the lower one).
bool encode_interleaved(CUtensorMap* map, const Fp8Gemm& g, int width) {
  if (g.ldb != g.ldb2 || g.b2 == g.b) return false;
  const uint64_t step = static_cast<uint64_t>(g.b2 - g.b);
  if (step >= (1ull << 40) || step % 16) return false;
  const uint64_t dims[4] = {static_cast<uint64_t>(g.K), 8, 2, static_cast<uint64_t>(width / 8)};
  const uint64_t strides[3] = {static_cast<uint64_t>(g.ldb), step, static_cast<uint64_t>(g.ldb) * 8};
  const uint32_t box[4] = {128, 8, 2, 8};
  return encode_tmap_nd(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, g.b, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool gemm_fp8_set_plan(int tokens, int split) {
  if (tokens == 0 && split == 0) {
    g_plan.store(0);
    return true;
  }
  if (split != 0 && split != 1 && split != 2 && split != 4) return false;
  if (!kernel_of(tokens, false, split != 0)) return false;
  g_plan.store(tokens * 8 + split);
  return true;
}

cudaError_t launch_gemm_fp8(const Fp8Gemm& call, cudaStream_t s) {
  Fp8Gemm g = call;
  if (g.M <= 0) return cudaSuccess;
  const bool up_first = g.epilogue == CB_FP8_SWIGLU_FP8 && g.b2 < g.b;
  if (up_first) {
    std::swap(g.b, g.b2);
    std::swap(g.ldb, g.ldb2);
    std::swap(g.b_scale, g.b2_scale);
    std::swap(g.ld_bs, g.ld_b2s);
  }
  const bool swiglu = g.epilogue == CB_FP8_SWIGLU_FP8, to_bf16 = g.epilogue == CB_FP8_STORE_BF16;
  const Plan pl = plan(g);
  if (pl.bt == 0 || pl.stages < n_acc(pl.bt)) return cudaErrorInvalidConfiguration;
  Params p{};
  p.g = g;
  p.width = swiglu ? g.N / 2 : g.N;
  p.bt = pl.bt;
  p.tok_tiles = (g.M + pl.bt - 1) / pl.bt;
  p.units = p.tok_tiles * (swiglu ? (p.width + 127) / 128 : (p.width + 255) / 256);
  p.split = pl.split;
  p.groups = (g.K + 127) / 128;
  p.stages = pl.stages;
  p.stage_bytes = A_BYTES + pl.bt * 64;
  p.out_off = pl.out_off;
  p.add_in_place = g.addend == g.c;
  p.up_first = up_first;
  p.ragged = !swiglu && p.width * (to_bf16 ? 2 : 4) % 16 != 0;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, F32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap mx, mw, mw2, ms, mc;
  bool ok = encode_tmap(&mx, U8, g.a, g.K, g.M, g.lda, 128, pl.bt / 2, SW) &&
            encode_tmap(&ms, F32, g.a_scale, g.M, p.groups, g.ld_as * 4, pl.bt, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (swiglu && encode_interleaved(&mw, g, p.width)) {
    p.interleaved = 1;
    mw2 = mw;
  } else if (swiglu) {
    ok = ok && encode_tmap(&mw, U8, g.b, g.K, p.width, g.ldb, 128, 8, SW) &&
         encode_tmap(&mw2, U8, g.b2, g.K, p.width, g.ldb2, 128, 8, SW);
  } else {
    ok = ok && encode_tmap(&mw, U8, g.b, g.K, p.width, g.ldb, 128, ROWS, SW);
    mw2 = mw;
  }
  mc = mx;
  if (!pl.via_smem)
    ok = ok && (swiglu    ? encode_tmap(&mc, U8, g.c, p.width, g.M, g.ldc, 64, pl.bt / 2, CU_TENSOR_MAP_SWIZZLE_64B)
                : to_bf16 ? encode_tmap(&mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.c, p.width, g.M, g.ldc * 2, 32, 16,
                                        CU_TENSOR_MAP_SWIZZLE_64B)
                          : encode_tmap(&mc, F32, g.c, p.width, g.M, g.ldc * 4, 32, 16, SW));
  if (!ok) return cudaErrorInvalidValue;
  Kernel fn = kernel_of(pl.bt, swiglu, pl.via_smem);
  static DeviceOnce once[2][2][17];
  cudaError_t e = max_dynamic_smem_once(reinterpret_cast<const void*>(fn), SMEM_ALLOC,
                                        once[swiglu][pl.via_smem][pl.bt / 16]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pl.split * std::min(pl.clusters, p.units));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * pl.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = launch_overlap_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, mw2, ms, mc, static_cast<const Params>(p));
}

}  // namespace cb
