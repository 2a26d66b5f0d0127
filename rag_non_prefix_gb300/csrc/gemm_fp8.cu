// Product of two e4m3 matrices with a scale per group of 128 channels of a row of A (tokens) and
// per 128 x 128 block of B (weights):
//   acc[m][n] = sum over groups g of  (sa[g][m] * sb[n / 128][g]) * sum_{k in g} A[m][k] B[n][k]
// The product of the two scales is one fp32 number, made once per token, weight block and group.
//
// The tensor core sums the products of one group (four tcgen05.mma kind::f8f6f4 of 32 channels)
// into tensor memory; eight warps then read that sum, multiply it by the group's two scales and
// add it to fp32 registers (packed fp32, fma.rn.f32x2), while the tensor core works on the next
// groups in the rest of tensor memory.  Two kernels, both on CTA pairs (one CTA per SM, M = 256), and a
// third one for a handful of tokens without tensor memory (below):
//   - tokens on the tensor core's rows, 256 tokens x 256 features per pair, for many tokens: a
//     thread's 128 sums belong to one token, so one factor per group scales them all.
//   - weights on the rows, 256 features x 16 .. 128 tokens per pair, for few tokens: the padding is
//     16 tokens, and a cluster of S pairs may split the channels.  Every factor is then another one
//     per column; tensor memory is read as 16 lanes x 256 bits, which leaves a thread the factors of
//     a quarter of the columns only (with 32 lanes x 1 column it would be all of them).  The factors
//     cost a shared-memory cycle per warp, group and four columns, which is why this form does not
//     serve many tokens: at 256 tokens a group took ~1100 cycles with them and ~850 without.
// Roles of the warps, in both:
//   warp 0: TMA producer of codes
//   warp 1: tensor-memory owner, in even CTAs the MMA issuer
//   warps 2, 3: load the token scales and multiply them by the weight blocks' scales, a group each
//   in turn
//   warps 4-11: scaling, sums and epilogue
// A barrier poll costs ~110 cycles even when the phase is long over (measured), so that every role
// waits for one barrier per group where it can: a stage's `full` barrier counts its codes, its
// factors and the readers of the accumulator that its MMAs overwrite.
// Every wait is bounded: a warp that gives up records ST_WAIT_TIMEOUT and runs on without waiting
// or storing, so that the barriers it shares are still met; the cluster meets at its closing
// barrier before any CTA frees its tensor memory or leaves.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cstdio>

#include "common.cuh"
#include "internal.h"

namespace cb {

namespace f8 {

constexpr int THREADS = 384;
constexpr int ROWS = 128;                  // rows of the tensor core's tile per CTA
constexpr int A_BYTES = ROWS * 128;        // 16 KiB: 128 rows x one group of channels
constexpr int MAX_STAGES = 12;
constexpr int FACTORS = 2 * 4 * 20;        // token times block scales: 128 tokens, or two warpgroups x four thread classes x (16 + 4)
constexpr int FACTOR_BYTES = 2 * FACTORS * 4;  // a stage's two lists (two weight blocks)
constexpr int RAW_SLOTS = 4;               // token scales as loaded, per factor warp: slots of 128 floats
constexpr int OFF_AMAX = 1024;             // after the barriers: 512 words for the epilogue
constexpr int OFF_RAW = OFF_AMAX + 2048;
constexpr int OFF_SC = OFF_RAW + 2 * RAW_SLOTS * 512;  // factors of every stage, then the ring
constexpr int SMEM_ALLOC = 232448;         // the per-block maximum (227 KiB), 1 KiB of it aligns the base
constexpr int SMEM_USE = SMEM_ALLOC - 1024;
constexpr uint32_t TMEM_COLS = 512;
// Parts (few tokens): per source CTA and token its 128 rows, row 32 q + 8 r + i as float r of 16-byte piece
// i + q + 2 (source & 1) (mod 8) of the q-th 128 bytes: a thread of the sums holds r = 0 .. 3 and writes
// them at once, and lanes that read consecutive rows meet no bank twice.
__device__ __forceinline__ int part_at(int source, int row) {
  const int q = row >> 5, r = (row >> 3) & 3;
  return q * 32 + (((row + q + 2 * (source & 1)) & 7) << 2) + r;
}
constexpr int SLAB = 2048;                 // many tokens: a warp stages 32 tokens x 64 bytes twice, or x 128 bytes

// Accumulators in tensor memory: as many groups' sums as fit may wait to be read.
__host__ __device__ constexpr int n_acc(int columns) { return columns <= 128 ? 4 : 2; }

struct Params {
  Fp8Gemm g;
  int width;        // output features
  int tok_tiles, units;
  int split;        // pairs per cluster, each taking a part of the groups
  int groups;       // ceil(K / 128)
  int stages, stage_bytes;
  int ring_off, out_off;  // codes of the stages; output area
};

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D, both K-major, M = 256, N = n.
__device__ __forceinline__ uint32_t idesc_pair(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
}
// D (128 lanes in each CTA of the pair) (+)= A . B^T over 32 channels; issued by the even CTA.  The
// whole warp runs the issue loop and one elected lane (el) issues: its operands then stay in
// uniform registers.  In a branch of one lane each group cost ~300 cycles more (measured at 16
// tokens: 49 -> 35 us for 112 groups).
__device__ __forceinline__ void mma_f8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(el)
      : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t el;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(el));
  return el;
}
// tma_load_2d_pair and the arrival that expects its bytes, by the elected lane of a converged warp
__device__ __forceinline__ void tma_load_2d_pair_elected(uint32_t smem_dst, const CUtensorMap* map, uint32_t bar, int c0,
                                                         int c1, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(el)
      : "memory");
}
__device__ __forceinline__ void arrive_expect_tx_elected(uint32_t bar, uint32_t bytes, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(el)
      : "memory");
}
// tc_commit_pair_mc by the elected lane of a converged warp
__device__ __forceinline__ void commit_pair_mc_elected(uint64_t* bar, uint16_t cta_mask, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(cta_mask), "r"(el)
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

// The same for any number of 8-column pieces, as the largest reads that add up to it.
template <int N8> __device__ __forceinline__ void tmem_ld16x256_all(uint32_t taddr, uint32_t* r) {
  if constexpr (N8 >= 4) {
    tmem_ld16x256<4>(taddr, r);
    tmem_ld16x256_all<N8 - 4>(taddr + 32, r + 16);
  } else if constexpr (N8 >= 2) {
    tmem_ld16x256<2>(taddr, r);
    tmem_ld16x256_all<N8 - 2>(taddr + 16, r + 8);
  } else if constexpr (N8 == 1) {
    tmem_ld16x256<1>(taddr, r);
  }
}
// 32 lanes x 16 fp32 columns, without waiting: thread t gets lane t's columns.
__device__ __forceinline__ void tmem_ld32x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for this thread's tensor-memory reads; what was read into r may be used after it only.
template <int N> __device__ __forceinline__ void tmem_wait_ld_of(uint32_t* r) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
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
// N pairs of factors from shared memory (16-byte aligned)
template <int N> __device__ __forceinline__ void read_factors(const float* s, uint64_t* f) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s + 2 * i);
    f[i] = v.x;
    f[i + 1] = v.y;
  }
  if (N % 2) f[N - 1] = *reinterpret_cast<const uint64_t*>(s + 2 * (N - 1));
}

// ----------------------------------------------------------------------------- cluster exchange
// Four values into another CTA's shared memory whose bytes complete on that CTA's barrier.
__device__ __forceinline__ void st_async_f32x4(uint32_t addr, float x, float y, float z, float w, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
               "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(__float_as_uint(z)), "r"(__float_as_uint(w)), "r"(bar)
               : "memory");
}
// mbar_wait_bounded with acquire at cluster scope (what other CTAs wrote is read after it)
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
// Arrival of one lane (el) on a barrier of the cluster that orders no memory access.  It announces
// that tensor memory was read (tcgen05.wait::ld and the tcgen05 fence order that) or that parts were
// read and their values used, or follows a fence of its own.  With release at cluster scope the same
// arrival took ~1200 cycles.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr),
      "r"(el)
      : "memory");
}
// Arrival of one lane (el) on a barrier of this CTA, with release to the CTA.
__device__ __forceinline__ void mbar_arrive_elected(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ void fence_cta() { asm volatile("fence.acq_rel.cta;" ::: "memory"); }
__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// SiLU with the hardware's exponential and quotient (2 + 1.2 |x| and 2 units in the last place): the
// IEEE quotient made a tile's epilogue ~1 us longer.  The exponential is that of -|x|, so that the
// quotient's divisor is at most 2 (beyond 2^126 its result is 0, and exp(-x) is infinite below -88).
__device__ __forceinline__ float silu(float x) {
  const float e = __expf(-fabsf(x));
  return __fdividef(x >= 0.0f ? x : x * e, 1.0f + e);
}

struct Bars {
  // even CTAs: the codes of a stage have landed, both CTAs' factors are written and the eight warps
  // of both CTAs have read the accumulator
  uint64_t full[MAX_STAGES];
  uint64_t done[MAX_STAGES];      // its MMAs are done: the stage is free and the group's sums are readable
  uint64_t read[MAX_STAGES];      // few tokens: the eight warps of this CTA have read its factors
  uint64_t raw_full[2][RAW_SLOTS];  // token scales of a factor warp have landed
  uint64_t part_full;             // few tokens: the cluster's parts of this CTA's tokens have arrived
  uint64_t part_free;             // every CTA of the cluster has read its parts
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(Bars) <= OFF_AMAX, "barriers overrun their area");

__device__ __forceinline__ void init_bars(Bars& bars, int split) {
  for (int s = 0; s < MAX_STAGES; ++s) {
    mbar_init(&bars.full[s], 3 + 16);  // the producer of codes, the factor warps, the readers
    mbar_init(&bars.done[s], 1);
    mbar_init(&bars.read[s], 8);
  }
  for (int s = 0; s < 2 * RAW_SLOTS; ++s) mbar_init(&bars.raw_full[0][s], 1);
  mbar_init(&bars.part_full, 1);
  mbar_init(&bars.part_free, 16 * split);
  mbar_init(&bars.drain, 1);
  bars.abort = 0;
  fence_mbar_init();
}

__device__ __forceinline__ void report_timeout(Bars& bars, int32_t* status) {
  *const_cast<volatile int*>(&bars.abort) = 1;
  set_status(status, ST_WAIT_TIMEOUT);
}

// A ring position and its barrier parity.
struct Pos {
  uint32_t i = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++i == n) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// MMA issuer (a whole warp of an even CTA): the group's four MMAs into accumulator after accumulator.
template <int COLUMNS>
__device__ __forceinline__ void issue_mmas(Bars& bars, const Params& p, uint8_t* ring, uint32_t tmem, int n_groups,
                                           int cid, int NC, int pair, uint32_t rank, int lane) {
  constexpr uint32_t NACC = n_acc(COLUMNS), ACC_STRIDE = TMEM_COLS / NACC;
  volatile int* abort = &bars.abort;
  const uint32_t idesc = idesc_pair(COLUMNS);
  const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * pair));
  const uint32_t ring_u32 = smem_u32(ring), stages = static_cast<uint32_t>(p.stages);
  const uint32_t el = elect_one();
  uint32_t s = 0, ph = 0, sa = ring_u32, b = 0;
  bool ok = true;
  for (int u = cid; ok && u < p.units; u += NC) {
    for (int g = 0; g < n_groups; ++g) {
      if (!mbar_wait_bounded(&bars.full[s], ph, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t da = sw128_desc(sa), db = sw128_desc(sa + A_BYTES);
      const uint32_t tacc = tmem + b * ACC_STRIDE;
      mma_f8_pair(tacc, da, db, idesc, 0u, el);
      mma_f8_pair(tacc, da + 2, db + 2, idesc, 1u, el);  // + 32 bytes along K (encoded >> 4)
      mma_f8_pair(tacc, da + 4, db + 4, idesc, 1u, el);
      mma_f8_pair(tacc, da + 6, db + 6, idesc, 1u, el);
      commit_pair_mc_elected(&bars.done[s], pair_mask, el);
      sa += static_cast<uint32_t>(p.stage_bytes);
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
        sa = ring_u32;
      }
      if (++b == NACC) b = 0;
    }
  }
  if (!ok && lane == 0) report_timeout(bars, p.g.status);
  // no MMA may still be running when the cluster meets at its closing barrier
  commit_pair_mc_elected(&bars.drain, static_cast<uint16_t>(1u << rank), el);
  mbar_wait_bounded(&bars.drain, 0u, nullptr);
}

// TMA producer of codes (a whole warp): `load` starts the copies of group g into stage s.  The
// stages are waited for in pairs: the second one's MMAs are done after the first one's.
template <typename Load>
__device__ __forceinline__ void load_codes(Bars& bars, const Params& p, int g0, int g1, int cid, int NC, int lane,
                                           Load load) {
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  Pos s;
  bool ok = true;
  for (int u = cid; ok && u < p.units; u += NC) {
    const int wt = u / p.tok_tiles, tt = u - wt * p.tok_tiles;
    for (int g = g0; g < g1; g += 2) {
      Pos second = s;
      if (g + 1 < g1) second.next(stages);
      if (!mbar_wait_bounded(&bars.done[second.i], second.ph ^ 1u, &bars.abort)) {
        ok = false;
        break;
      }
      load(s.i, wt, tt, g);
      if (g + 1 < g1) load(second.i, wt, tt, g + 1);
      s = second;
      s.next(stages);
    }
  }
  if (!ok && lane == 0) report_timeout(bars, p.g.status);
}

// Factor warp `which` of two (all lanes): loads the token scales of every second group, RAW_SLOTS of
// them ahead, and multiplies them by the scales of two weight blocks, sb0 and sb1 of a unit's weight
// tile; `put` stores token t's two factors into the stage's lists.  When a list is free (the relaxed
// arrival that frees an accumulator orders no read of the lists):
//   few tokens: once its readers have announced that they hold the stage's previous factors (`read`,
//   an arrival that releases their reads to this CTA);
//   many tokens: once the MMAs n_acc groups later are done, which waited for the accumulator.  Readers
//   free it after the last of eight reads of tensor memory, when the sums of all reads but the last two
//   have used both factors (the values of more reads would not fit the registers).  (An arrival on
//   `read` of its own: 2048 x 7168 x 7168 with an addend 94 -> 100 us, 1357 x 7168 x 20480 170 -> 176.)
template <int TILE, int TOKENS, typename Blocks, typename Put>
__device__ __forceinline__ void multiply_scales(Bars& bars, const Params& p, const CUtensorMap* tmS, uint8_t* smem,
                                                int g0, int g1, int cid, int NC, int which, int lane, uint32_t lead,
                                                int tok_off, Blocks blocks, Put put) {
  constexpr bool MANY = TILE == 256;
  const uint32_t stages = static_cast<uint32_t>(p.stages), ahead = stages - n_acc(256);
  const uint32_t full_lead = mapa_shared(smem_u32(bars.full), lead), el = lane == 0;
  float* raw = reinterpret_cast<float*>(smem + OFF_RAW) + which * RAW_SLOTS * 128;
  uint8_t* sc = smem + OFF_SC;
  // the groups of this warp in their order, for the copies: unit, group
  int lu = cid, lg = g0 + which;
  while (lu < p.units && lg >= g1) {
    lg -= g1 - g0;
    lu += NC;
  }
  uint32_t slot_in = 0;
  auto load_next = [&]() {
    if (lu >= p.units) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars.raw_full[which][slot_in], TOKENS * 4);
      tma_load_2d(raw + slot_in * 128, tmS, &bars.raw_full[which][slot_in], (lu % p.tok_tiles) * TILE + tok_off, lg);
    }
    if (++slot_in == RAW_SLOTS) slot_in = 0;
    lg += 2;
    while (lu < p.units && lg >= g1) {
      lg -= g1 - g0;
      lu += NC;
    }
  };
  for (int i = 0; i < RAW_SLOTS; ++i) load_next();
  Pos s, done, r;
  uint32_t n = 0;  // groups so far
  bool ok = true;
  for (int u = cid; ok && u < p.units; u += NC) {
    const float *sb0, *sb1;
    blocks(u / p.tok_tiles, sb0, sb1);
    float b0 = 0.f, b1 = 0.f;  // 32 groups' block scales, one per lane
    for (int g = g0; g < g1; ++g, ++n) {
      const int i = (g - g0) & 31;
      if (i == 0 && g + lane < g1) {
        b0 = __ldg(sb0 + g + lane);
        b1 = __ldg(sb1 + g + lane);
      }
      if ((n & 1u) == static_cast<uint32_t>(which)) {
        const float f0 = __shfl_sync(0xffffffffu, b0, i), f1 = __shfl_sync(0xffffffffu, b1, i);
        ok = mbar_wait_bounded(&bars.raw_full[which][r.i], r.ph, &bars.abort) &&
             (MANY ? n < ahead || mbar_wait_bounded(&bars.done[done.i], done.ph, &bars.abort)
                   : mbar_wait_bounded(&bars.read[s.i], s.ph ^ 1u, &bars.abort));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        float* lists = reinterpret_cast<float*>(sc + s.i * FACTOR_BYTES);
#pragma unroll
        for (int t = lane; t < TOKENS; t += 32) {
          const float v = raw[r.i * 128 + t];
          put(lists, t, v * f0, v * f1);
        }
        fence_cta();  // the factors are read in this CTA only
        __syncwarp();
        mbar_arrive_cluster_relaxed(full_lead + s.i * 8, el);
        load_next();  // into the slot just read
        r.next(RAW_SLOTS);
      }
      s.next(stages);
      if (MANY && n >= ahead) done.next(stages);
    }
  }
  if (!ok && lane == 0) report_timeout(bars, p.g.status);
}

// Eight reader warps: the accumulators are free at first.
__device__ __forceinline__ void free_accumulators(Bars& bars, uint32_t lead, uint32_t n_accumulators, uint32_t el) {
  const uint32_t full_lead = mapa_shared(smem_u32(bars.full), lead);
  for (uint32_t s = 0; s < n_accumulators; ++s) mbar_arrive_cluster_relaxed(full_lead + s * 8, el);
}

// What every thread does last.
__device__ __forceinline__ void finish(Bars& bars, uint32_t tmem, int warp) {
  tc_fence_before();
  __syncthreads();
  // No CTA leaves, or frees the pair's tensor memory, while another may still reach its barriers or
  // shared memory: every issuer has drained its MMAs, every producer and epilogue has finished.
  cluster_sync_all();
  // After a timeout copies issued for stages that were never consumed may still be in flight to this
  // CTA: give them time to land before the memory is released.  (Its own flag says so: where a stage
  // was not consumed, its readers gave up too.)
  if (*const_cast<volatile int*>(&bars.abort)) {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 200000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// Registers: 384 threads launch with 168 each; the four service warps keep 40, the eight others take
// 232 (128 x 40 + 256 x 232 = 64,512 = 384 x 168).
__device__ __forceinline__ void few_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
__device__ __forceinline__ void many_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }

// ============================================================================= many tokens
// Tokens on the rows: thread r of a warpgroup holds token r of this CTA's 128, warpgroup w the
// features 128 w .. of the tile's 256 (SwiGLU: gate and up of features 64 w .. of 128; the pair's
// even CTA stages the gate rows, the odd one the up rows).  Bound by those eight warps: a group takes
// ~770 cycles of reading tensor memory and multiplying (~190 instructions a warp) against 512 of
// tensor core (active 65 % of 2048 x 7168 x 7168 bf16, 69 % with SwiGLU), and by the power limit in
// long runs.  2048 x 7168 x 7168 bf16 71 us (2.95 PFLOP/s), fp32 72 us, with an addend 88 us; 8320 x
// 40960 x 7168 SwiGLU 1530 us (3.2 PFLOP/s) before the power limit, 1815 us under it.
template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp8_tokens_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                           const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmS,
                           const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr uint32_t ACC_STRIDE = 256;
  constexpr bool SWIGLU = EPI == CB_FP8_SWIGLU_FP8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem);
  uint8_t* sc = smem + OFF_SC;
  uint32_t* amax = reinterpret_cast<uint32_t*>(smem + OFF_AMAX);  // [2][2][128]
  uint8_t* ring = smem + p.ring_off;
  volatile int* abort = &bars.abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int h = static_cast<int>(rank & 1u);
  const int cid = static_cast<int>(cluster_id_x()), NC = static_cast<int>(n_clusters_x());
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  const int G = p.groups;

  pdl_trigger();
  if (threadIdx.x == 0) init_bars(bars, 1);
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmS);
    if (SWIGLU || EPI == CB_FP8_STORE_BF16) prefetch_tmap(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars.tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers are initialised before another CTA reaches them
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  pdl_wait();

  if (warp < 4) {
    few_registers();
    if (warp == 0) {
      const uint32_t el = elect_one(), ring_u32 = smem_u32(ring), full_lead = mapa_shared(smem_u32(bars.full), 0);
      const CUtensorMap* w_map = SWIGLU && h ? &tmW2 : &tmW;
      load_codes(bars, p, 0, G, cid, NC, lane, [&](uint32_t s, int wt, int tt, int g) {
        const uint32_t a = ring_u32 + s * static_cast<uint32_t>(p.stage_bytes), bar = full_lead + s * 8;
        if (h == 0) arrive_expect_tx_elected(smem_u32(&bars.full[s]), 4u * A_BYTES, el);
        tma_load_2d_pair_elected(a, &tmX, bar, g * 128, tt * 256 + h * 128, el);
        tma_load_2d_pair_elected(a + A_BYTES, w_map, bar, g * 128, SWIGLU ? wt * 128 : wt * 256 + h * 128, el);
      });
    } else if (warp == 1 && h == 0) {
      issue_mmas<256>(bars, p, ring, tmem, G, cid, NC, 0, rank, lane);
    } else if (warp >= 2) {
      multiply_scales<256, 128>(
          bars, p, &tmS, smem, 0, G, cid, NC, warp - 2, lane, 0, h * 128,
          [&](int wt, const float*& sb0, const float*& sb1) {
            // features past the last block are zeros: any block's scale will do
            const int last = (p.width - 1) >> 7;
            sb0 = p.g.b_scale + static_cast<long long>(SWIGLU ? wt : wt * 2) * p.g.ld_bs;
            sb1 = SWIGLU ? p.g.b2_scale + static_cast<long long>(wt) * p.g.ld_b2s
                         : p.g.b_scale + static_cast<long long>(min(wt * 2 + 1, last)) * p.g.ld_bs;
          },
          [&](float* slot, int t, float v0, float v1) {
            slot[t] = v0;
            slot[FACTORS + t] = v1;
          });
    }
    __syncwarp();
  } else {
    many_registers();
    const int quarter = warp & 3, w = (warp >> 2) - 1;
    const int row = threadIdx.x & 127;  // this thread's token of the CTA's
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t full_lead = mapa_shared(smem_u32(bars.full), 0);
    // first column of the eight reads of 16: SwiGLU takes 64 of the gate and 64 of the up features
    const auto column = [&](int c) {
      return static_cast<uint32_t>(SWIGLU ? (c >> 2) * 128 + w * 64 + (c & 3) * 16 : w * 128 + c * 16);
    };
    uint8_t* mine = smem + p.out_off + (warp - 4) * 2 * SLAB;
    const uint32_t el = lane == 0;
    free_accumulators(bars, 0, 2, el);
    Pos st;
    uint32_t b = 0, slab_no = 0, next_use = 2;  // next_use: the stage whose MMAs overwrite accumulator b
    bool ok = true;
    int nth = 0;
    for (int u = cid; u < p.units; u += NC, ++nth) {
      uint64_t acc[4][16];  // [32 features][pair of them]
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[c][j] = 0;
      // Two register buffers: the next read of tensor memory runs under the sums of the current one.
      // (Reads of 32 columns, the next group's first among them, leave the compiler too few
      // registers: it moves sums about between groups, and 2048 x 7168 x 7168 takes 78 instead of
      // 72 us in bf16.)
      uint32_t v[2][16];
#pragma unroll 1
      for (int g = 0; g < G; ++g) {
        if (ok && !mbar_wait_bounded(&bars.done[st.i], st.ph, abort)) {
          ok = false;
          report_timeout(bars, p.g.status);
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t tacc = tmem + b * ACC_STRIDE + lane_base;
        tmem_ld32x16(tacc + column(0), v[0]);
        const float* f = reinterpret_cast<const float*>(sc + st.i * FACTOR_BYTES) + row;
        const float fa = f[SWIGLU ? 0 : w * FACTORS], fb = SWIGLU ? f[FACTORS] : fa;
        const uint64_t m0 = pack2(fa, fa), m1 = SWIGLU ? pack2(fb, fb) : m0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t* sum = v[c & 1];
          tmem_wait_ld_of<16>(v[c & 1]);
          if (c < 7) {
            tmem_ld32x16(tacc + column(c + 1), v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            mbar_arrive_cluster_relaxed(full_lead + next_use * 8, el);
            if (++next_use == stages) next_use = 0;
            b ^= 1u;
            st.next(stages);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint64_t& x = acc[c / 2][c % 2 * 8 + j];
            x = fma2(pack2u(sum[2 * j], sum[2 * j + 1]), c < 4 ? m0 : m1, x);
          }
        }
      }

      // ------------------------------------------------------------------ epilogue
      // (an index the compiler cannot know earlier: addresses computed before the sums would be spilled)
      int tile = u;
      asm volatile("" : "+r"(tile));
      const int wt = tile / p.tok_tiles, tt = tile - wt * p.tok_tiles;
      const int t0 = tt * 256 + h * 128 + quarter * 32;  // the warp's first token
      // 64 bytes of this thread's token into the next slab (64-byte swizzle), stored by TMA at feature f
      auto put = [&](const uint4* q, int f) {
        uint8_t* slab = mine + (slab_no++ & 1u) * SLAB;
        if (lane == 0) bulk_wait_read_all_but_1();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(slab + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = q[i];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && ok) tma_store_2d(&tmC, slab, f, t0);
        if (lane == 0) bulk_commit();
      };
      if constexpr (SWIGLU) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 gate = unpack2(acc[c][j]), up = unpack2(acc[c + 2][j]);
            const float2 y = make_float2(silu(gate.x) * up.x, silu(gate.y) * up.y);
            acc[c][j] = pack2(y.x, y.y);
            m = max(m, max(__float_as_uint(y.x) & 0x7fffffffu, __float_as_uint(y.y) & 0x7fffffffu));
          }
        // the group's other 64 features are the other warpgroup's (two buffers: the next tile's
        // maxima may be written before these are read)
        uint32_t* x = amax + (nth & 1) * 256;
        x[w * 128 + row] = m;
        named_bar(1, 256);
        const float a = __uint_as_float(max(max(x[row], x[128 + row]), __float_as_uint(FP8_AMAX_MIN)));
        const float inv = FP8_MAX / a;
        const int tok = t0 + lane;
        if (w == 0 && ok && tok < p.g.M) p.g.c_scale[static_cast<long long>(wt) * p.g.ld_cs + tok] = a / FP8_MAX;
        const int f = wt * 128 + w * 64;
        if (t0 < p.g.M && f < p.width) {  // (uniform in the warp)
          uint4 q[4];
          uint32_t* qw = reinterpret_cast<uint32_t*>(q);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 y0 = unpack2(acc[i >> 3][(i & 7) * 2]), y1 = unpack2(acc[i >> 3][(i & 7) * 2 + 1]);
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y0.x * inv, y0.y * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y1.x * inv, y1.y * inv), __NV_SATFINITE, __NV_E4M3);
            qw[i] = lo | (hi << 16);
          }
          put(q, f);
        }
      } else {
        // A warp's 32 tokens x 32 features turn in its slab (rows of 128 bytes, 8-byte pieces
        // exchanged by row), so that C is written and the addend read in whole lines, 8 lanes a row.
        // (The addend read by the tokens' own threads, row by row, cost ~9 us a tile.  16-byte stores
        // would tie the sums to aligned groups of four registers, which the compiler then moves about
        // in the main loop: 2048 x 7168 x 7168 in 92 instead of 71 us.)
        const int r4 = lane >> 3, q4 = (lane & 7) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int f = wt * 256 + w * 128 + c * 32 + q4;
          if (t0 >= p.g.M || f - q4 >= p.width) continue;  // (uniform in the warp)
          const bool whole = f + 4 <= p.width;
          if (EPI == CB_FP8_STORE_BF16 && (p.width % 8 == 0 || f - q4 + 32 <= p.width)) {
            // (a TMA store ends at 16 bytes: rows that end elsewhere take the other way)
            uint4 q[4];
            uint32_t* qw = reinterpret_cast<uint32_t*>(q);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = unpack2(acc[c][j]);
              qw[j] = pack_bf16x2(x.x, x.y);
            }
            put(q, f - q4);
            continue;
          }
          const long long o = static_cast<long long>(t0 + r4) * p.g.ldc + f;
          const int rows = p.g.M - t0 - r4;  // this lane's rows 4 i below it exist
          const long long step = 4 * p.g.ldc;
          // the addends of all eight rows are under way at once (four: 2048 x 7168 x 7168 in 95 instead
          // of 88 us, which is the burst of all tiles' addends and outputs at HBM's rate)
          float4 d[8];
          if constexpr (EPI == CB_FP8_ADD_F32) {
            const float* from = p.g.addend + o;
#pragma unroll
            for (int i = 0; i < 8; ++i, from += step)
              if (whole && 4 * i < rows) d[i] = *reinterpret_cast<const float4*>(from);
          }
          if (EPI == CB_FP8_STORE_BF16 && lane == 0) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 16; ++j) *reinterpret_cast<uint64_t*>(mine + lane * 128 + ((j ^ (lane & 15)) << 3)) = acc[c][j];
          __syncwarp();
          const auto turned = [&](int i) {
            const int row = r4 + 4 * i;
            const float4 x = *reinterpret_cast<const float4*>(mine + row * 128 + ((((lane & 7) * 2) ^ (row & 14)) << 3));
            return row & 1 ? make_float4(x.z, x.w, x.x, x.y) : x;
          };
          uint8_t* to = static_cast<uint8_t*>(p.g.c) + o * (EPI == CB_FP8_STORE_BF16 ? 2 : 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 x = turned(i);
            if (EPI == CB_FP8_ADD_F32) {
              const float4 a = d[i];
              x = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
            }
            if (ok && whole && 4 * i < rows) {
              if (EPI == CB_FP8_STORE_BF16)
                *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
              else
                *reinterpret_cast<float4*>(to) = x;
            }
            to += step * (EPI == CB_FP8_STORE_BF16 ? 2 : 4);
          }
          if (ok && !whole) {  // rows that end inside four features
#pragma unroll 1
            for (int i = 0; i < 8 && t0 + r4 + 4 * i < p.g.M; ++i) {
              const float4 x = turned(i);
              const float y[3] = {x.x, x.y, x.z};
#pragma unroll
              for (int k = 0; k < 3; ++k) {
                if (f + k >= p.width) continue;
                const long long at = o + 4 * i * p.g.ldc + k;
                if (EPI == CB_FP8_STORE_BF16)
                  static_cast<bf16*>(p.g.c)[at] = __float2bfloat16_rn(y[k]);
                else
                  static_cast<float*>(p.g.c)[at] = EPI == CB_FP8_ADD_F32 ? p.g.addend[at] + y[k] : y[k];
              }
            }
          }
        }
      }
    }
    if (SWIGLU || EPI == CB_FP8_STORE_BF16) bulk_wait_all();
  }
  finish(bars, tmem, warp);
}

// ============================================================================= few tokens
// Weights on the rows: BT tokens per pair, warpgroup w takes tokens w BT / 2 .. .  SwiGLU: a CTA's
// rows are 64 gate rows and the 64 up rows of the same features.  A cluster of S pairs splits the
// groups; each of its 2 S CTAs finishes 1 / (2 S) of the tokens for all 256 rows, adding the S parts
// in a fixed order.  The parts are pushed into the finishing CTA's shared memory (st.async, counted
// in bytes on its barrier): a barrier with release at cluster scope and reads from the other side
// took ~1.3 us longer.  Bound by the weights' bytes; what a call of few groups spends on top is the
// way through the chip (set-up 0.9 us, first codes 1.7 us, parts and output ~1 us), and the last round
// of tiles, which may leave pairs idle: 16 x 4096 x 14336 with an addend 15 us (4.0 TB/s), 16 x 28672 x
// 4096 bf16 25 us (4.7 TB/s), 64 x 28672 x 4096 SwiGLU 28.5 us, 77 x 11008 x 4112 bf16 16 us.  (A second
// launch for the last round, which pays for many tokens, made these 2 to 5 us slower.)  Parts pushed
// four bytes at a time took 64 x 4096 x 14336 from 16.7 to 17.8 us, 128 x 4096 x 4096 from 13.0 to 17.4.
template <int BT, bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp8_weights_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                            const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmS,
                            const __grid_constant__ CUtensorMap, const Params p) {
  constexpr int HB = BT / 2;  // tokens per warpgroup
  constexpr int N8 = HB / 8;
  constexpr uint32_t NACC = n_acc(BT), ACC_STRIDE = TMEM_COLS / NACC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem);
  uint8_t* sc = smem + OFF_SC;
  uint8_t* ring = smem + p.ring_off;
  volatile int* abort = &bars.abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(rank >> 1), h = static_cast<int>(rank & 1u);
  const uint32_t lead = rank & ~1u;
  const int cid = static_cast<int>(cluster_id_x()), NC = static_cast<int>(n_clusters_x());
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  // this pair's groups of channels
  const int g0 = static_cast<int>(static_cast<long long>(p.groups) * pair / p.split);
  const int g1 = static_cast<int>(static_cast<long long>(p.groups) * (pair + 1) / p.split);

  pdl_trigger();
  if (threadIdx.x == 0) init_bars(bars, p.split);
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmS);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars.tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers are initialised before another CTA reaches them
  tc_fence_after();
  const uint32_t tmem = bars.tmem_slot;
  pdl_wait();

  if (warp < 4) {
    few_registers();
    if (warp == 0) {
      const uint32_t el = elect_one(), ring_u32 = smem_u32(ring), full_lead = mapa_shared(smem_u32(bars.full), lead);
      load_codes(bars, p, g0, g1, cid, NC, lane, [&](uint32_t s, int wt, int tt, int g) {
        const uint32_t a = ring_u32 + s * static_cast<uint32_t>(p.stage_bytes), bar = full_lead + s * 8;
        if (h == 0) arrive_expect_tx_elected(smem_u32(&bars.full[s]), 2u * (A_BYTES + HB * 128), el);
        if (SWIGLU) {
          tma_load_2d_pair_elected(a, &tmW, bar, g * 128, wt * 128 + h * 64, el);
          tma_load_2d_pair_elected(a + A_BYTES / 2, &tmW2, bar, g * 128, wt * 128 + h * 64, el);
        } else {
          tma_load_2d_pair_elected(a, &tmW, bar, g * 128, wt * 256 + h * 128, el);
        }
        tma_load_2d_pair_elected(a + A_BYTES, &tmX, bar, g * 128, tt * BT + h * HB, el);
      });
    } else if (warp == 1 && h == 0) {
      issue_mmas<BT>(bars, p, ring, tmem, g1 - g0, cid, NC, pair, rank, lane);
    } else if (warp >= 2) {
      multiply_scales<BT, BT>(
          bars, p, &tmS, smem, g0, g1, cid, NC, warp - 2, lane, lead, 0,
          [&](int wt, const float*& sb0, const float*& sb1) {
            // rows past the last block are zeros: any block's scale will do
            const int blk = SWIGLU ? wt : min(wt * 2 + h, (p.width - 1) >> 7);
            sb0 = p.g.b_scale + static_cast<long long>(blk) * p.g.ld_bs;
            sb1 = SWIGLU ? p.g.b2_scale + static_cast<long long>(blk) * p.g.ld_b2s : sb0;
          },
          [](float* slot, int t, float v0, float v1) {
            // Thread class c of the readers takes tokens 8 j + 2 c, + 1: stored class by class, so that
            // one 16-byte read gives four factors, the classes 20 floats apart in different banks.
            const int tw = t < HB ? 0 : 1, x = t - tw * HB;
            const int o = tw * (FACTORS / 2) + ((x >> 1) & 3) * 20 + (x >> 3) * 2 + (x & 1);
            slot[o] = v0;
            if (SWIGLU) slot[FACTORS + o] = v1;
          });
    }
    __syncwarp();
  } else {
    many_registers();
    const int quarter = warp & 3, w = (warp >> 2) - 1;  // tensor-memory lanes 32 quarter .., tokens w HB ..
    const int et = threadIdx.x - 128;  // thread of the eight warps
    const int ri = lane >> 2, ci = (lane & 3) * 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t full_lead = mapa_shared(smem_u32(bars.full), lead);
    float* part = reinterpret_cast<float*>(smem + p.out_off);  // [CS][per][ROWS]
    const uint32_t piece = part_at(rank, quarter * 32 + ri);  // of the rows quarter * 32 + ri + 8 r
    const uint32_t part_u32 = smem_u32(part), part_full_u32 = smem_u32(&bars.part_full);
    const int CS = 2 * p.split;
    const int per = (BT / 2 + CS - 1) / CS * 2;  // tokens that each CTA of the cluster finishes, an even number
    const int mine = max(0, min(per, BT - static_cast<int>(rank) * per));
    const uint32_t per_inverse = 65536u / per + 1;  // tok / per = tok * per_inverse >> 16 for tok < 128
    const uint32_t el = lane == 0;
    free_accumulators(bars, lead, NACC, el);
    Pos st;
    uint32_t b = 0, next_use = NACC;  // next_use: the stage whose MMAs overwrite accumulator b
    bool ok = true;
    int nth = 0;
    auto give_up = [&]() {
      ok = false;
      report_timeout(bars, p.g.status);
    };
    for (int u = cid; u < p.units; u += NC, ++nth) {
      const int wt = u / p.tok_tiles, tt = u - wt * p.tok_tiles;
      const int t0 = tt * BT;
      uint64_t acc[HB / 8][4];  // per 8 tokens: rows i/4, + 8, + 16, + 24 of the quarter, 2 tokens each
#pragma unroll
      for (int j = 0; j < HB / 8; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0;
#pragma unroll 1
      for (int g = g0; g < g1; ++g) {
        if (ok && !mbar_wait_bounded(&bars.done[st.i], st.ph, abort)) give_up();
        __syncwarp();
        tc_fence_after();
        const uint32_t tacc = tmem + b * ACC_STRIDE + lane_base + static_cast<uint32_t>(w * HB);
        uint32_t lo[N8 * 4], hi[N8 * 4];
        tmem_ld16x256_all<N8>(tacc, lo);
        tmem_ld16x256_all<N8>(tacc + (16u << 16), hi);
        uint64_t f[N8];
        read_factors<N8>(reinterpret_cast<const float*>(sc + st.i * FACTOR_BYTES) +
                             (SWIGLU && quarter >= 2 ? FACTORS : 0) + w * (FACTORS / 2) + (lane & 3) * 20,
                         f);
        tmem_wait_ld_of<N8 * 4>(lo);
        tmem_wait_ld_of<N8 * 4>(hi);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_elected(&bars.read[st.i], el);
        mbar_arrive_cluster_relaxed(full_lead + next_use * 8, el);
        if (++next_use == stages) next_use = 0;
        if (++b == NACC) b = 0;
        st.next(stages);
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          acc[j][0] = fma2(pack2u(lo[4 * j], lo[4 * j + 1]), f[j], acc[j][0]);
          acc[j][1] = fma2(pack2u(lo[4 * j + 2], lo[4 * j + 3]), f[j], acc[j][1]);
          acc[j][2] = fma2(pack2u(hi[4 * j], hi[4 * j + 1]), f[j], acc[j][2]);
          acc[j][3] = fma2(pack2u(hi[4 * j + 2], hi[4 * j + 3]), f[j], acc[j][3]);
        }
      }

      // ------------------------------------------------------------------ epilogue
      const uint32_t parity = nth & 1;
      const int n = min(mine, p.g.M - t0 - static_cast<int>(rank) * per);  // tokens to finish here (none: <= 0)
      const int tok0 = t0 + static_cast<int>(rank) * per;
      if (et == 0) mbar_arrive_expect_tx(&bars.part_full, static_cast<uint32_t>(mine * (CS - 1) * ROWS * 4));
      // the parts of the previous tile have been read by the whole cluster
      if (ok && !mbar_wait_cluster(&bars.part_free, parity ^ 1u, abort)) give_up();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        const int tok = w * HB + j * 8 + ci;  // and the next one: the same CTA finishes both
        const uint32_t to = static_cast<uint32_t>(tok) * per_inverse >> 16;
        const uint32_t at = (rank * per + tok - to * per) * ROWS + piece;
        const float2 v0 = unpack2(acc[j][0]), v1 = unpack2(acc[j][1]), v2 = unpack2(acc[j][2]), v3 = unpack2(acc[j][3]);
        if (to == rank) {
          *reinterpret_cast<float4*>(part + at) = make_float4(v0.x, v1.x, v2.x, v3.x);
          *reinterpret_cast<float4*>(part + at + ROWS) = make_float4(v0.y, v1.y, v2.y, v3.y);
        } else {
          const uint32_t bar = mapa_shared(part_full_u32, to), d = mapa_shared(part_u32 + at * 4, to);
          st_async_f32x4(d, v0.x, v1.x, v2.x, v3.x, bar);
          st_async_f32x4(d + ROWS * 4, v0.y, v1.y, v2.y, v3.y, bar);
        }
      }
      named_bar(1, 256);  // this CTA's own parts are written
      if constexpr (!SWIGLU) {
        // thread: 4 features of every fourth token
        const int q4 = et & 63, f = wt * 256 + q4 * 4, tg = et >> 6;
        const float* src = part + (q4 >> 5) * per * ROWS;
        int at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = part_at(q4 >> 5, (q4 & 31) * 4 + i);
        const bool add = p.g.epilogue == CB_FP8_ADD_F32, whole = f + 4 <= p.width;
        constexpr int AHEAD = 4;  // addends read before the parts are there
        float4 d[AHEAD];
        if (add && whole)
#pragma unroll
          for (int i = 0; i < AHEAD; ++i)
            if (tg + 4 * i < n)
              d[i] = *reinterpret_cast<const float4*>(p.g.addend + static_cast<long long>(tok0 + tg + 4 * i) * p.g.ldc + f);
        if (ok && !mbar_wait_cluster(&bars.part_full, parity, abort)) give_up();
        __syncwarp();
        auto finish_token = [&](int j, bool have, float4 ahead) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s = 0; s < p.split; ++s) {
            const float* x = src + (2 * s * per + j) * ROWS;
            v.x += x[at[0]];
            v.y += x[at[1]];
            v.z += x[at[2]];
            v.w += x[at[3]];
          }
          const long long o = static_cast<long long>(tok0 + j) * p.g.ldc + f;
          if (!ok) return;
          if (whole) {
            if (p.g.epilogue == CB_FP8_STORE_BF16) {
              *reinterpret_cast<uint2*>(static_cast<bf16*>(p.g.c) + o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
              return;
            }
            if (add) {
              const float4 a = have ? ahead : *reinterpret_cast<const float4*>(p.g.addend + o);
              v = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
            }
            *reinterpret_cast<float4*>(static_cast<float*>(p.g.c) + o) = v;
            return;
          }
          const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (f + i >= p.width) continue;
            if (p.g.epilogue == CB_FP8_STORE_BF16)
              static_cast<bf16*>(p.g.c)[o + i] = __float2bfloat16_rn(x[i]);
            else
              static_cast<float*>(p.g.c)[o + i] = add ? p.g.addend[o + i] + x[i] : x[i];
          }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (tg + 4 * i < n) finish_token(tg + 4 * i, true, d[i]);
        for (int j = tg + 4 * AHEAD; j < n; j += 4) finish_token(j, false, make_float4(0.f, 0.f, 0.f, 0.f));
      } else {
        // a warp per token, lane x takes features 4 x .. of the tile's 128
        const float* src = part + (lane >> 4) * per * ROWS;
        int ga[4], ua[4];  // gate rows, up rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga[i] = part_at(lane >> 4, (lane & 15) * 4 + i);
          ua[i] = part_at(lane >> 4, 64 + (lane & 15) * 4 + i);
        }
        const int f = wt * 128 + lane * 4;
        if (ok && !mbar_wait_cluster(&bars.part_full, parity, abort)) give_up();
        __syncwarp();
        constexpr int AT_ONCE = 4;  // tokens of a warp whose latencies overlap
        for (int jb = warp - 4; jb < n; jb += 8 * AT_ONCE) {
          float y[AT_ONCE][4];
          uint32_t m[AT_ONCE];
#pragma unroll
          for (int q = 0; q < AT_ONCE; ++q) {
            const int j = min(jb + 8 * q, n - 1);  // (past the last token: computed again, not stored)
            float4 gate = make_float4(0.f, 0.f, 0.f, 0.f), up = gate;
            for (int s = 0; s < p.split; ++s) {
              const float* x = src + (2 * s * per + j) * ROWS;
              gate = make_float4(gate.x + x[ga[0]], gate.y + x[ga[1]], gate.z + x[ga[2]], gate.w + x[ga[3]]);
              up = make_float4(up.x + x[ua[0]], up.y + x[ua[1]], up.z + x[ua[2]], up.w + x[ua[3]]);
            }
            y[q][0] = silu(gate.x) * up.x;
            y[q][1] = silu(gate.y) * up.y;
            y[q][2] = silu(gate.z) * up.z;
            y[q][3] = silu(gate.w) * up.w;
            m[q] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) m[q] = max(m[q], __float_as_uint(y[q][i]) & 0x7fffffffu);
            if (f >= p.width) m[q] = 0u;
          }
#pragma unroll
          for (int q = 0; q < AT_ONCE; ++q) m[q] = __reduce_max_sync(0xffffffffu, m[q]);
#pragma unroll
          for (int q = 0; q < AT_ONCE; ++q) {
            const int j = jb + 8 * q;
            const float a = __uint_as_float(max(m[q], __float_as_uint(FP8_AMAX_MIN))), inv = FP8_MAX / a;
            const uint32_t c01 =
                __nv_cvt_float2_to_fp8x2(make_float2(y[q][0] * inv, y[q][1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t c23 =
                __nv_cvt_float2_to_fp8x2(make_float2(y[q][2] * inv, y[q][3] * inv), __NV_SATFINITE, __NV_E4M3);
            if (!ok || j >= n) continue;
            if (f < p.width)
              *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.g.c) + static_cast<long long>(tok0 + j) * p.g.ldc + f) =
                  c01 | (c23 << 16);
            if (lane == 0) p.g.c_scale[static_cast<long long>(wt) * p.g.ld_cs + tok0 + j] = a / FP8_MAX;
          }
        }
      }
      __syncwarp();
      // (the reads are over: their values were used)
      mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&bars.part_free), lane < CS ? lane : 0), lane < CS);
    }
  }
  finish(bars, tmem, warp);
}

// ============================================================================= a handful of tokens
// Up to 16 tokens: the weights are streamed once through registers and the warps' own matrix instruction
// (mma.sync m16n8k32, weights on its 16 rows, 8 tokens a column block), without tensor memory,
// clusters and barriers, whose set-up and hand-over take longer than a few MB.  A CTA per 16 features, its
// 8 warps taking every eighth group; their sums are added in order.  Both operands take their 32
// channels in the same permuted order: lane c of four holds 16 consecutive bytes of a row, words 0 and 1
// for one product and 2 and 3 for the next.  Bound by the latency of its few reads (1 x 6144 x 4096 6.4 us,
// 3.9 TB/s) and by HBM for larger matrices (1 x 32000 x 4096 24 us, 5.4 TB/s); the instruction is slow here
// (~70 cycles each), which ends its use at more tokens (handful_applies).
__device__ __forceinline__ void mma_e4m3(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load16_or_zero(const uint8_t* p, bool in) {
  return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

template <int NT>
__global__ void __launch_bounds__(256, NT == 1 ? 3 : 2) gemm_fp8_handful_kernel(const Fp8Gemm p) {
  constexpr int WARPS = 8, UNROLL = 2;  // groups whose reads are under way together
  __shared__ float red[WARPS][16][NT * 8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int groups = (p.K + 127) / 128, row0 = blockIdx.x * 16;
  // (rows past the last one read the last one again; their sums are not stored)
  const uint8_t* w0 = p.b + min(row0 + r, p.N - 1) * p.ldb + c * 16;
  const uint8_t* w8 = p.b + min(row0 + r + 8, p.N - 1) * p.ldb + c * 16;
  const float* sb = p.b_scale + static_cast<long long>(row0 >> 7) * p.ld_bs;
  float acc[NT][4] = {};
  for (int gb = warp; gb < groups; gb += WARPS * UNROLL) {
    uint4 a[UNROLL][2][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const int k = (gb + u * WARPS) * 128 + ch * 64;
        const bool in = k + c * 16 < p.K;
        a[u][ch][0] = load16_or_zero(w0 + k, in);
        a[u][ch][1] = load16_or_zero(w8 + k, in);
      }
    // (tokens and scales come with the weights, not after them: 1 x 6144 x 4096 6.6 instead of 7.3 us)
    uint4 xs[UNROLL][NT][2];
    float fs[UNROLL], ss[UNROLL][NT][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int g = gb + u * WARPS;
      const bool here = g < groups;
      fs[u] = here ? __ldg(sb + g) : 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int tok = n * 8 + r, t = n * 8 + 2 * c;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const int k = g * 128 + ch * 64 + c * 16;
          xs[u][n][ch] = load16_or_zero(p.a + tok * p.lda + k, tok < p.M && k < p.K);
        }
        const float* sa = p.a_scale + g * p.ld_as + t;
        ss[u][n][0] = here && t < p.M ? __ldg(sa) : 0.f;
        ss[u][n][1] = here && t + 1 < p.M ? __ldg(sa + 1) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int g = gb + u * WARPS;
      if (g >= groups) break;
      const float f = fs[u];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float part[4] = {};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const uint4 x = xs[u][n][ch];
          const uint4 lo = a[u][ch][0], hi = a[u][ch][1];
          mma_e4m3(part, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
          mma_e4m3(part, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
        }
        const float s0 = ss[u][n][0] * f, s1 = ss[u][n][1] * f;
        acc[n][0] = fmaf(part[0], s0, acc[n][0]);
        acc[n][1] = fmaf(part[1], s1, acc[n][1]);
        acc[n][2] = fmaf(part[2], s0, acc[n][2]);
        acc[n][3] = fmaf(part[3], s1, acc[n][3]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][r + (i >> 1) * 8][n * 8 + 2 * c + (i & 1)] = acc[n][i];
  __syncthreads();
  const int row = threadIdx.x & 15, tok = threadIdx.x >> 4, f = row0 + row;
  if (tok >= p.M || f >= p.N) return;
  float v = 0.f;
#pragma unroll
  for (int s = 0; s < WARPS; ++s) v += red[s][row][tok];
  const long long o = tok * p.ldc + f;
  if (p.epilogue == CB_FP8_STORE_BF16)
    static_cast<bf16*>(p.c)[o] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.c)[o] = p.epilogue == CB_FP8_ADD_F32 ? p.addend[o] + v : v;
}

}  // namespace f8

// ============================================================================= planner + launcher
namespace {

using namespace f8;

typedef void (*Kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                       const Params);

// The kernel for `bt` tokens per tile: 256 has the tokens on the rows.
Kernel kernel_of(int bt, int epilogue) {
  const bool swiglu = epilogue == CB_FP8_SWIGLU_FP8;
  switch (bt) {
    case 16: return swiglu ? gemm_fp8_weights_kernel<16, true> : gemm_fp8_weights_kernel<16, false>;
    case 32: return swiglu ? gemm_fp8_weights_kernel<32, true> : gemm_fp8_weights_kernel<32, false>;
    case 48: return swiglu ? gemm_fp8_weights_kernel<48, true> : gemm_fp8_weights_kernel<48, false>;
    case 64: return swiglu ? gemm_fp8_weights_kernel<64, true> : gemm_fp8_weights_kernel<64, false>;
    case 80: return swiglu ? gemm_fp8_weights_kernel<80, true> : gemm_fp8_weights_kernel<80, false>;
    case 96: return swiglu ? gemm_fp8_weights_kernel<96, true> : gemm_fp8_weights_kernel<96, false>;
    case 128: return swiglu ? gemm_fp8_weights_kernel<128, true> : gemm_fp8_weights_kernel<128, false>;
    case 256:
      return swiglu                            ? gemm_fp8_tokens_kernel<CB_FP8_SWIGLU_FP8>
             : epilogue == CB_FP8_ADD_F32    ? gemm_fp8_tokens_kernel<CB_FP8_ADD_F32>
             : epilogue == CB_FP8_STORE_BF16 ? gemm_fp8_tokens_kernel<CB_FP8_STORE_BF16>
                                             : gemm_fp8_tokens_kernel<CB_FP8_STORE_F32>;
    default: return nullptr;
  }
}

// Clusters of one to four pairs that are resident at once (one CTA per SM); 0 where the query fails.
struct Resident {
  int clusters[4];
};
int query_resident_clusters(int cs) {
  const void* fn = reinterpret_cast<const void*>(kernel_of(16, CB_FP8_STORE_F32));
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
  return n;
}
Resident resident_clusters() {
  static std::atomic<int> cache[64][4];  // per device
  Resident r{};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return r;
  for (int i = 0; i < 4; ++i) {
    const bool cached = dev >= 0 && dev < 64;
    if (cached) r.clusters[i] = cache[dev][i].load(std::memory_order_relaxed);
    if (r.clusters[i] > 0) continue;
    r.clusters[i] = query_resident_clusters(2 * i + 2);
    if (cached) cache[dev][i].store(r.clusters[i], std::memory_order_relaxed);
  }
  return r;
}

// cb_gemm_scaled_set_plan: tokens per tile (0: the model decides) * 8 + pairs per cluster.  A call reads
// it once and hands it down (`hook`), so that all its decisions agree.
std::atomic<int> g_plan{0};

constexpr int HANDFUL_PLAN = 1 * 8;  // cb_gemm_scaled_set_plan(1, 0)

struct Plan {
  int bt, split, clusters, stages, stage_bytes, ring_off, out_off;
  double us;  // expected time
};

// Time model (microseconds, fitted to 3000 runs on GB300 at ~1.9 GHz over 1 .. 1000 tokens of nine decoder
// shapes; over 145 of them measured again, each under every tiling, its choice (two products among them)
// is as fast as the best tiling on average and 11 percent slower at worst): a group takes 0.39 us with
// 256 tokens on the rows and 0.18 + 0.0017 bt us with the weights on them, a unit's output 1.9 us and
// 1.7 + 0.017 bt us; units go round the resident clusters (76 of one pair, 36 of two, 23 of three, 15
// of four); the weights come at 6.5 TB/s at the most.
Plan plan(const Fp8Gemm& g, const Resident& resident, int hook) {
  const bool swiglu = g.epilogue == CB_FP8_SWIGLU_FP8;
  const int width = swiglu ? g.N / 2 : g.N, groups = (g.K + 127) / 128;
  const int w_tiles = swiglu ? (width + 127) / 128 : (width + 255) / 256;
  const int forced = hook == HANDFUL_PLAN ? 0 : hook;
  Plan best{};
  double best_us = 1e30;
  auto consider = [&](int bt, int split) {
    if (forced && forced != bt * 8 + split) return;
    split = std::min(split, groups);
    const int clusters = resident.clusters[split - 1];
    if (clusters <= 0) return;
    const long long tiles = (g.M + bt - 1) / bt, units = tiles * w_tiles;
    const double waves = static_cast<double>((units + clusters - 1) / clusters);
    const bool tokens = bt == 256;
    const double group_us = tokens ? 0.39 : 0.18 + 0.0017 * bt;
    const double epi_us = tokens ? 1.9 : 1.7 + 0.017 * bt;
    const double work = waves * ((groups + split - 1) / split * group_us + epi_us);
    const double stream = static_cast<double>(g.N) * g.K / 6.5e6;
    const double us = std::max(work, stream) + 0.13 * std::min(work, stream);
    if (us < best_us) {
      const int stage = A_BYTES + (tokens ? A_BYTES : bt * 64);
      // (parts: 2 split CTAs' sums of as many tokens as one CTA finishes)
      const int per = (bt / 2 + 2 * split - 1) / (2 * split) * 2;
      const int out = tokens ? 16 * SLAB : (2 * split * per * ROWS * 4 + 1023) / 1024 * 1024;
      best_us = us;
      const int room = SMEM_USE - OFF_SC - 1023 - out;
      best = Plan{bt, split, clusters, std::min(MAX_STAGES, room / (stage + FACTOR_BYTES)), stage, 0, 0, us};
      best.ring_off = (OFF_SC + best.stages * FACTOR_BYTES + 1023) / 1024 * 1024;
      best.out_off = best.ring_off + best.stages * stage;
    }
  };
  for (int bt : {16, 32, 48, 64, 80, 96, 128}) {
    for (int split = 1; split <= 4; ++split) consider(bt, split);
    if (bt >= g.M && !forced) break;  // (larger tiles only pad)
  }
  consider(256, 1);
  return best;
}

// Where the kernel for a handful of tokens is the faster one.  Up to 8 tokens nearly everywhere but for
// long sums (us, this kernel and the other, one token): 4096 x 4096 6.0 / 7.7, 6144 x 4096 6.4 / 8.8, 7168 x
// 7168 11.2 / 12.8, 28672 x 1024 8.7 / 9.3, 57344 x 8192 73 / 80, but 8192 x 8192 15.6 / 15.0 and 4096 x
// 14336 15.3 / 14.9; and where its many CTAs have little to do each (43776 x 512 9.5 / 8.5, 100000 x
// 1024 26 / 25).  Up to 16 for one wave of its CTAs (two an SM) and short sums: 16 tokens 6.9 / 7.9 at 4096
// x 4096, but 10.7 / 9.1 at 6144 x 4096 and 11.0 / 10.8 at 4096 x 8192.
constexpr int GB300_SMS = 152;
bool handful_applies(const Fp8Gemm& g, int hook) {
  if (g.M > 16 || g.epilogue == CB_FP8_SWIGLU_FP8) return false;
  if (hook) return hook == HANDFUL_PLAN;
  if (g.M > 8) return g.K <= 4096 && g.N <= 16 * GB300_SMS * 2;
  return g.K <= 8192 && (g.K >= 2048 || g.N <= 4 * 16 * GB300_SMS * 3);
}

// The product of the first `n` tokens, or of the first `n` output features, and the rest of it.
Fp8Gemm first_tokens(const Fp8Gemm& g, int n) {
  Fp8Gemm r = g;
  r.M = n;
  return r;
}
long long element_size(const Fp8Gemm& g) {
  return g.epilogue == CB_FP8_SWIGLU_FP8 ? 1 : g.epilogue == CB_FP8_STORE_BF16 ? 2 : 4;
}
Fp8Gemm other_tokens(const Fp8Gemm& g, int n) {
  Fp8Gemm r = g;
  r.M = g.M - n;
  r.a += n * g.lda;
  r.a_scale += n;
  r.c = static_cast<uint8_t*>(g.c) + n * g.ldc * element_size(g);
  if (g.addend) r.addend += n * g.ldc;
  if (g.c_scale) r.c_scale += n;
  return r;
}
Fp8Gemm first_features(const Fp8Gemm& g, int n) {
  Fp8Gemm r = g;
  r.N = g.epilogue == CB_FP8_SWIGLU_FP8 ? 2 * n : n;
  return r;
}
Fp8Gemm other_features(const Fp8Gemm& g, int n) {
  Fp8Gemm r = g;
  r.N = g.N - first_features(g, n).N;
  r.b += n * g.ldb;
  r.b_scale += n / 128 * g.ld_bs;
  if (g.b2) {
    r.b2 += n * g.ldb2;
    r.b2_scale += n / 128 * g.ld_b2s;
  }
  r.c = static_cast<uint8_t*>(g.c) + n * element_size(g);
  if (g.addend) r.addend += n;
  if (g.c_scale) r.c_scale += n / 128 * g.ld_cs;
  return r;
}

// Many tokens leave most pairs idle in the last round of 256 x 256 tiles when that round is short.
// Then the tiles that fill whole rounds are computed first and the remaining tokens or features as
// a product of their own, whose plan spreads them over all pairs (smaller tiles, split channels).
// Measured on GB300 (us, one part and two): 535 x 7168 x 7168 56 / 40, 535 x 7168 x 20480 136 / 97,
// 1100 x 4096 x 14336 99 / 70, 1357 x 7168 x 20480 206 / 176, 8320 x 8192 x 8192 433 / 410; where the model promises less than
// 4 percent two parts took up to 9 percent longer (700 x 8192 x 8192 58 / 63).
constexpr double SECOND_LAUNCH_US = 4, WORTH_IT = 0.96;
// How a call runs: the kernel for a handful of tokens, or one or two products with their plans.
struct Schedule {
  bool handful = false;
  int n = 0;
  Fp8Gemm g[2];
  Plan pl[2];
};
Schedule schedule(const Fp8Gemm& g, int hook) {
  Schedule one;
  one.handful = handful_applies(g, hook);
  if (one.handful) return one;
  const Resident resident = resident_clusters();
  one.n = 1;
  one.g[0] = g;
  one.pl[0] = plan(g, resident, hook);
  const int pairs = resident.clusters[0];
  if (pairs <= 0 || g.M <= 256 || hook) return one;
  const int tile = g.epilogue == CB_FP8_SWIGLU_FP8 ? 128 : 256;
  const int width = g.epilogue == CB_FP8_SWIGLU_FP8 ? g.N / 2 : g.N;
  const int t = (g.M + 255) / 256, w = (width + tile - 1) / tile;
  const long long rounds = (static_cast<long long>(t) * w + pairs - 1) / pairs;
  // the most tiles along one axis that stay within one round less
  const long long fewer = (rounds - 1) * pairs;
  const int tk = static_cast<int>(fewer / w), fk = static_cast<int>(fewer / t);
  Schedule best = one;
  double us = WORTH_IT * one.pl[0].us;
  auto consider = [&](const Fp8Gemm& first, const Fp8Gemm& rest) {
    const Plan a = plan(first, resident, hook), b = plan(rest, resident, hook);
    if (a.us + b.us + SECOND_LAUNCH_US >= us) return;
    us = a.us + b.us + SECOND_LAUNCH_US;
    best.n = 2;
    best.g[0] = first, best.g[1] = rest;
    best.pl[0] = a, best.pl[1] = b;
  };
  if (tk > 0) consider(first_tokens(g, tk * 256), other_tokens(g, tk * 256));
  if (fk > 0) consider(first_features(g, fk * tile), other_features(g, fk * tile));
  return best;
}

}  // namespace

bool gemm_fp8_set_plan(int tokens, int split) {
  if ((tokens == 0 || tokens == 1) && split == 0) {
    g_plan.store(tokens * 8);
    return true;
  }
  if (!kernel_of(tokens, CB_FP8_STORE_F32) || split < 1 || split > 4 || (tokens == 256 && split != 1)) return false;
  g_plan.store(tokens * 8 + split);
  return true;
}

void gemm_fp8_describe(int M, int N, int K, int epilogue, char* buf, size_t len) {
  Fp8Gemm g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.epilogue = epilogue;
  const Schedule sched = schedule(g, g_plan.load());
  if (sched.handful || sched.pl[0].bt == 0) {
    snprintf(buf, len, sched.handful ? "handful" : "none");
    return;
  }
  size_t used = 0;
  for (int i = 0; i < sched.n && used < len; ++i) {
    const Fp8Gemm& p = sched.g[i];
    const Plan& pl = sched.pl[i];
    used += snprintf(buf + used, len - used, "%stokens=%d features=%d token_tile=%d split=%d clusters=%d stages=%d model_us=%.1f",
                     i ? "; " : "", p.M, epilogue == CB_FP8_SWIGLU_FP8 ? p.N / 2 : p.N, pl.bt, pl.split, pl.clusters,
                     pl.stages, pl.us);
  }
}

// One product ready to be launched.
struct Prepared {
  CUtensorMap mx, mw, mw2, ms, mc;
  Params p;
  Kernel fn;
  int ctas, cluster;
};
static cudaError_t prepare(const Fp8Gemm& g, const Plan& pl, Prepared& r) {
  const bool swiglu = g.epilogue == CB_FP8_SWIGLU_FP8;
  // (readers of a group arrive for the one n_acc further on, whose stage must have ended its previous phase)
  if (pl.bt == 0 || pl.stages <= n_acc(pl.bt)) return cudaErrorInvalidConfiguration;
  const bool tokens = pl.bt == 256;
  Params& p = r.p;
  p.g = g;
  p.width = swiglu ? g.N / 2 : g.N;
  p.tok_tiles = (g.M + pl.bt - 1) / pl.bt;
  p.units = p.tok_tiles * (swiglu ? (p.width + 127) / 128 : (p.width + 255) / 256);
  p.split = pl.split;
  p.groups = (g.K + 127) / 128;
  p.stages = pl.stages;
  p.stage_bytes = pl.stage_bytes;
  p.ring_off = pl.ring_off;
  p.out_off = pl.out_off;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, F32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  const int w_rows = swiglu && !tokens ? 64 : 128;
  bool ok = encode_tmap(&r.mx, U8, g.a, g.K, g.M, g.lda, 128, tokens ? 128 : pl.bt / 2, SW) &&
            encode_tmap(&r.ms, F32, g.a_scale, g.M, p.groups, g.ld_as * 4, tokens ? 128 : pl.bt, 1,
                        CU_TENSOR_MAP_SWIZZLE_NONE) &&
            encode_tmap(&r.mw, U8, g.b, g.K, p.width, g.ldb, 128, w_rows, SW);
  r.mw2 = r.mw;
  if (swiglu) ok = ok && encode_tmap(&r.mw2, U8, g.b2, g.K, p.width, g.ldb2, 128, w_rows, SW);
  r.mc = r.mx;
  if (tokens && swiglu) ok = ok && encode_tmap(&r.mc, U8, g.c, p.width, g.M, g.ldc, 64, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (tokens && g.epilogue == CB_FP8_STORE_BF16)
    ok = ok && encode_tmap(&r.mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.c, p.width, g.M, g.ldc * 2, 32, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B);
  if (!ok) return cudaErrorInvalidValue;
  r.fn = kernel_of(pl.bt, g.epilogue);
  r.ctas = 2 * pl.split * std::min(pl.clusters, p.units);
  r.cluster = 2 * pl.split;
  static DeviceOnce once[4][17];
  return max_dynamic_smem_once(reinterpret_cast<const void*>(r.fn), SMEM_ALLOC, once[g.epilogue][pl.bt / 16]);
}
static cudaError_t launch(const Prepared& r, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(r.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_ALLOC;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = r.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = launch_overlap_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, r.fn, r.mx, r.mw, r.mw2, r.ms, r.mc, r.p);
}

cudaError_t launch_gemm_fp8(const Fp8Gemm& g, cudaStream_t s) {
  if (g.M <= 0) return cudaSuccess;
  const Schedule sched = schedule(g, g_plan.load());
  if (sched.handful) {
    const dim3 grid((g.N + 15) / 16), block(256);
    return g.M <= 8 ? launch_chain(gemm_fp8_handful_kernel<1>, grid, block, 0, s, g)
                    : launch_chain(gemm_fp8_handful_kernel<2>, grid, block, 0, s, g);
  }
  // (both parts are prepared before one is launched: nothing is enqueued for a call that is refused)
  Prepared part[2];
  cudaError_t e = cudaSuccess;
  for (int i = 0; e == cudaSuccess && i < sched.n; ++i) e = prepare(sched.g[i], sched.pl[i], part[i]);
  for (int i = 0; e == cudaSuccess && i < sched.n; ++i) e = launch(part[i], s);
  return e;
}

}  // namespace cb
