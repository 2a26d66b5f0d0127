// Tokens drawn from rows of logits with temperature, top-k, top-p and min-p, from given random numbers.
//
//   w_i = exp((x_i - max) / t); tokens stand by falling x, equal ones by rising index.  Every filter keeps a prefix of that
//   order: the first k; of those the shortest whose mass reaches p times theirs; those with w >= min_p.  The
//   token is the first whose running kept mass exceeds u times the kept mass, along that order or by rising index.
// So a filter and the draw are the same question, "at which token does the running count or mass reach a
// target", answered exactly: weights are whole numbers of 2^-44 of the largest (before they are cut to one, off by less than 2^-28 of
// themselves, 2^-28.7 measured: the exponent (x - max) / t log2(e) is carried in two fp32 numbers), and sums of whole numbers do not depend
// on their order.  min_p is compared by logits, x >= max + t log(min_p): weights of few units say little.
//
// A row is dealt with by the 1 to 8 CTAs of a cluster, which read it from memory once and again, two or three
// times, from the second-level cache (so that two CTAs fit an SM, one working while the other waits).  Three ways, each of
// which leaves a row that it cannot settle to the next:
//   1. top-k of up to half of the cluster's threads: the k-th largest of the threads' own largest logits is a lower
//      bound for the k-th largest of all, and not many more than k tokens pass it; they are sorted and summed one by one.
//   2. all tokens: a histogram of near masses over 8192 ranges of (max - x) / t says in which range the
//      target of top-p and that of the draw lie; one pass over the exact weights sums what lies before those
//      ranges and collects their tokens, which are sorted; the exact sums show whether the ranges were the right ones.
//   3. an exact histogram of counts or masses, whose range that holds the target is cut further by the bits of x and of the
//      index until at most LIST tokens are left (flat rows, crowds of equal logits, top-k beyond 1.'s).
// A draw by rising index needs the filters' last token alone: 1. sorts what is kept once more, by index; for the others one pass over the
// exact weights sums what is kept of each 32 vectors, and the 32 that hold the target are weighed once more, token by token.
//
// Bounds: a few rows by the chain of their passes and cluster barriers (one row of 32000 with top-k: 10.2 us, by index 11.3; 64 rows of
// 64000 fp32 with top-p: 35.1 us, of these the exact pass 6.4, the merge of the near masses 5.9, their own pass 3.3, by index 44.6), many by the
// passes' instructions: 512 rows of 64000 bf16 with top-k and top-p 38.3 us, by index 41.4, 1.7 TB/s (a row 12 us on half an SM: its loads and maxima 3.9, the bound 1.5,
// collecting 3.5, sorting and sums 3.0; 1.7 rounds of rows); with top-p alone 147 us (38 us a row and SM: near masses 10, the exact
// pass 23, near 90 issue slots a logit and warp), by index 201; with temperature alone 132, by index, with one pass, 86.  512 threads, two CTAs an SM: 1024 threads and one were slower.  Rows that 1. and 2.
// leave to 3. cost 20 us more in small batches and 3 to 8 times as much in large ones: more than 512 logits within 1/256 of
// each other (spread of 64000 logits below about a quarter of the temperature), or top-k beyond 256 a CTA.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace cb {

namespace {

namespace cg = cooperative_groups;

constexpr int ST = 512;      // threads
constexpr int SW = ST / 32;
constexpr int LIST = ST;     // tokens that are sorted
constexpr int BUCKETS = 4096;
constexpr int NEAR = 8192;   // of the near masses
constexpr float REACH = 32.f;  // of (max - x) / t: exp(-31.98) is less than half of 2^-44, weight 0
constexpr int SHIFT = 44;      // the largest weight is 2^SHIFT
typedef unsigned long long u64;

// 2^30 2^(j / 32)
__constant__ uint32_t kExp2[32] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

struct SampleArgs {
  const void* logits;
  long long ld;
  int vocab;
  const float *temperature, *top_p, *min_p, *uniform;
  const int32_t* top_k;
  int32_t* out;
  int chunk;  // tokens per CTA
  int rows, wave;  // rows whose CTAs run at once
};

// What the cluster's first CTA decides for all of them.
struct Ctl {
  int bucket;   // of the level just looked at
  int count;    // tokens in it
  u64 excl;     // sum before the bucket
  u64 comp;     // the token found
  u64 incl;     // sum up to and with it
};

struct __align__(16) Smem {
  uint32_t hist[3][BUCKETS];
  u64 tot[BUCKETS];     // first CTA: inclusive sums
  u64 list[2][LIST];    // tokens that this CTA collected
  u64 warp[32];
  u64 part[6];          // this CTA's: see the uses
  uint32_t above[SW];   // bounds, a warp's each
  float near[4];
  float c_hi, c_lo;     // (64-bit floating point is slow: one thread computes these for all)
  float m_hi, m_lo;     // t log(min_p)
  Ctl ctl[2];
  int n_list[2];
  // (while no histogram is in use: a row's first vectors, and the first CTA's own)
  static constexpr int STASH = (sizeof(uint32_t) * 3 * BUCKETS + sizeof(u64) * BUCKETS) / 16;
  __device__ uint4* stash() { return reinterpret_cast<uint4*>(hist[0]); }
  __device__ u64* work() { return reinterpret_cast<u64*>(hist[1]); }
  __device__ u64* sums() { return reinterpret_cast<u64*>(hist[2]); }
};

// order of the tokens as one number: by logit, then the lower index first
__device__ __forceinline__ u64 composite(float x, int idx) {
  uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<u64>(u) << 32 | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float logit_of(u64 comp) {
  const uint32_t u = static_cast<uint32_t>(comp >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int index_of(u64 comp) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(comp)); }

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// m f for a fraction f (below 0 and NaN: 0, above 1: m), exactly, rounded down or up
__device__ __forceinline__ u64 part_of(u64 m, float f, bool up) {
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return m;
  const uint32_t bits = __float_as_uint(f), e = max(bits >> 23, 1u);
  const u64 frac = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);  // f = frac 2^(e - 150)
  const int s = 150 - static_cast<int>(e);                              // 24 to 149
  const u64 lo = m * frac, hi = __umul64hi(m, frac);                    // (m is below 2^63: hi below 2^23)
  const u64 q = s < 64 ? lo >> s | hi << (64 - s) : s < 128 ? hi >> (s - 64) : 0;
  const bool exact = s < 64 ? (lo & ((1ull << s) - 1)) == 0 : lo == 0 && (s < 128 ? (hi & ((1ull << (s - 64)) - 1)) == 0 : hi == 0);
  return q + (up && !exact);
}

template <typename T> struct Sampler {
  static constexpr int VEC = 16 / sizeof(T);

  const SampleArgs& a;
  Smem& s;
  // this CTA's tokens: 16-byte vectors as they lie in memory, the first and last perhaps with a neighbour's elements
  const T* src;      // its first token
  int off, n;        // elements before it in its vector; tokens
  int n_vec, first;  // vectors, to a multiple of 32; index of the first vector's first element
  bool inf = false;  // the largest logit is +infinity: those tokens count as 0, the others are none
  cg::cluster_group cl;
  int rank, ranks, tid, lane, warp;
  int phase = 0;
  // row
  float top, c_hi, c_lo, reach;  // largest logit, log2(e) / t in two parts, buckets per unit of max - x
  uint32_t tab;
  float floor_x = -INFINITY;  // the least logit that min_p keeps
  u64 eligible = 0; // composite of the last token that top-k keeps

  __device__ Sampler(const SampleArgs& args, Smem& sm) : a(args), s(sm), cl(cg::this_cluster()) {
    rank = cl.block_rank();
    ranks = cl.num_blocks();
    tid = threadIdx.x;
    lane = tid & 31;
    warp = tid >> 5;
    tab = kExp2[lane];
  }

  // Weight of a token, 2^SHIFT for the largest (top is finite).  All lanes of a warp take part.
  __device__ __forceinline__ u64 weight(float x) const {
    const float d = x - top;
    // the difference's own rounding (two-sum), then the exponent in two parts
    const float b = d - x, de = (x - (d - b)) + (-top - b);
    const float e = d * c_hi, el = fmaf(d, c_hi, -e) + fmaf(d, c_lo, de * c_hi);
    int k;
    const uint32_t m = exp2_of(e, el, &k);
    return (static_cast<u64>(m) << (SHIFT - 30)) >> -k;
  }
  // 2^(e + el) as m 2^(k - 30), m of 31 bits.  All lanes of a warp take part.
  __device__ __forceinline__ uint32_t exp2_of(float e, float el, int* whole) const {
    // e = k / 32 + r: 2^(k / 32) from the table, 2^r - 1 by its series (|r ln 2| < 0.011: terms to the fourth); below
    // 2^-47 every 32 bits shifted that far are 0, whatever r is
    const float ec = fmaxf(e, -47.f), km = fmaf(ec, 32.f, 12582912.f);
    const int k = __float_as_int(km) - 0x4b400000;
    const float r = fmaf(km - 12582912.f, -0.03125f, ec) + el;
    const float y = fmaf(r, 0.693147182f, r * -1.90465421e-9f);
    const float p = fmaf(y * y, fmaf(y, fmaf(y, 1.f / 24.f, 1.f / 6.f), 0.5f), y);
    const int t = static_cast<int>(__shfl_sync(0xffffffffu, tab, k & 31));
    *whole = k >> 5;
    return static_cast<uint32_t>(t + __mulhi(t, __float2int_rn(p * 4294967296.f)));
  }
  // log(x) of 2^-46 <= x <= 1 in two parts, as exactly as weights are: an estimate, and what its exponential is off by.  All lanes of a
  // warp take part.
  __device__ __forceinline__ float2 log_of(float x) const {
    const float l = logf(x), e = l * 1.44269502f;
    int k;
    const uint32_t m = exp2_of(e, fmaf(l, 1.44269502f, -e) + l * 1.92596299e-8f, &k);
    const uint32_t want = static_cast<uint32_t>(x * __int_as_float((157 - k) << 23));  // x 2^(30 - k), a whole number
    return make_float2(l, static_cast<float>(static_cast<int>(want - m)) / static_cast<float>(m));
  }
  // (max - x) / t in buckets, at most the last one; that is 2^-46 and weighs nothing
  __device__ __forceinline__ float fall(float x) const { return fminf((top - x) * reach, static_cast<float>(BUCKETS - 1)); }
  __device__ __forceinline__ int bucket0(float x) const {  // the nearest whole number, from a float's last bits
    return __float_as_int(fall(x) + 8388608.f) & (BUCKETS - 1);
  }

  // vector v, what is not a token (a NaN too) as -infinity
  __device__ __forceinline__ uint4 raw_vector(int v) const {
    const int at = v * VEC - off;
    if (at >= 0 && at + VEC <= n) return __ldg(reinterpret_cast<const uint4*>(src + at));
    T x[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = at + i >= 0 && at + i < n ? src[at + i] : from_f<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(x);
  }
  __device__ __forceinline__ uint4 cleaned(uint4 e) const {
    uint32_t w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
        const uint32_t good = __heq2_mask(h, h);
        w[i] = (w[i] & good) | (0xff80ff80u & ~good);
      } else {
        const float x = __uint_as_float(w[i]);
        w[i] = x == x ? w[i] : 0xff800000u;
      }
    }
    if (inf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 2)
          w[i] = ((w[i] & 0xffffu) == 0x7f80u ? 0u : 0xff80u) | (w[i] >> 16 == 0x7f80u ? 0u : 0xff800000u);
        else
          w[i] = w[i] == 0x7f800000u ? 0u : 0xff800000u;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the largest number of a cleaned vector
  static __device__ __forceinline__ float largest(uint4 e) {
    const uint32_t w[4] = {e.x, e.y, e.z, e.w};
    if (sizeof(T) == 2) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
      const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
      return fmaxf(f.x, f.y);
    }
    return fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])), fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
  }
  static __device__ __forceinline__ float element(uint4 e, int i) {
    const uint32_t w[4] = {e.x, e.y, e.z, e.w};
    if (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    return __uint_as_float(w[i % 4]);
  }
  __device__ __forceinline__ float near_fall(float x) const {
    return fminf((top - x) * (reach * (NEAR / BUCKETS)), static_cast<float>(NEAR - 1));
  }
  __device__ __forceinline__ int near_bucket(float x) const { return __float_as_int(near_fall(x) + 8388608.f) & (NEAR - 1); }

  // f(logit, index) for all of this CTA's tokens (and some places of -infinity), whole warps together: f may use
  // warp-wide operations.
  template <typename F> __device__ __forceinline__ void each(F f) const {
    each([&](float x, int idx, int) { f(x, idx); }, [](int) {});
  }
  // f(logit, index, place in its vector), and g(index of its first element) after each vector
  template <typename F, typename G> __device__ __forceinline__ void each(F f, G g) const {
    uint4 next = {};
    if (tid < n_vec) next = raw_vector(tid);
#pragma unroll 1
    for (int v = tid; v < n_vec; v += ST) {  // (n_vec is a multiple of 32)
      const uint4 e = cleaned(next);
      if (v + ST < n_vec) next = raw_vector(v + ST);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f(element(e, i), first + v * VEC + i, i);
      g(first + v * VEC);
    }
  }
  // f(vector, its number) over this CTA's tokens from vector v0 on, some loads ahead
  template <typename F> __device__ __forceinline__ void vectors(int v0, F f) const {
    constexpr int BATCH = 8;
#pragma unroll 1
    for (v0 += tid; v0 < n_vec; v0 += BATCH * ST) {
      uint4 e[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (v0 + j * ST < n_vec) e[j] = raw_vector(v0 + j * ST);
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (v0 + j * ST < n_vec) f(cleaned(e[j]), v0 + j * ST);
    }
  }
  // The tokens of at least `least` into list 0, by the threads whose largest is one; the first vectors are in the stash.
  __device__ __forceinline__ void collect_from(float least, float own) {
    if (own < least) return;
    uint32_t some = 0;  // this thread's vectors (at most 32) that hold one
#pragma unroll 4
    for (int v = tid; v < min(n_vec, Smem::STASH); v += ST)
      if (largest(s.stash()[v]) >= least) some |= 1u << v / ST;
    vectors(Smem::STASH, [&](uint4 e, int v) {
      if (largest(e) >= least) some |= 1u << v / ST;
    });
#pragma unroll 1
    while (some) {
      const int v = tid + (__ffs(some) - 1) * ST;
      some &= some - 1;
      const uint4 e = cleaned(raw_vector(v));
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) hits |= (element(e, i) >= least ? 1u : 0u) << i;
      collect_hits(0, hits, first + v * VEC);
    }
  }
  // The tokens idx + i of the bits i of a mask into a list (few do: one small loop, as the kernel's time on few rows is that of
  // fetching its instructions).
  __device__ __forceinline__ void collect_hits(int which, uint32_t hits, int idx) {
#pragma unroll 1
    while (hits) {
      const int at = idx + __ffs(hits) - 1;
      hits &= hits - 1;
      if (static_cast<unsigned>(at - first - off) >= static_cast<unsigned>(n)) continue;  // (a neighbour's element)
      const float x = to_f(src[at - first - off]);
      collect(which, inf ? 0.f : x, at);
    }
  }

  // The draw by rising index over the tokens from `cut` on (as composites) that min_p keeps: the masses of the warps' 32 vectors,
  // one after the other in memory, then the tokens of those that hold the target of the mass, reach(mass).
  template <typename R> __device__ __forceinline__ void draw_by_id(u64 cut, R reach, int32_t* out) {
    auto kept = [&](float x, int idx) {
      const u64 w = weight(x);
      return composite(x, idx) >= cut && x >= floor_x ? w : 0;
    };
    u64* masses = s.sums();
    __syncthreads();
    masses[tid] = 0;
    __syncthreads();
    u64 sum = 0;
    each([&](float x, int idx, int) { sum += kept(x, idx); },
         [&](int idx) {
           sum = warp_sum64(sum);
           if (lane == 0) masses[(idx - first) / (32 * VEC)] = sum;
           sum = 0;
         });
    __syncthreads();
    const u64 mine = masses[tid], incl = block_scan(mine);
    if (tid == ST - 1) s.part[4] = incl;  // (part[0] may still be on its way to another CTA)
    meet();
    const u64 each_cta = of_each(&s.part[4], static_cast<u64>(0));
    const u64 total = warp_sum64(each_cta), before = warp_sum64(lane < rank ? each_cta : 0);
    const u64 want = reach(total);  // (at least 1: the largest logit's token is kept)
    if (before < want && want - before <= __shfl_sync(0xffffffffu, each_cta, rank)) {
      const u64 target = want - before;
      if (incl - mine < target && target <= incl) {
        s.part[5] = target - (incl - mine);
        s.n_list[1] = tid;
      }
      __syncthreads();
      if (warp == 0) {
        const int v = s.n_list[1] * 32 + lane;
        const uint4 e = cleaned(raw_vector(v));
        u64 w[VEC], own = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) own += w[i] = kept(element(e, i), first + v * VEC + i);
        u64 run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += y;
        }
        run -= own;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (run < s.part[5] && s.part[5] <= run + w[i]) *out = first + v * VEC + i;
          run += w[i];
        }
      }
    }
    meet();
  }

  __device__ __forceinline__ void meet() {  // all CTAs of the row
    if (ranks == 1)
      __syncthreads();
    else
      cl.sync();
  }

  __device__ __forceinline__ Ctl decide() {  // what the first CTA wrote into ctl[phase], for everyone
    meet();
    const Ctl c = *cl.map_shared_rank(&s.ctl[phase], 0);
    phase ^= 1;
    return c;
  }

  // Histogram over the cluster: tokens for which bucket() is not negative, by count or mass; the first CTA gets the
  // inclusive sums in tot.
  template <bool MASS, typename B> __device__ __forceinline__ void histogram(B bucket) {
    for (int i = tid; i < BUCKETS * (MASS ? 3 : 1); i += ST) s.hist[0][i] = 0;
    __syncthreads();
    u64 over = 0;
    each([&](float x, int idx) {
      const int b = x > -INFINITY ? bucket(x, idx) : -1;
      // tokens of one value come in crowds (bf16, flat rows): one lane adds for a warp that agrees
      const u64 w = MASS ? weight(x) : 1;
      const bool add = b >= 0 && w > 0;
      if (MASS && add && x >= floor_x) over += w;
      const unsigned who = __ballot_sync(0xffffffffu, add);
      if (who == 0) return;
      const int b0 = __shfl_sync(0xffffffffu, b, __ffs(who) - 1);
      if (__all_sync(0xffffffffu, !add || b == b0)) {
        if (MASS) {
          const uint32_t p0 = __reduce_add_sync(0xffffffffu, add ? static_cast<uint32_t>(w) & 0x7fffu : 0u);
          const uint32_t p1 = __reduce_add_sync(0xffffffffu, add ? static_cast<uint32_t>(w >> 15) & 0x7fffu : 0u);
          const uint32_t p2 = __reduce_add_sync(0xffffffffu, add ? static_cast<uint32_t>(w >> 30) : 0u);
          if (lane == 0) {
            atomicAdd(&s.hist[0][b0], p0);
            atomicAdd(&s.hist[1][b0], p1);
            atomicAdd(&s.hist[2][b0], p2);
          }
        } else if (lane == 0) {
          atomicAdd(&s.hist[0][b0], static_cast<uint32_t>(__popc(who)));
        }
      } else if (add) {
        if (MASS) {
          atomicAdd(&s.hist[0][b], static_cast<uint32_t>(w) & 0x7fffu);
          atomicAdd(&s.hist[1][b], static_cast<uint32_t>(w >> 15) & 0x7fffu);
          if (w >> 30) atomicAdd(&s.hist[2][b], static_cast<uint32_t>(w >> 30));
        } else {
          atomicAdd(&s.hist[0][b], 1u);
        }
      }
    });
    if (MASS) {
      over = warp_sum64(over);
      if (lane == 0) s.warp[warp] = over;
      __syncthreads();
      if (warp == 0) {
        over = warp_sum64(lane < SW ? s.warp[lane] : 0);
        if (lane == 0) s.part[1] = over;
      }
    }
    meet();
    // each CTA sums a slice of the buckets over the cluster
    const int slice = BUCKETS / ranks;
    u64* tot = cl.map_shared_rank(s.tot, 0);
    for (int i = rank * slice + tid; i < (rank + 1) * slice; i += ST) {
      u64 sum = 0;
      for (int r = 0; r < ranks; ++r) {
        const uint32_t* h = cl.map_shared_rank(&s.hist[0][0], r);
        sum += h[i];
        if (MASS) sum += (static_cast<u64>(h[BUCKETS + i]) << 15) + (static_cast<u64>(h[2 * BUCKETS + i]) << 30);
      }
      tot[i] = sum;
    }
    meet();
    if (rank == 0) {
      running_sums();
    }
  }

  __device__ __forceinline__ void running_sums() {  // first CTA: tot
    constexpr int EACH = BUCKETS / ST;
    u64 x[EACH], sum = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) x[i] = sum += s.tot[EACH * tid + i];
    const u64 before = block_scan(sum) - sum;
#pragma unroll
    for (int i = 0; i < EACH; ++i) s.tot[EACH * tid + i] = x[i] + before;
    __syncthreads();
  }

  template <typename V> __device__ __forceinline__ V block_scan(V v) {  // inclusive, one value a thread
    V* warps = reinterpret_cast<V*>(s.warp);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    // (every warp sums the ones before it)
    V w = lane < warp ? warps[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    __syncthreads();
    return v + w;
  }

  // first CTA: the bucket in which the running sum reaches target
  __device__ __forceinline__ void find_bucket(u64 target) {
    for (int b = tid; b < BUCKETS; b += ST) {
      const u64 incl = s.tot[b], excl = b ? s.tot[b - 1] : 0;
      if (excl < target && target <= incl) {
        s.ctl[phase].bucket = b;
        s.ctl[phase].excl = excl;
      }
    }
  }

  // A token into one of this CTA's lists (the count goes on where the list is full).
  __device__ __forceinline__ void collect(int which, float x, int idx) {
    const int at = atomicAdd(&s.n_list[which], 1);
    if (at < LIST) s.list[which][at] = composite(x, idx);
  }
  // One value of each CTA (a reading from another takes long: each lane reads one), lane r that of CTA r; `rest` beyond
  template <typename V> __device__ __forceinline__ V of_each(V* mine, V rest) const {
    return lane < ranks ? *cl.map_shared_rank(mine, lane) : rest;
  }
  // After the CTAs have collected and the cluster has met: tokens in all lists.
  __device__ __forceinline__ int collected(int which) const {
    return __reduce_add_sync(0xffffffffu, of_each(&s.n_list[which], 0));
  }
  // first CTA: the i-th token of all CTAs' lists (i below their number)
  __device__ __forceinline__ u64 token_of(int which, int at, bool in) const {
    int end = of_each(&s.n_list[which], 0);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    int r = 0, before = 0;  // the list that holds it
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const int e = __shfl_sync(0xffffffffu, end, i);
      if (at >= e) {
        r = i + 1;
        before = e;
      }
    }
    return in ? cl.map_shared_rank(&s.list[which][0], r)[at - before] : 0;
  }
  // first CTA: its threads' first n numbers (at most LIST), largest first; thread i gets the i-th
  __device__ __forceinline__ u64 sorted(u64 v, int n) {
    u64* work = s.work();
    if (n <= ST / 2) {  // each token's place counted: two threads a token, half of the others each (fewer steps than a sort's)
      constexpr int HALF = ST / 2;
      const int i = tid & (HALF - 1), mid = (n + 1) / 2;
      if (tid < HALF) work[tid] = tid < n ? v : 0;
      __syncthreads();
      const u64 mine = work[i];
      int place = 0;
      if (i < n) {
        const int j0 = tid < HALF ? 0 : mid, j1 = tid < HALF ? mid : n;
#pragma unroll 4
        for (int j = j0; j < j1; ++j) place += work[j] > mine;
      }
      int* upper = reinterpret_cast<int*>(work + 2 * HALF);
      if (tid >= HALF) upper[i] = place;
      __syncthreads();
      u64* out = work + HALF;
      if (tid < n) out[place + upper[i]] = mine;
      __syncthreads();
      v = tid < n ? out[tid] : 0;
      __syncthreads();
      return v;
    }
    int size = 32;
    while (size < n) size <<= 1;
    // (the warps that hold tokens only, with a barrier of their own)
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(size) : "memory"); };
    for (int k = 2; tid < size && k <= size; k <<= 1) {
      for (int j = k >> 1; j > 0; j >>= 1) {
        u64 o;
        if (j >= 32) {
          meet();
          work[tid] = v;
          meet();
          o = work[tid ^ j];
        } else {
          o = __shfl_xor_sync(0xffffffffu, v, j);
        }
        const bool keep_max = ((tid & k) == 0) == ((tid & j) == 0);
        v = keep_max ? max(v, o) : min(v, o);
      }
    }
    __syncthreads();
    return v;
  }

  // The tokens for which take() holds into the lists 0; their number for everyone.
  template <typename P> __device__ __forceinline__ int gather(P take) {
    if (tid == 0) s.n_list[0] = 0;
    __syncthreads();
    each([&](float x, int idx) {
      if (x > -INFINITY && take(x, idx)) collect(0, x, idx);
    });
    meet();
    return collected(0);
  }

  // Token at which the running count (of live tokens) or mass reaches target, from the histogram in tot (first CTA) of
  // bucket0; all CTAs return it, and the sum up to and with it.  LIVE: whether a token counts.
  template <bool MASS, typename L> __device__ __forceinline__ Ctl select(u64 target, L live, bool* refined) {
    if (rank == 0) find_bucket(target);
    Ctl c = decide();
    const int b0 = c.bucket;
    u64 excl = c.excl;
    // the tokens still in question agree in bucket0 and in the leading bits of their composite
    int bits = 0;
    u64 lead = 0;
    for (;;) {
      auto in = [&](float x, int idx) {
        return live(x, idx) && bucket0(x) == b0 && (bits == 0 || composite(x, idx) >> (64 - bits) == lead);
      };
      const int n = gather(in);
      if (n <= LIST) {
        if (rank == 0) {
          const u64 t = sorted(token_of(0, tid, tid < n), n);
          const u64 mine = MASS ? weight(logit_of(t)) : 1;  // (all lanes)
          const u64 w = tid < n ? mine : 0;
          const u64 incl = excl + block_scan(w);
          if (tid < n && (incl - w < target && target <= incl)) {
            s.ctl[phase].comp = t;
            s.ctl[phase].incl = incl;
          }
          __syncthreads();
        }
        return decide();
      }
      *refined = true;
      // the next bits: 8 of the logit at a time, then the upper 11 of the index's 18 (the 14 before them are ones)
      const int step = bits < 32 ? 8 : 11, at = bits < 32 ? bits : 46;
      histogram<MASS>([&](float x, int idx) {
        const u64 comp = composite(x, idx);
        return in(x, idx) ? static_cast<int>((1u << step) - 1 - (static_cast<uint32_t>(comp >> (64 - at - step)) & ((1u << step) - 1))) : -1;
      });
      if (rank == 0) find_bucket(target - excl);
      c = decide();
      excl += c.excl;
      const u64 digit = static_cast<u64>((1 << step) - 1 - c.bucket);
      if (bits == 32) lead = lead << 14 | 0x3fff;
      lead = lead << step | digit;
      bits = at + step;
    }
  }
};

// BY_ID: the draw goes by rising index.
template <typename T, bool BY_ID> __global__ void __launch_bounds__(ST, 2) sample_kernel(SampleArgs a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  Sampler<T> z(a, s);
  constexpr int VEC = Sampler<T>::VEC;
  const int row = blockIdx.x / z.ranks, tid = z.tid, lane = z.lane, warp = z.warp;
  const int i0 = min(a.vocab, z.rank * a.chunk), n = min(a.vocab, i0 + a.chunk) - i0;
  z.src = static_cast<const T*>(a.logits) + static_cast<long long>(row) * a.ld + i0;
  z.off = static_cast<int>(reinterpret_cast<uintptr_t>(z.src) & 15) / sizeof(T);
  z.n = n;
  z.n_vec = n > 0 ? ((z.off + n + VEC - 1) / VEC + 31) / 32 * 32 : 0;
  z.first = i0 - z.off;
  // the row that takes this one's place on the SM, on its way into the second-level cache meanwhile
  if (tid == 0 && row + a.wave < a.rows && n * sizeof(T) >= 32) {
    const uintptr_t p = (reinterpret_cast<uintptr_t>(z.src + static_cast<long long>(a.wave) * a.ld) + 15) & ~static_cast<uintptr_t>(15);
    const uint32_t bytes = (static_cast<uint32_t>(n) * sizeof(T) - 15) / 16 * 16;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
  }
  float t = a.temperature ? a.temperature[row] : 1.f;
  int k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
  const float u = a.uniform[row];
  if (!(t > 0.f) || top_p <= 0.f) k = 1;  // (top_p of 0 keeps the first token: 64 rows of 64000 fp32 9.5 us, by the near masses 69)
  if (k <= 0 || k >= a.vocab) k = a.vocab;
  if (tid == ST - 1) {
    const double c = 1.4426950408889634 / static_cast<double>(fminf(fmaxf(t, 1e-20f), 1e20f));
    s.c_hi = static_cast<float>(c);
    s.c_lo = static_cast<float>(c - static_cast<double>(s.c_hi));
  }
  // w >= min_p is x >= max + t log(min_p): by logits, as weights of few units of 2^-44 say little (and those below 2^-45 nothing)
  const bool with_m = min_p >= 0x1p-45f;
  if (with_m && warp == SW - 1) {
    const float2 l = z.log_of(fminf(min_p, 1.f));
    const float ts = fminf(fmaxf(t, 1e-20f), 1e20f), hi = ts * l.x;
    if (lane == 0) {
      s.m_hi = hi;
      s.m_lo = fmaf(ts, l.x, -hi) + ts * l.y;
    }
  }
  float own = -INFINITY;  // this thread's largest
  const bool keep = k > 1 && k <= z.ranks * (ST / 2) && k < a.vocab;  // (way 1)
  z.vectors(0, [&](uint4 e, int v) {
    own = fmaxf(own, z.largest(e));
    if (keep && v < Smem::STASH) s.stash()[v] = e;
  });
  uint32_t key = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(composite(own, 0) >> 32));
  if (lane == 0) s.warp[warp] = key;
  __syncthreads();
  if (warp == 0) {
    key = __reduce_max_sync(0xffffffffu, lane < SW ? static_cast<uint32_t>(s.warp[lane]) : 0u);
    if (lane == 0) s.part[0] = key;
  }
  z.meet();
  key = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(z.of_each(&s.part[0], 0ull)));
  z.top = logit_of(static_cast<u64>(key) << 32);
  // (no CTA leaves while another reads its shared memory)
  if (!(z.top > -INFINITY)) {
    if (z.rank == 0 && tid == 0) a.out[row] = -1;
    z.meet();
    return;
  }
  if (z.top == INFINITY) {  // its tokens are equally likely, the others are none
    z.inf = true;
    z.top = 0.f;
    own = own == INFINITY ? 0.f : -INFINITY;
  }
  const uint32_t own_key = static_cast<uint32_t>(composite(own, 0) >> 32);
  if (k == 1) {  // the largest logit's first token
    unsigned at = 0xffffffffu;
    z.each([&](float x, int idx) {
      if (x == z.top) at = min(at, static_cast<unsigned>(idx));
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.warp[warp] = at;
    __syncthreads();
    if (warp == 0) {
      at = __reduce_min_sync(0xffffffffu, lane < SW ? static_cast<unsigned>(s.warp[lane]) : 0xffffffffu);
      if (lane == 0) s.part[1] = at;
    }
    z.meet();
    at = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(z.of_each(&s.part[1], 0xffffffffull)));
    if (z.rank == 0 && tid == 0) a.out[row] = static_cast<int>(at);
    z.meet();
    return;
  }

  t = fminf(fmaxf(t, 1e-20f), 1e20f);
  z.c_hi = s.c_hi;
  z.c_lo = s.c_lo;
  z.reach = BUCKETS / REACH / t;
  if (with_m) {  // the smallest number not below max + t log(min_p): their sum (two-sum), and what it left out, rounded up
    const float f = z.top + s.m_hi, b = f - z.top;
    z.floor_x = __fadd_ru(f, (z.top - (f - b)) + (s.m_hi - b) + s.m_lo);
  }
  // targets of a mass m: the smallest whole numbers not below top_p m, and above u m
  auto reach_p = [&](u64 m) { return top_p < 1.f ? max(1ull, part_of(m, top_p, true)) : m; };
  auto reach_u = [&](u64 m) { return min(m, part_of(m, u, false) + 1); };
  // first CTA, list 0 sorted: the token of a row whose first k tokens are in it
  auto settle = [&](int n) {
    const u64 tok = z.sorted(z.token_of(0, tid, tid < n), n);
    const u64 w = z.weight(logit_of(tok));  // (all lanes)
    const u64 mine = tid < k && tid < n ? w : 0;
    u64* sums = s.sums();
    const u64 incl = z.block_scan(mine);
    sums[tid] = incl;
    __syncthreads();
    const u64 pm = reach_p(sums[ST - 1]);
    // kept mass: of the shorter prefix
    if (mine && incl - mine < pm && pm <= incl) s.part[2] = incl;
    const int over = __syncthreads_count(mine && logit_of(tok) >= z.floor_x);
    const u64 mass = min(s.part[2], sums[over - 1]), want = reach_u(mass);
    if (!BY_ID) {
      if (mine && incl - mine < want && want <= incl) a.out[row] = index_of(tok);
      return;
    }
    // the kept tokens by rising index, their weights by their places in the order
    const bool kept = mine && incl <= mass;
    const int n_kept = __syncthreads_count(kept);
    s.tot[tid] = mine;
    const u64 at = z.sorted(kept ? tok << 32 | static_cast<unsigned>(tid) : 0, n_kept);
    const u64 here = tid < n_kept ? s.tot[static_cast<uint32_t>(at)] : 0, run = z.block_scan(here);
    if (here && run - here < want && want <= run) a.out[row] = index_of(at >> 32);
  };

  bool refined = false;
  auto all = [](float, int) { return true; };
  if (k < a.vocab) {
    if (keep) {
      // k / ranks of the threads' largest in each CTA, the least of these over the CTAs: at least k tokens pass it.
      // Each warp sorts its threads' and names the one that its share of k reaches; of these 16 the largest that
      // enough threads pass (all but the least may be too large).
      const int each_k = (k + z.ranks - 1) / z.ranks, in_warp = (each_k + SW - 1) / SW;
      uint32_t x = own_key;
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) {
          const uint32_t o = __shfl_xor_sync(0xffffffffu, x, j);
          x = ((lane & size) == 0 || size == 32) == ((lane & j) == 0) ? max(x, o) : min(x, o);
        }
      if (lane == in_warp - 1) s.above[warp] = x;
      __syncthreads();
      x = s.above[lane & (SW - 1)];
#pragma unroll
      for (int size = 2; size <= SW; size <<= 1)
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) {
          const uint32_t o = __shfl_xor_sync(0xffffffffu, x, j);
          x = ((lane & size) == 0 || size == SW) == ((lane & j) == 0) ? max(x, o) : min(x, o);
        }
      int lo = 0, hi = SW - 1;
#pragma unroll
      for (int i = 1; i < SW; i <<= 1) {
        const int mid = (lo + hi) >> 1;
        const bool enough = __syncthreads_count(own_key >= __shfl_sync(0xffffffffu, x, mid)) >= each_k;
        hi = enough ? mid : hi;
        lo = enough ? lo : min(mid + 1, hi);
      }
      uint32_t bound = __shfl_sync(0xffffffffu, x, hi);
      if (tid == 0) s.part[1] = bound;
      z.meet();
      bound = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(z.of_each(&s.part[1], 0xffffffffull)));
      // (at least: a number, and of a weight, exp(-33) being none; a row masked by its type's lowest value has its few tokens)
      const float least = fmaxf(logit_of(static_cast<u64>(max(bound, 0x00800000u)) << 32), z.top - 33.f * t);
      if (tid == 0) s.n_list[0] = 0;
      __syncthreads();
      z.collect_from(least, own);
      z.meet();
      const int n_list = z.collected(0);
      if (n_list <= LIST) {
        if (z.rank == 0) settle(n_list);
        z.meet();
        return;
      }
    }
    z.template histogram<false>([&](float x, int) { return z.bucket0(x); });
    // the bucket of the k-th token; the last one's tokens weigh nothing
    if (z.rank == 0) {
      if (tid == 0) {
        s.ctl[z.phase].bucket = BUCKETS - 1;
        s.ctl[z.phase].excl = 0;
      }
      __syncthreads();
      z.find_bucket(k);
      __syncthreads();
    }
    if (z.decide().bucket < BUCKETS - 1) {
      const u64 last = z.template select<false>(k, all, &refined).comp;
      if (k <= LIST) {  // the first CTA has all that counts
        z.gather([&](float x, int idx) { return composite(x, idx) >= last; });
        if (z.rank == 0) settle(k);
        z.meet();
        return;
      }
      z.eligible = last;
    }
  }

  const u64 eligible = z.eligible;
  auto live = [&](float x, int idx) { return eligible == 0 || composite(x, idx) >= eligible; };
  if (BY_ID && !(top_p < 1.f)) {  // (nothing to find first)
    z.draw_by_id(eligible, reach_u, a.out + row);
    return;
  }
  if (eligible == 0) {
    // near masses: each bucket's in 2^-18 of the weight at its middle (a weight changes by 1/256 over a bucket: two terms of
    // its series).  More than 16000 tokens of a CTA in one bucket pass 32 bits: such a row goes the third way.
    for (int i = tid; i < NEAR; i += ST) s.hist[0][i] = 0;
    if (tid < 2) s.n_list[tid] = 0;
    __syncthreads();
    constexpr float STEP = REACH / NEAR, UNIT = 1 << 18;
    z.each([&](float x, int) {
      const float y = z.near_fall(x), r = y + 8388608.f, f = y - (r - 8388608.f);
      const float v = fmaf(f, fmaf(f, 0.5f * UNIT * STEP * STEP, -UNIT * STEP), UNIT + 8388608.f);
      if (y < NEAR - 1.5f) atomicAdd(&s.hist[0][__float_as_int(r) & (NEAR - 1)], __float_as_uint(v) - 0x4b000000u);
    });
    z.meet();
    {  // each CTA sums a slice over the cluster, into the first one's tot
      const int slice = NEAR / z.ranks;
      float* tot = reinterpret_cast<float*>(z.cl.map_shared_rank(s.tot, 0));
      for (int b = z.rank * slice + tid; b < (z.rank + 1) * slice; b += ST) {
        uint32_t h[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) h[r] = r < z.ranks ? z.cl.map_shared_rank(&s.hist[0][0], r)[b] : 0;
        float m = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) m += static_cast<float>(h[r]);
        tot[b] = m * (1.f / UNIT) * exp2f(static_cast<float>(b) * (-STEP * 1.44269504f));
      }
    }
    z.meet();
    if (z.rank == 0) {
      // running masses of this thread's buckets, 1 for the largest logit's token
      constexpr int EACH = NEAR / ST;
      auto middle = [&](int i) { return exp2f(static_cast<float>(EACH * tid + i) * (-STEP * 1.44269504f)); };
      float m[EACH], sum = 0.f;
#pragma unroll
      for (int i = 0; i < EACH; ++i) m[i] = sum += reinterpret_cast<const float*>(s.tot)[EACH * tid + i];
      const float before = z.block_scan(sum) - sum;
      const float last_p = -logf(fminf(min_p, 1.f)) / STEP;  // min_p's own place
      const int at_m = with_m ? static_cast<int>(fminf(last_p + 0.5f, NEAR - 1.f)) : NEAR - 1;
      if (tid == 0) {
        s.ctl[z.phase] = {0, 0, NEAR - 1, 0, NEAR - 1};  // first and last range of the draw (bucket, excl), of top_p (count, incl)
        s.near[1] = INFINITY;
        s.near[3] = 0.f;
      }
      if (tid == ST - 1) s.near[0] = before + sum;
      __syncthreads();
      // top_p's range, and the mass up to and with its last token: as if the range's tokens all weighed the same.  Near masses
      // are off by some 2^-20: where a target lies that near to a border, two ranges stand for one (else about one row
      // in 4000 went the third way, 20 us more).
      const float near_p = top_p * s.near[0], room = s.near[0] * 0x1p-19f;
      const float above_p = fminf(near_p + room, 0.5f * (near_p + s.near[0]));  // (targets below the end stay below it)
      float excl = before;
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const float incl = before + m[i];
        if (top_p < 1.f && excl < near_p && near_p <= incl) {
          const float w = middle(i);
          s.near[1] = excl + ceilf((near_p - excl) / w) * w;
          s.near[3] = w;
        }
        if (excl < near_p - room && near_p - room <= incl) s.ctl[z.phase].count = EACH * tid + i;
        if (excl < above_p && above_p <= incl) s.ctl[z.phase].incl = EACH * tid + i;
        if (EACH * tid + i == at_m) s.near[2] = excl + fminf(last_p + 0.5f - static_cast<float>(at_m), 1.f) * (incl - excl);
        excl = incl;
      }
      __syncthreads();
      if (!BY_ID) {
      // (the mass kept is known to a token at its end, and no token before weighs less)
      const bool p_ends = s.near[1] <= s.near[2];
      const float near_u = u * (p_ends ? s.near[1] : s.near[2]), room_u = room + (p_ends ? s.near[3] : with_m ? fminf(min_p, 1.f) : 0.f);
      const float above_u = fminf(near_u + room_u, 0.5f * (near_u + s.near[0]));
      excl = before;
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const float incl = before + m[i];
        if (excl <= near_u - room_u && near_u - room_u < incl) s.ctl[z.phase].bucket = EACH * tid + i;
        if (excl <= above_u && above_u < incl) s.ctl[z.phase].excl = EACH * tid + i;
        excl = incl;
      }
      __syncthreads();
      }
    }
    const Ctl guess = z.decide();
    const bool with_p = top_p < 1.f;
    // (not the last range, which has the tokens of no weight and what is none)
    int bp = min(guess.count, NEAR - 2), bu = min(guess.bucket, NEAR - 2);
    // ranges after the first: none where the last would lie before it (they come from fp32 sums, whose rounding may turn neighbours round; the
    // exact sums show what was missed)
    unsigned more_p = max(min(static_cast<int>(guess.incl), NEAR - 2) - bp, 0), more_u = max(min(static_cast<int>(guess.excl), NEAR - 2) - bu, 0);
    if (BY_ID) bu = bp, more_u = more_p;
    const bool one = bp <= bu + static_cast<int>(more_u);  // both are in the same ranges
    if (with_p && one) {
      more_u = max(bp + more_p, bu + more_u) - min(bp, bu);
      bp = bu = min(bp, bu);
      more_p = more_u;
    }
    // exact sums: all, before bp, before bu, over min_p; and the tokens of the two ranges
    u64 sum[4] = {};
    uint32_t hits[2] = {};
    auto exact = [&](auto with_top_p, auto with_min_p) {
      constexpr bool p_on = decltype(with_top_p)::value, m_on = decltype(with_min_p)::value;
      z.each([&](float x, int, int i) {
        const u64 w = z.weight(x);
        const int b = z.near_bucket(x);
        sum[0] += w;
        if (p_on) sum[1] += b < bp ? w : 0;
        sum[2] += b < bu ? w : 0;
        if (m_on) sum[3] += x >= z.floor_x ? w : 0;
        hits[0] |= (static_cast<unsigned>(b - bu) <= more_u ? 1u : 0u) << i;
        if (p_on) hits[1] |= (static_cast<unsigned>(b - bp) <= more_p ? 1u : 0u) << i;
      }, [&](int idx) {
        if (p_on && one) hits[1] = 0;
        if (hits[0] | hits[1]) {
          z.collect_hits(0, hits[0], idx);
          if (p_on) z.collect_hits(1, hits[1], idx);
          hits[0] = hits[1] = 0;
        }
      });
      if (!m_on) sum[3] = sum[0];
    };
    typedef std::integral_constant<bool, true> On;
    typedef std::integral_constant<bool, false> Off;
    if (BY_ID || with_p)
      with_m ? exact(On(), On()) : exact(On(), Off());
    else
      with_m ? exact(Off(), On()) : exact(Off(), Off());
    u64* scratch = s.sums();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 v = warp_sum64(sum[i]);
      if (lane == 0) scratch[i * 32 + warp] = v;
    }
    __syncthreads();
    if (warp < 4) {
      const u64 v = warp_sum64(lane < SW ? scratch[warp * 32 + lane] : 0);
      if (lane == 0) s.part[1 + warp] = v;
    }
    z.meet();
    const int n_u = z.collected(0), n_p = one ? n_u : z.collected(1);
    // (every CTA comes to the same result, the first one's below)
    if (z.rank == 0) {
      if (tid == 0) s.ctl[z.phase].count = 0;  // settled
      // lane 8 i + r: sum i of CTA r
      u64 total[4], v = (lane & 7) < z.ranks ? z.cl.map_shared_rank(&s.part[1], lane & 7)[lane >> 3] : 0;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) total[i] = __shfl_sync(0xffffffffu, v, 8 * i);
      u64 mass = total[3];  // what min_p keeps
      const u64 pm = reach_p(total[0]);
      const bool need_p = with_p && pm <= mass, two = need_p && !one;
      const int n = n_u + (two ? n_p : 0);
      if (n <= LIST) {
        // the draw's range comes first in the order
        const u64 a0 = z.token_of(0, tid, tid < n_u), a1 = two ? z.token_of(1, tid - n_u, tid >= n_u && tid < n) : 0;
        const u64 tok = z.sorted(tid < n_u ? a0 : a1, n);
        const u64 w = z.weight(logit_of(tok));  // (all lanes)
        const u64 mine = tid < n ? w : 0, scan = z.block_scan(mine);
        if (tid == 0) s.part[0] = s.part[5] = 0;
        __syncthreads();
        if (tid == n_u - 1) s.part[5] = scan;
        __syncthreads();
        const u64 incl = tid < n_u ? total[2] + scan : total[1] + scan - s.part[5];
        if (BY_ID) {  // top_p's last token, or that min_p keeps fewer
          if (need_p ? mine && incl - mine < pm && pm <= incl : tid == 0) {
            s.ctl[z.phase].comp = need_p ? tok : 0;
            s.ctl[z.phase].count = 1;
          }
        } else {
          if (need_p) {
            if (mine && incl - mine < pm && pm <= incl) s.part[0] = incl;
            __syncthreads();
            mass = s.part[0];
          }
          const u64 want = reach_u(mass);
          if (mass > 0 && mine && tid < n_u && incl - mine < want && want <= incl) {
            a.out[row] = index_of(tok);
            s.ctl[z.phase].count = 1;
          }
        }
      }
      __syncthreads();
    }
    const Ctl found = z.decide();
    if (found.count) {
      if (BY_ID)
        z.draw_by_id(found.comp, reach_u, a.out + row);
      else
        z.meet();
      return;
    }
  }
  auto masses = [&] { z.template histogram<true>([&](float x, int idx) { return live(x, idx) ? z.bucket0(x) : -1; }); };
  masses();
  if (z.rank == 0 && tid == 0) {
    u64 over = 0;
    for (int r = 0; r < z.ranks; ++r) over += *z.cl.map_shared_rank(&s.part[1], r);
    s.ctl[z.phase].excl = s.tot[BUCKETS - 1];
    s.ctl[z.phase].incl = over;
  }
  const Ctl sums = z.decide();
  u64 mass = sums.incl;  // what min_p keeps
  const u64 pm = reach_p(sums.excl);
  u64 cut = eligible;
  if (pm <= mass && pm < sums.excl) {  // top_p keeps less
    refined = false;
    const Ctl last = z.template select<true>(pm, live, &refined);
    mass = last.incl;
    cut = last.comp;
    if (!BY_ID && refined) masses();
  }
  if (BY_ID) {
    z.draw_by_id(cut, reach_u, a.out + row);
    return;
  }
  const u64 comp = z.template select<true>(reach_u(mass), live, &refined).comp;
  if (z.rank == 0 && tid == 0) a.out[row] = index_of(comp);
  z.meet();
}

template <typename T, bool BY_ID> cudaError_t launch(SampleArgs a, int rows, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  static DeviceOnce configured;
  if ((e = max_dynamic_smem_once(reinterpret_cast<const void*>(sample_kernel<T, BY_ID>), static_cast<int>(sizeof(Smem)), configured)) != cudaSuccess)
    return e;
  // CTAs of a row: as its size needs, and more while all rows' CTAs still run at once, two on an SM
  // sums of 15-bit parts and of near masses stay within 32 bits; 32 fp32 vectors a thread, the first off a boundary too
  constexpr int MAX_CHUNK = 65536 - 3;
  static_assert(MAX_CHUNK + 3 <= 32 * ST * 4 && SAMPLE_MAX_VOCAB <= 8 * MAX_CHUNK, "collect_from keeps a bit for each of a thread's vectors");
  int ranks = 1;
  auto chunk = [&](int r) { return (a.vocab + r - 1) / r; };
  while (ranks < 8 && (chunk(ranks) > MAX_CHUNK || (1ll * rows * ranks <= sms && chunk(ranks) > 4096))) ranks *= 2;
  a.chunk = chunk(ranks);
  a.rows = rows;
  a.wave = std::max(1, 2 * sms / ranks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * ranks);
  cfg.blockDim = dim3(ST);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = launch_overlap_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, BY_ID>, a);
}

}  // namespace

cudaError_t launch_sample(const void* logits, long long ld, cb_dtype dt, int rows, int vocab, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const float* uniform, bool by_id,
                          int32_t* out, cudaStream_t s) {
  SampleArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.vocab = vocab;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniform = uniform;
  a.out = out;
  if (dt == CB_BF16) return by_id ? launch<bf16, true>(a, rows, s) : launch<bf16, false>(a, rows, s);
  return by_id ? launch<float, true>(a, rows, s) : launch<float, false>(a, rows, s);
}

}  // namespace cb
