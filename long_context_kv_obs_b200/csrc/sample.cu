// Token sampling: temperature, top-k, top-p, min-p and one given random number a row.
//
// Which tokens stay is decided on the row's order (logit down, index up): each filter keeps a
// head of it, so the outcome is one cut (key, index), and the token is found where the kept
// mass, summed in index order, passes u times its total.  No sort of the row.
//
// Masses.  A vocabulary of 10^5 flat probabilities puts borders 10^-5 apart, and a sum of n weights
// w that carry independent errors e is off by e w sqrt(n): fp32 weights (e = 2^-24, 2e-5 w at n =
// 10^5; worse where equal logits repeat one error) with fp32 sums (3e-3 w) would move a border once in
// a hundred rows.  So weights carry 31 bits and are summed in fp64.  2^t, t = (z - max) log2(e) / T:
// t in fp64 is rounded to 32 fraction bits, whose upper 8 pick 2^(j / 256) from a table that the CUDA
// function exp2 fills (an integer in 2^-30 units) and whose lower 24 give x = r ln 2 < 2.8e-3 and
// 2^r - 1 = x + x^2 / 2 + x^3 / 6 in fp32 (2^-24 of it, 2^-32 of the weight); integer and product
// add up to the mantissa, and exponent and mantissa are put together as an fp64.  That is 4 fp64
// operations an element where the Taylor series in fp64 took 13, which bound pass D.  The largest
// logit's weight is 1 exactly.  Weights below 2^-64 of it count as nothing: all of them together are
// below 2^-46 of the mass.  Sums run in a fixed order.
//
// A row is a cluster of CTAs, each with a slice of it in shared memory, read from HBM once.
//   A  the maximum
//   B  top-k, few: the k-th largest of the threads' own maxima is a bound that k elements reach; what
//      reaches it goes to one CTA, which sorts it, sums it in that order for top-p, and again in
//      index order for the token
//   C  else the cut is searched: counts or masses by bins below the maximum (shared-memory integer
//      atomics: order does not matter), summed over the cluster through distributed shared memory.
//      bf16: 2048 bins hold one value each (those nearest zero share one), so counts give masses to
//      fp64, the border's bin is the cut's value, and of its ties the lowest indices stay.  4096 bins
//      leave fewer rows in doubt (below), but take too long to sum (a row over 16 CTAs: 33 -> 62 us).
//      fp32: 512 bins of the distance below the maximum.  A quarter of the row is summed first, in
//      fp32: a lower bound S of the mass.  Tokens below (1 - top_p) S / V together hold less than the
//      1 - top_p that is cut: they stay out, and the bins spread over what is left (atomics that meet in
//      a bin wait for one another: bins of 1/8 octave cost a flat row 26k cycles).  The bins hold
//      masses to 16 bits only: the exact sums of D decide whether the bin is the right one (else its
//      neighbour is taken).
//      A bin of several values is searched again by ranges of the key, in 2^-31 units of the bin's
//      weights, or exactly once a bin is one key.
//   D  fp64 sums of the kept weights by 32-vector stretches of a warp, in index order.  For top-p the
//      whole mass is summed beside them, a weight an element, unless the counts bound it well enough to
//      know the cut: then vectors that hold nothing kept cost a packed comparison
//   E  the stretch, lane and element where u * total falls
#include <cooperative_groups.h>

#include <climits>

#include "kernels.cuh"
#include "tc_sm100.cuh"

namespace kvc {
namespace cg = cooperative_groups;

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 512;
constexpr int SP_WIDE = 2048;                   // bins of a count by bf16 keys
constexpr int SP_MAXC = 16;
constexpr int SP_LIST = 4096;                   // candidates that one CTA sorts
constexpr float SP_ONE = 8388608.f;             // 2^23: adding it leaves the rounded integer in a float's low bits

struct alignas(16) SpShared {                   // the slice follows: its vectors are 16-byte aligned
  union {
    struct {
      unsigned hist[2 * SP_BINS];               // counts or masses; two 16-bit limbs of a mass
      unsigned sum[2 * SP_BINS];                // the cluster's
      unsigned wide[SP_WIDE];                   // counts by value
      unsigned total[SP_WIDE];                  // the cluster's
    };
    unsigned long long list[SP_LIST];
  };
  uint2 table[256];                             // 2^(j / 256): in 2^-30 units, and as an fp32
  double part;                                  // beside a histogram: the mass of the slice, to fp32
  unsigned long long xch[2][SP_MAXC][2];        // values of every CTA of the cluster, two steps deep
  double red[SP_WARPS];
  double found[4];
  int ifound[2];
  int cand[SP_WARPS][2];
  int nlist;
};

template <typename T> struct SpVec;
template <> struct SpVec<__nv_bfloat16> {
  static constexpr int N = 8, KSHIFT = 16;      // keys differ in their upper 16 bits only
  // NaN to -infinity and -0 to +0
  __device__ __forceinline__ static uint4 clean(uint4 u) {
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(w + i);
      x = __hadd2(__hmax2(x, __float2bfloat162_rn(-INFINITY)), __float2bfloat162_rn(0.f));
      w[i] = *reinterpret_cast<uint32_t*>(&x);
    }
    return u;
  }
  __device__ __forceinline__ static float largest(uint4 u) {
    const uint32_t* w = &u.x;
    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(w);
#pragma unroll
    for (int i = 1; i < 4; ++i) x = __hmax2(x, *reinterpret_cast<const __nv_bfloat162*>(w + i));
    return fmaxf(__low2float(x), __high2float(x));
  }
  // whether any element lies in [lo, hi]; the bounds as the nearest values inside, two to a word
  struct Range {
    __nv_bfloat162 lo, hi;
    __device__ __forceinline__ Range(float l, float h)
        : lo(__bfloat162bfloat162(__float2bfloat16_ru(l))), hi(__bfloat162bfloat162(__float2bfloat16_rd(h))) {}
    __device__ __forceinline__ bool any(uint4 u) const {
      const uint32_t* w = &u.x;
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(w + i);
        m |= __hge2_mask(x, lo) & __hle2_mask(x, hi);
      }
      return m != 0;
    }
  };
};
template <> struct SpVec<float> {
  static constexpr int N = 4, KSHIFT = 0;
  __device__ __forceinline__ static uint4 clean(uint4 u) {
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]), -INFINITY) + 0.f);
    return u;
  }
  __device__ __forceinline__ static float largest(uint4 u) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  struct Range {
    float lo, hi;
    __device__ __forceinline__ Range(float l, float h) : lo(l), hi(h) {}
    __device__ __forceinline__ bool any(uint4 u) const {
      const uint32_t* w = &u.x;
      bool m = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) m |= __uint_as_float(w[i]) >= lo && __uint_as_float(w[i]) <= hi;
      return m;
    }
  };
};

__device__ __forceinline__ uint32_t sp_key(float z, int shift) { return f2key(z) >> shift; }
template <int KSHIFT>
__device__ __forceinline__ float sp_value(uint32_t key) {
  // the dropped low bits of a negative value's key are ones
  if (KSHIFT) key = (key << KSHIFT) | (key >> (31 - KSHIFT) ? 0u : (1u << KSHIFT) - 1u);
  return key2f(key);
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 sp_load(const T* row, int64_t i, int V) {
  constexpr int N = SpVec<T>::N;
  if (ALIGNED && i + N <= V) return ld_stream16(row + i);
  union {
    T e[N];
    uint4 u;
  } x;
#pragma unroll
  for (int j = 0; j < N; ++j) x.e[j] = i + j < V ? row[i + j] : T(-INFINITY);
  return x.u;
}

extern __shared__ __align__(16) uint8_t sp_raw[];   // SpShared, the slice, a double a stretch of it
__device__ __forceinline__ SpShared& sp_sh() { return *reinterpret_cast<SpShared*>(sp_raw); }
__device__ __forceinline__ uint4* sp_slice() { return reinterpret_cast<uint4*>(sp_raw + sizeof(SpShared)); }

// Functions of several callers are kept out of line, and their state comes by value or from shared
// memory: a row runs each pass a few times only, so code that is not there need not be fetched.
__device__ __forceinline__ double sp_warp_scan(double inc) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double y = __shfl_up_sync(FULL, inc, d);
    if ((int)(threadIdx.x & 31) >= d) inc += y;
  }
  return inc;
}
__device__ __forceinline__ int sp_warp_scan(int inc) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(FULL, inc, d);
    if ((int)(threadIdx.x & 31) >= d) inc += y;
  }
  return inc;
}
// Sum over the CTA, in a fixed order, known to every thread.
__device__ __noinline__ double sp_block_sum(double v) {
  SpShared& sh = sp_sh();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum_d(v);
  __syncthreads();
  if (lane == 0) sh.red[warp] = v;
  __syncthreads();
  v = sh.red[lane & (SP_WARPS - 1)];
#pragma unroll
  for (int o = SP_WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
// Sum of the threads before (x) and of the CTA (y).
__device__ __noinline__ double2 sp_block_scan(double mine) {
  SpShared& sh = sp_sh();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const double inc = sp_warp_scan(mine);
  __syncthreads();
  if (lane == 31) sh.red[warp] = inc;
  __syncthreads();
  const double x = sh.red[lane & (SP_WARPS - 1)];
  double b = (lane & (SP_WARPS - 1)) < warp ? x : 0.0, t = x;
#pragma unroll
  for (int o = SP_WARPS / 2; o > 0; o >>= 1) {
    b += __shfl_xor_sync(FULL, b, o);
    t += __shfl_xor_sync(FULL, t, o);
  }
  return make_double2(b + inc - mine, t);
}
// Two values of every CTA (known to all its threads) to all: each CTA writes its own into every other's
// shared memory (a store does not wait), and after the cluster barrier the reads are local.  A slot
// is written again two exchanges later: by then its reader has passed the barrier between.
__device__ __noinline__ void sp_exchange(int C, int rank, int slot, unsigned long long a, unsigned long long b) {
  cg::cluster_group cl = cg::this_cluster();
  if ((int)threadIdx.x < C) {
    unsigned long long* o = cl.map_shared_rank(&sp_sh().xch[slot][rank][0], threadIdx.x);
    o[0] = a;
    o[1] = b;
  }
  cl.sync();
}
// The weight of logit z: 2^((z - zmax) c), for z within 2^-64 of the largest.
__device__ __forceinline__ double sp_raw_weight(float z, float zmax, double c) {
  const double r = ((double)z - (double)zmax) * c + 1572864.0;   // 1.5 * 2^20: 32 fraction bits, the low word
  const uint32_t f = (uint32_t)__double2loint(r);
  const uint2 tab = sp_sh().table[f >> 24];
  // r in 2^-24 units, without its last bit, and 2^r - 1
  const float x = (__uint_as_float(0x4B000000u | ((f & 0xffffffu) >> 1)) - SP_ONE) * (float)(0.6931471805599453 / 2147483648.0);
  const float q = fmaf(x * x, fmaf(x, 1.f / 6.f, 0.5f), x);
  const uint32_t m = tab.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(tab.y) * q, 1073741824.f, SP_ONE)) - 0x4B000000);
  // m 2^(k - 30), 2^30 <= m < 2^31, k = high word - 0x41380000: exponent field k + 1023 over m's low 30 bits
  const uint32_t hi = ((uint32_t)__double2hiint(r) << 20) + (uint32_t)((1022u - 0x41380000u) << 20) + (m >> 10);
  return __hiloint2double((int)hi, (int)(m << 22));
}
// The same times 2^e, 0 below zlow.
__device__ __noinline__ double sp_weight(float z, float zmax, float zlow, double c, int e) {
  if (!(z >= zlow)) return 0.0;
  const double w = sp_raw_weight(z, zmax, c);
  return __hiloint2double(__double2hiint(w) + (e << 20), __double2loint(w));
}

// The sums over the cluster of `words` words at src, in every CTA's `sum` (both at one place in all
// of them; words a multiple of 4 C).  Each CTA adds up its share of the words, 16 bytes from a CTA a thread, and
// hands the result to all: a load and a store a thread, where reading all histograms by all CTAs
// took 19k cycles for 2048 bins on 16 of them.  After the call src may be written again.
__device__ __noinline__ void sp_cluster_add(unsigned* src, unsigned* sum, int words, int C, int rank) {
  cg::cluster_group cl = cg::this_cluster();
  const int quads = words / (4 * C);            // of a CTA's share
  for (int j = threadIdx.x; j < quads; j += SP_THREADS)
    reinterpret_cast<uint4*>(sum)[rank * quads + j] = make_uint4(0, 0, 0, 0);
  cl.sync();
  for (int j = threadIdx.x; j < quads * C; j += SP_THREADS) {
    const int r = j / quads, w = 4 * (rank * quads + j - r * quads);
    const uint4 x = *reinterpret_cast<const uint4*>(cl.map_shared_rank(src + w, (rank + r) & (C - 1)));
    if (x.x) atomicAdd(sum + w, x.x);
    if (x.y) atomicAdd(sum + w + 1, x.y);
    if (x.z) atomicAdd(sum + w + 2, x.z);
    if (x.w) atomicAdd(sum + w + 3, x.w);
  }
  __syncthreads();
  for (int j = threadIdx.x + quads; j < quads * C; j += SP_THREADS) {   // (the first share: its own)
    const int r = j / quads, w = 4 * (rank * quads + j - r * quads);
    *reinterpret_cast<uint4*>(cl.map_shared_rank(sum + w, (rank + r) & (C - 1))) = *reinterpret_cast<const uint4*>(sum + w);
  }
  cl.sync();
}

enum { SP_COUNT, SP_SHARE, SP_LIMBS, SP_KEYS };
// The first bin at which the sum over the cluster's histograms reaches `target` (SHARE: that share of
// the cluster's `part`), or the last that holds something: returned, with the sum before it in
// found[0] and the bin's own value in found[1].  What a word of bin i stands for: COUNT, 1; SHARE, 2^-15
// of the weight at the bin's middle (bins `octaves` wide); LIMBS, 1, and a word of the histogram's second half 2^16; KEYS,
// the weight of key first - i in 2^-(31 + e) units.  A thread has one bin.
// A CTA's words hold what its slice (40960 elements at most) can bring: 65535 or 2^(15 + 1/16) each, below
// 2^32.  A row's need not: SHARE gives up its last e bits before the cluster's sum, and a CTA's limbs
// (below 2^48 together) are cut anew at bit 28, so that 16 CTAs' lower halves stay below 2^32.  (Below a
// temperature of 2^-124 bins are wider than 1/8 octave and SHARE's words may wrap: pass D then moves on from
// a border that is wrong.)
template <int KS>
__device__ __noinline__ int sp_border(int kind, double target, int C, int rank, uint32_t first, int e, float zmax,
                                      float zlow, double c, float octaves) {
  static_assert(SP_BINS == SP_THREADS, "a bin a thread");
  cg::cluster_group cl = cg::this_cluster();
  SpShared& sh = sp_sh();
  if (kind == SP_LIMBS || (kind == SP_SHARE && e > 0)) {
    __syncthreads();
    unsigned& lo = sh.hist[threadIdx.x];
    if (kind == SP_LIMBS) {
      unsigned& hi = sh.hist[SP_BINS + threadIdx.x];
      const unsigned long long v = ((unsigned long long)hi << 16) + lo;
      lo = (unsigned)v & 0xfffffffu;
      hi = (unsigned)(v >> 28);
    } else {
      lo = (lo + (1u << (e - 1))) >> e;
    }
  }
  sp_cluster_add(sh.hist, sh.sum, kind == SP_LIMBS ? 2 * SP_BINS : SP_BINS, C, rank);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long h = sh.sum[threadIdx.x];
  if (kind == SP_LIMBS) h += (unsigned long long)sh.sum[SP_BINS + threadIdx.x] << 28;
  if (kind == SP_SHARE) h <<= e;
  if (kind == SP_SHARE && warp == 0) {
    double m = lane < C ? *cl.map_shared_rank(&sh.part, lane) : 0.0;
    m = warp_sum_d(m);
    if (lane == 0) sh.found[3] = target * m;
  }
  double v = (double)h;
  if (kind == SP_SHARE) v *= (double)(tc::ex2((float)threadIdx.x * -octaves) * 0x1p-15f);
  if (kind == SP_KEYS && h) v *= sp_weight(sp_value<KS>(first - threadIdx.x), zmax, zlow, c, 31 + e);
  const double2 sc = sp_block_scan(v);
  const double inc = sc.x + v;
  if (kind == SP_SHARE) target = sh.found[3];
  const unsigned some = __ballot_sync(FULL, v > 0.0);
  const unsigned hit = __ballot_sync(FULL, v > 0.0 && inc >= target);
  if (lane == 0) {
    sh.cand[warp][0] = hit ? warp * 32 + __ffs(hit) - 1 : INT_MAX;
    sh.cand[warp][1] = some ? warp * 32 + 31 - __clz(some) : -1;
  }
  __syncthreads();
  const int at = __reduce_min_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][0]);
  const int end = __reduce_max_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][1]);
  const int b = at == INT_MAX ? max(end, 0) : at;
  if ((int)threadIdx.x == b) {
    sh.found[0] = sc.x;
    sh.found[1] = v;
  }
  __syncthreads();
  return b;
}

// Bins of the bf16 values from a row's maximum down to `low`, one to a value: bin o(max) - o(z), where o
// is the value's bits below the sign, signed.  Values near zero have the most bits for the least
// difference: where the span is more than SP_WIDE, magnitudes up to `k0` bits share the bin o = 0.
struct SpWide {
  int k0, omax, n;
  __device__ __forceinline__ int order(float z) const {
    const int b = (int)(__float_as_uint(z) >> 16), m = max((b & 0x7fff) - k0, 0);
    return b & 0x8000 ? -m : m;
  }
  __device__ __forceinline__ SpWide(float zmax, float low) {   // both bf16 values, low <= zmax
    const int mz = (int)(__float_as_uint(zmax) >> 16) & 0x7fff, ml = (int)(__float_as_uint(low) >> 16) & 0x7fff;
    const bool across = zmax >= 0.f && low < 0.f;
    const int big = max(mz, ml), less = min(mz, ml);
    k0 = 0;
    if (across && mz + ml + 1 > SP_WIDE) k0 = (mz + ml + 2 - SP_WIDE) / 2;
    if (across ? k0 > less : big - less + 1 > SP_WIDE) k0 = big + 1 - SP_WIDE;
    omax = order(zmax);
    n = omax - order(low) + 1;
  }
  __device__ __forceinline__ SpWide() {}
  __device__ __forceinline__ static float of_order(int o) {    // k0 counted in
    return __uint_as_float((uint32_t)(o < 0 ? 0x8000 - o : o) << 16);
  }
  __device__ __forceinline__ bool single(int b) const { return b != omax || k0 == 0; }
  __device__ __forceinline__ float high(int b) const {
    const int o = omax - b;
    return of_order(o < 0 ? o - k0 : o + k0);
  }
  __device__ __forceinline__ float low(int b) const {
    const int o = omax - b;
    return of_order(o > 0 ? o + k0 : o - k0);
  }
  __device__ __forceinline__ float middle(int b) const { return omax == b ? 0.f : high(b); }
};
// The first of these bins at which the cluster's counts (mass: masses, to fp64 except in a bin of several
// values, taken at its middle) reach `target`, a share of their sum for masses, or the last that holds
// something: returned, with the sum before it in found[0] and all of them in found[1].  For masses found[2] and
// found[3] bound the mass of the row, of at most V tokens.  A thread has four bins.
__device__ __noinline__ int sp_wide_border(bool mass, double target, int C, int rank, SpWide wd, float zmax,
                                           float zlow, double c, int V) {
  static_assert(SP_WIDE == 4 * SP_THREADS, "four bins a thread");
  SpShared& sh = sp_sh();
  sp_cluster_add(sh.wide, sh.total, (wd.n + 4 * C - 1) / (4 * C) * (4 * C), C, rank);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = 4 * threadIdx.x;
  uint4 h = make_uint4(0, 0, 0, 0);
  if (b0 < wd.n) h = *reinterpret_cast<const uint4*>(sh.total + b0);
  double v[4], sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned cnt = (&h.x)[i];
    v[i] = (double)cnt;
    if (mass && cnt) v[i] *= sp_weight(fminf(wd.middle(b0 + i), zmax), zmax, zlow, c, 0);
    sum += v[i];
  }
  const double2 sc = sp_block_scan(sum);
  if (mass) target *= sc.y;
  int at = INT_MAX, end = -1;
  double run = sc.x, before = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (v[i] > 0.0) {
      end = b0 + i;
      if (at == INT_MAX && run + v[i] >= target) {
        at = b0 + i;
        before = run;
      }
    }
    run += v[i];
  }
  int first = __reduce_min_sync(FULL, at), last = __reduce_max_sync(FULL, end);
  if (lane == 0) {
    sh.cand[warp][0] = first;
    sh.cand[warp][1] = last;
  }
  __syncthreads();
  first = __reduce_min_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][0]);
  last = __reduce_max_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][1]);
  const int b = first == INT_MAX ? max(last, 0) : first;
  if (b >> 2 == (int)threadIdx.x) {
    if (first == INT_MAX) {
      before = sc.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) before += b0 + i < b ? v[i] : 0.0;
    }
    sh.found[0] = before;
    sh.found[1] = sc.y;
    if (mass) {
      double least = sc.y, most = sc.y + (double)V * sp_weight(wd.low(wd.n - 1), zmax, zlow, c, 0);
      if (wd.k0 > 0 && wd.omax >= 0 && wd.omax < wd.n) {
        const double cnt = (double)sh.total[wd.omax], mid = sp_weight(fminf(0.f, zmax), zmax, zlow, c, 0);
        least -= cnt * (mid - sp_weight(wd.low(wd.omax), zmax, zlow, c, 0));
        most += cnt * (sp_weight(fminf(wd.high(wd.omax), zmax), zmax, zlow, c, 0) - mid);
      }
      sh.found[2] = least;
      sh.found[3] = most;
    }
  }
  __syncthreads();
  return b;
}

template <typename T>
struct SpRow {
  static constexpr int N = SpVec<T>::N, KS = SpVec<T>::KSHIFT;
  int C, rank, nvec, i0;                        // cluster size, rank, vectors of the slice, its first index
  int step;
  float zmax, ybin;                             // bins below the maximum: (zmax - z) * ybin
  float zlow;                                   // weights below this one's, 2^-64 of the largest, are nothing
  double c;                                     // log2(e) / T
  bool cut;                                     // top-k left: key > ck, or key == ck and index <= ci
  uint32_t ck;
  int ci;

  __device__ __forceinline__ void exchange(unsigned long long a, unsigned long long b) {
    sp_exchange(C, rank, step & 1, a, b);
    ++step;
  }
  __device__ __forceinline__ void exchange(double a, double b) {
    exchange((unsigned long long)__double_as_longlong(a), (unsigned long long)__double_as_longlong(b));
  }
  __device__ __forceinline__ unsigned long long got(int r, int k) const { return sp_sh().xch[(step - 1) & 1][r][k]; }
  __device__ __forceinline__ double got_d(int r, int k) const { return __longlong_as_double((long long)got(r, k)); }
  // The sum of a value of every CTA, in their order; `before` the sum of the lower ranks'.
  __device__ __forceinline__ double cluster_sum(double x, double& before) {
    exchange(x, 0.0);
    double all = 0.0;
    before = 0.0;
#pragma unroll 1
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = all;
      all += got_d(r, 0);
    }
    return all;
  }
  __device__ __forceinline__ int border(int kind, double target, uint32_t first, int e) {
    return sp_border<KS>(kind, target, C, rank, first, e, zmax, zlow, c, octaves());
  }
  __device__ __forceinline__ float octaves() const { return ybin > 0.f ? (float)(c / (double)ybin) : 0.f; }   // a bin's width
  __device__ __forceinline__ double weight(float z, int e = 0) const { return sp_weight(z, zmax, zlow, c, e); }

  // use(value, index) for the elements of vector v, in order, U of its four words at a time.
  template <int U, typename F>
  __device__ __forceinline__ void each(int v, F&& use) const {
#pragma unroll U
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = reinterpret_cast<const uint32_t*>(sp_slice() + v)[w];
      const int idx = i0 + v * N + w * (N / 4);
      if (N == 8) {
        use(bf_lo(x), idx);
        use(bf_hi(x), idx + 1);
      } else {
        use(__uint_as_float(x), idx);
      }
    }
  }
  // Monotone in z; the maximum is in bin 0, the last bin holds all that is farther.
  __device__ __forceinline__ int bin(float z) const {
    const float r = fmaf(zmax - z, ybin, SP_ONE);
    return min(__float_as_int(r) - 0x4B000000, SP_BINS - 1);
  }
  __device__ __forceinline__ bool left(float z, int idx) const {
    if (!cut) return z > -INFINITY;
    const uint32_t key = sp_key(z, KS);
    return key > ck || (key == ck && idx <= ci);
  }
  // A lower and an upper bound on the values of bin b, outside by a thousandth of a bin (the
  // roundings of bin() are below 2^-11 of one) and a step of z.
  __device__ __forceinline__ float edge_low(int b) const {
    if (b >= SP_BINS - 1 || !(ybin > 0.f)) return -INFINITY;
    const float x = zmax - ((float)b + 0.501f) / ybin;
    return x > -3.4028234663852886e38f ? key2f(f2key(x) - 1u) : -INFINITY;
  }
  __device__ __forceinline__ float edge_high(int b) const {
    if (b == 0 || !(ybin > 0.f)) return zmax;
    return fminf(zmax, key2f(f2key(zmax - ((float)b - 0.501f) / ybin) + 1u));
  }

  // The histogram, cleared for use.
  __device__ __forceinline__ unsigned* clear_hist(int words) {
    unsigned* h = sp_sh().hist;
#pragma unroll 1
    for (int j = threadIdx.x; j < words / 4; j += SP_THREADS) reinterpret_cast<uint4*>(h)[j] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    return h;
  }

  // use(value, index) for every element of the slice with lo <= value <= hi: two instructions an
  // element where there are none
  template <typename F>
  __device__ __forceinline__ void in_range(float lo, float hi, F&& use) {
    const typename SpVec<T>::Range range(lo, hi);
#pragma unroll 1
    for (int v = threadIdx.x; v < nvec; v += SP_THREADS)
      if (range.any(sp_slice()[v]))
        each<1>(v, [&](float z, int idx) {
          if (z >= lo && z <= hi) use(z, idx);
        });
  }

  // Counts of the tokens left, by bins of one bf16 value each (of zero's neighbours, see SpWide).
  __device__ __forceinline__ void wide_hist(const SpWide& wd) const {
    unsigned* h = sp_sh().wide;
    *reinterpret_cast<uint4*>(h + 4 * threadIdx.x) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (cut) {
#pragma unroll 1
      for (int v = threadIdx.x; v < nvec; v += SP_THREADS)
        each<4>(v, [&](float z, int idx) {
          const int b = wd.omax - wd.order(z);
          if (b < wd.n && left(z, idx)) atomicAdd(h + b, 1u);
        });
      return;
    }
    const uint32_t less = (uint32_t)(-wd.k0 & 0xffff) * 0x10001u;
    // (-infinity lies beyond the last bin)
#pragma unroll 1
    for (int v = threadIdx.x; v < nvec; v += SP_THREADS) {
      const uint4 u = sp_slice()[v];
      const bool same = u.x == u.y && u.z == u.w && u.x == u.z && u.x >> 16 == (u.x & 0xffffu);   // flat rows
      const uint32_t* w = &u.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i == 0 || !same) {
          const uint32_t m = __viaddmax_s16x2_relu(w[i] & 0x7fff7fffu, less, 0u);
          const int m0 = (int)(m & 0xffffu), m1 = (int)(m >> 16);
          const int c0 = w[i] & 0x8000u ? wd.omax + m0 : wd.omax - m0, c1 = (int)w[i] < 0 ? wd.omax + m1 : wd.omax - m1;
          if (c0 < wd.n) atomicAdd(h + c0, same ? 8u : 1u);
          if (c1 < wd.n && !same) atomicAdd(h + c1, 1u);
        }
      }
    }
  }
  __device__ __forceinline__ int wide_border(bool mass, double target, const SpWide& wd, int V) {
    return sp_wide_border(mass, target, C, rank, wd, zmax, zlow, c, V);
  }

  // The index of tie `want` (from 1) of zt in this slice, by the ties of every stretch: ifound[1], set by one thread.
  __device__ __forceinline__ void find_tie(const unsigned* count, float zt, int want) const {
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x, nst = (nvec + 31) / 32;
    int st = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < nst; s0 += 32) {
      const int n = s0 + lane < nst ? (int)count[s0 + lane] : 0;
      const int inc = sp_warp_scan(n);
      const unsigned hit = __ballot_sync(FULL, inc >= want);
      if (hit) {
        st = s0 + __ffs(hit) - 1;
        want -= __shfl_sync(FULL, inc - n, __ffs(hit) - 1);
        break;
      }
      want -= __shfl_sync(FULL, inc, 31);
    }
    const int v = st * 32 + lane;
    int n = 0;
    if (v < nvec) each<1>(v, [&](float z, int idx) { n += z == zt && left(z, idx); });
    int k = sp_warp_scan(n) - n;
    if (k < want && want <= k + n)
      each<1>(v, [&](float z, int idx) {
        if (z == zt && left(z, idx) && ++k == want) sp_sh().ifound[1] = idx;
      });
  }

  // Of the values zl to zh (b0 >= 0: those of bin b0 alone) that top-k left, the key at which the count
  // (mass: the mass, in units of 2^-(31 + e)) reaches `need`, and the index of the last tie that stays.
  // False if there is less than that (then nothing else is set).  known >= 0: zl is zh, and so many there are.
  __device__ __forceinline__ bool refine(bool mass, float zl, float zh, int b0, int known, double need, int e,
                                         uint32_t& tkey, int& tidx) {
    SpShared& sh = sp_sh();
    uint32_t hi = sp_key(zh, KS), lo = max(sp_key(zl, KS), sp_key(-INFINITY, KS) + 1u);
    double above = 0.0, value = 0.0;
    bool first_search = true;
    int shift = 0;
    if (known >= 0) {
      value = mass ? (double)known * weight(zh, 31 + e) : (double)known;
      if (mass && value < need) return false;
    }
    while (((hi - lo) >> shift) >= SP_BINS) ++shift;
    while (known < 0) {
      const bool limbs = mass && shift > 0;
      unsigned* hist = clear_hist(limbs ? 2 * SP_BINS : SP_BINS);
      in_range(sp_value<KS>(lo), sp_value<KS>(hi), [&](float z, int idx) {
        if ((b0 >= 0 && bin(z) != b0) || !left(z, idx)) return;
        const uint32_t hb = (hi - sp_key(z, KS)) >> shift;
        if (limbs) {
          const unsigned long long q = (unsigned long long)__double2ll_rn(weight(z, 31 + e));
          atomicAdd(hist + hb, (unsigned)(q & 0xffffu));
          atomicAdd(hist + SP_BINS + hb, (unsigned)(q >> 16));
        } else {
          atomicAdd(hist + hb, 1u);
        }
      });
      const int hb = border(limbs ? SP_LIMBS : mass ? SP_KEYS : SP_COUNT, need - above, hi, e);
      const double ab = sh.found[0];
      value = sh.found[1];
      if (mass && first_search && ab + value < need) return false;
      first_search = false;
      above += ab;
      const uint32_t top = hi - ((uint32_t)hb << shift);
      const uint32_t span = (1u << shift) - 1u;
      lo = top - lo > span ? top - span : lo;
      hi = top;
      if (shift == 0) break;
      shift = 0;
      while (((hi - lo) >> shift) >= SP_BINS) ++shift;
    }
    tkey = hi;
    // of the ties of tkey the first `take` in index order stay; `value` tells how many there are
    double take = need - above, ties = value;
    if (mass) {
      const double w = weight(sp_value<KS>(tkey), 31 + e);
      take = w > 0.0 ? ceil(take / w) : 1.0;
      ties = w > 0.0 ? rint(value / w) : 1.0;
    }
    if (take < 1.0) take = 1.0;
    tidx = INT_MAX;
    if (take >= ties) return true;
    // ties of every 32-vector stretch, in the histogram's words
    const int lane = threadIdx.x & 31;
    const float zt = sp_value<KS>(tkey);
    unsigned* count = sh.hist;
    double mine = 0.0;
    const typename SpVec<T>::Range range(zt, zt);
#pragma unroll 1
    for (int v0 = threadIdx.x - lane; v0 < nvec; v0 += SP_THREADS) {
      const int v = v0 + lane;
      int n = 0;
      if (v < nvec && range.any(sp_slice()[v])) each<1>(v, [&](float z, int idx) { n += z == zt && left(z, idx); });
      n = __reduce_add_sync(FULL, n);
      if (lane == 0) {
        count[v0 >> 5] = (unsigned)n;
        mine += n;
      }
    }
    mine = sp_block_sum(mine);
    double before;
    cluster_sum(mine, before);
    const bool here = before < take && take <= before + mine;
    if (here) find_tie(count, zt, (int)(take - before));        // this slice holds the last tie that stays
    __syncthreads();
    tidx = (int)cluster_sum(here ? (double)sh.ifound[1] : 0.0, before);   // one CTA's
    return true;
  }
};

// a[0, m) sorted downwards, all different.  Few: each finds its place by counting what is above it, two
// to a read that all lanes share (256 rows, top-k 50: 84 us with the merges below, 76 so).  More: bitonic
// merges over n >= m, a power of two, the rest zeros.
constexpr int SP_COUNTED = 256;
__device__ __noinline__ void sp_sort(unsigned long long* a, int m, int n) {
  if (m <= SP_COUNTED) {
    __syncthreads();
    const unsigned long long x = (int)threadIdx.x < m ? a[threadIdx.x] : ~0ull;
    int place = 0;
    if ((int)(threadIdx.x & ~31u) < m) {
#pragma unroll 4
      for (int j = 0; j + 1 < m; j += 2) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(a + j);
        place += (y.x > x) + (y.y > x);
      }
      if (m & 1) place += a[m - 1] > x;
    }
    __syncthreads();
    if ((int)threadIdx.x < m) a[place] = x;
    __syncthreads();
    return;
  }
  for (int i = m + threadIdx.x; i < n; i += SP_THREADS) a[i] = 0ull;
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
#pragma unroll 1
      for (int p = threadIdx.x; p < n / 2; p += SP_THREADS) {
        const int i = 2 * p - (p & (j - 1)), q = i + j;
        const unsigned long long x = a[i], y = a[q];
        if ((x < y) == ((i & k) == 0)) {
          a[i] = y;
          a[q] = x;
        }
      }
    }
  __syncthreads();
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(SP_THREADS, 2) sample_kernel(SampleParams p, int per_cta) {
  constexpr int N = SpVec<T>::N, KS = SpVec<T>::KSHIFT;
  static_assert(sizeof(SpShared) % 16 == 0, "vectors follow");
  SpShared& sh = sp_sh();
  uint4* slice = sp_slice();
  double* wsum = reinterpret_cast<double*>(slice + per_cta / N);   // kept mass of every 32-vector stretch
  cg::cluster_group cl = cg::this_cluster();
  SpRow<T> s;
  cl.barrier_arrive();                          // every CTA of the cluster runs before its shared memory is written
  s.C = (int)cl.num_blocks();
  s.rank = (int)cl.block_rank();
  const int row = blockIdx.x / s.C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  s.i0 = s.rank * per_cta;
  s.nvec = max(0, min(per_cta, p.V - s.i0) + N - 1) / N;
  s.step = 0;
  s.cut = false;
  const T* z0 = reinterpret_cast<const T*>(p.logits) + row * p.row_stride;

  // A: the slice into shared memory and the maximum
  float best = -INFINITY;
#pragma unroll 4
  for (int v = tid; v < s.nvec; v += SP_THREADS) {
    const uint4 u = SpVec<T>::clean(sp_load<T, ALIGNED>(z0, s.i0 + (int64_t)v * N, p.V));
    slice[v] = u;
    best = fmaxf(best, SpVec<T>::largest(u));
  }
  if (tid < 256) {
    const double x = exp2((double)tid / 256.0);
    sh.table[tid] = make_uint2((unsigned)__double2uint_rn(x * 1073741824.0), __float_as_uint((float)x));
  }
  const float T_ = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float pf = p.top_p ? p.top_p[row] : 1.f, mf = p.min_p ? p.min_p[row] : 0.f;
  {
    const float m = warp_max(best);
    if (lane == 0) sh.red[warp] = (double)m;
    __syncthreads();
    double x = sh.red[lane & (SP_WARPS - 1)];
    x = (double)warp_max((float)x);
    cl.barrier_wait();
    s.exchange(x, 0.0);
    s.zmax = -INFINITY;
#pragma unroll 1
    for (int r = 0; r < s.C; ++r) s.zmax = fmaxf(s.zmax, (float)s.got_d(r, 0));
  }
  if (s.zmax == -INFINITY || !(T_ > 0.f)) {
    // nothing to take, or the first token of the order
    int at = INT_MAX;
    if (s.zmax > -INFINITY)
      s.in_range(s.zmax, s.zmax, [&](float, int idx) { at = min(at, idx); });
    at = __reduce_min_sync(FULL, at);
    __syncthreads();
    if (lane == 0) sh.cand[warp][0] = at;
    __syncthreads();
    at = __reduce_min_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][0]);
    s.exchange((unsigned long long)at, 0ull);
    unsigned long long first = INT_MAX;
#pragma unroll 1
    for (int r = 0; r < s.C; ++r) first = min(first, s.got(r, 0));
    if (s.rank == 0 && tid == 0) {
      const bool any = s.zmax > -INFINITY;
      p.token[row] = any ? (int)first : -1;
      if (p.logprob) p.logprob[row] = any ? 0.f : -INFINITY;
      if (p.kept) p.kept[row] = any;
    }
    return;
  }
  if (s.zmax == INFINITY) {
    // infinite logits share the mass: they become 0, all others -infinity
#pragma unroll 1
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      T* e = reinterpret_cast<T*>(slice + v);
#pragma unroll 1
      for (int j = 0; j < N; ++j) e[j] = (float)e[j] == INFINITY ? T(0.f) : T(-INFINITY);
    }
    best = best == INFINITY ? 0.f : -INFINITY;
    s.zmax = 0.f;
  }
  double temp = (double)T_;
  if (N == 4 && s.zmax > 1e30f && T_ > 1e36f) {
    // differences of such logits may pass fp32's range, and count at such a temperature: all are halved, the
    // temperature too (exactly, but for the last bit of logits below 2^-125)
#pragma unroll 1
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      float* e = reinterpret_cast<float*>(slice + v);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] *= 0.5f;
    }
    best *= 0.5f;
    s.zmax *= 0.5f;
    temp *= 0.5;
  }
  s.c = 1.4426950408889634 / temp;
  s.ybin = fminf((float)(8.0 * s.c), 3e38f);
  {
    const double x = (double)s.zmax - 64.0 / s.c;   // (an infinite temperature: -infinity, held above it)
    s.zlow = x > -3.4028234663852886e38 ? __double2float_ru(x) : -3.4028234663852886e38f;
  }
  const double top_p = (double)pf;
  const bool use_p = pf < 1.f;
  // p_i >= min_p max p  <=>  z_i >= max z + T ln(min_p); as the least such value of the dtype's keys
  float zcut = -INFINITY;
  if (mf > 0.f) {
    const double x = (double)s.zmax + (mf < 1.f ? temp * log((double)mf) : 0.0);
    zcut = x > -3.4028234663852886e38 ? __double2float_ru(x) : -INFINITY;
  }
  float u = p.u[row];
  u = u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f;   // NaN and negatives: 0

  if (k > 0 && k < p.V) {
    if (k <= s.C * (SP_THREADS / 4)) {
      // B: a bin that the k-th largest cannot lie beyond, from the threads' own maxima
      unsigned* hist = s.clear_hist(SP_BINS);
      if (best > -INFINITY) atomicAdd(hist + s.bin(best), 1u);
      const int far = s.border(SP_COUNT, (double)k, 0, 0);
      const float low = sh.found[0] + sh.found[1] >= (double)k ? s.edge_low(far) : -INFINITY;
      const float floor_ = fmaxf(low, -3.4028234663852886e38f);   // never -infinity itself
      // what reaches it, first counted
      double n = 0.0, off;
      s.in_range(floor_, INFINITY, [&](float, int) { n += 1.0; });
      n = sp_block_sum(n);
      const int m = (int)s.cluster_sum(n, off);
      if (m <= SP_LIST) {
        // the candidates, to the first CTA (its histograms are read no more: all have passed the exchange)
        if (tid == 0) sh.nlist = (int)off;
        __syncthreads();
        unsigned long long* list = cl.map_shared_rank(&sh.list[0], 0);
        s.in_range(floor_, INFINITY, [&](float z, int idx) {
          list[atomicAdd(&sh.nlist, 1)] = ((unsigned long long)f2key(z) << 32) | (unsigned)~idx;
        });
        cl.sync();
        if (s.rank != 0) return;                // the rest is the first CTA's own
        int np = 2;
        while (np < m) np <<= 1;
        sp_sort(sh.list, m, np);
        const int kk = min(k, m);
        // weights in the order, a stretch a thread, and their running sum
        const int Q = (np + SP_THREADS - 1) / SP_THREADS;
        auto value = [&](int i) { return key2f((uint32_t)(sh.list[i] >> 32)); };
        double sum = 0.0, nkeep = 0.0;
#pragma unroll 1
        for (int i = tid * Q; i < min(kk, tid * Q + Q); ++i) sum += s.weight(value(i));
        double2 sc = sp_block_scan(sum);
        double run = sc.x;
#pragma unroll 1
        for (int i = tid * Q; i < min(kk, tid * Q + Q); ++i) {
          // kept: a head of the order, both conditions only turn false
          nkeep += i == 0 || ((!use_p || run < top_p * sc.y) && value(i) >= zcut);
          run += s.weight(value(i));
        }
        const int keep = (int)sp_block_sum(nkeep);
        // the kept ones in index order
        int nk = 2;
        while (nk < keep) nk <<= 1;
#pragma unroll 1
        for (int i = tid; i < keep; i += SP_THREADS) {
          const unsigned long long x = sh.list[i];
          sh.list[i] = (x << 32) | (x >> 32);   // sorted downwards: index up is ~index down
        }
        sp_sort(sh.list, keep, nk);
        sum = 0.0;
        const int Qk = (nk + SP_THREADS - 1) / SP_THREADS;
#pragma unroll 1
        for (int i = tid * Qk; i < min(keep, tid * Qk + Qk); ++i) sum += s.weight(key2f((uint32_t)sh.list[i]));
        sc = sp_block_scan(sum);
        run = sc.x;
        const double goal = (double)u * sc.y;
        // the first whose running sum passes the goal (else, by rounding, the last with mass)
        int at = INT_MAX, last = -1;
#pragma unroll 1
        for (int i = tid * Qk; i < min(keep, tid * Qk + Qk); ++i) {
          const double w = s.weight(key2f((uint32_t)sh.list[i]));
          if (w > 0.0) {
            last = i;
            if (at == INT_MAX && run + w > goal) at = i;
          }
          run += w;
        }
        at = __reduce_min_sync(FULL, at);
        last = __reduce_max_sync(FULL, last);
        if (lane == 0) {
          sh.cand[warp][0] = at;
          sh.cand[warp][1] = last;
        }
        __syncthreads();
        if (tid == 0) {
          for (int q = 0; q < SP_WARPS; ++q) {
            at = min(at, sh.cand[q][0]);
            last = max(last, sh.cand[q][1]);
          }
          const unsigned long long x = sh.list[at == INT_MAX ? last : at];
          p.token[row] = (int)~(unsigned)(x >> 32);
          if (p.logprob) p.logprob[row] = (float)log(s.weight(key2f((uint32_t)x)) / sc.y);
          if (p.kept) p.kept[row] = keep;
        }
        return;
      }
    }
    // C: the k-th key by counts
    uint32_t tk = 0;
    int ti = INT_MAX;
    if constexpr (N == 8) {
      // over the positive values, then as far below zero, then to the lowest value, until k are there (the
      // wider the span, the more values share the bin at zero, and the last span is a few bins only)
      SpWide wd;
      int b;
      for (int span = s.zmax > 0.f && k <= p.V / 2 ? 0 : 1;; ++span) {
        const float lowest = -3.3895313892515355e38f;
        wd = SpWide(s.zmax, span == 0 ? s.zmax * 0x1p-15f
                            : span == 2 ? lowest
                            : s.zmax > 0.f ? -s.zmax : fmaxf(s.zmax * 0x1p15f, lowest));
        s.wide_hist(wd);
        b = s.wide_border(false, (double)k, wd, p.V);
        if ((double)k <= sh.found[1] || span == 2) break;
      }
      if ((double)k <= sh.found[1]) {
        s.refine(false, wd.low(b), fminf(wd.high(b), s.zmax), -1, wd.single(b) ? (int)sh.total[b] : -1,
                 (double)k - sh.found[0], 0, tk, ti);
        s.cut = true;
      }
    } else {
      unsigned* hist = s.clear_hist(SP_BINS);
      double have = 0.0;
#pragma unroll 1
      for (int v = tid; v < s.nvec; v += SP_THREADS) {
        int run = 0, rb = -1;                     // equal neighbours in one atomic
        s.template each<1>(v, [&](float z, int) {
          if (!(z > -INFINITY)) return;
          have += 1.0;
          const int bb = s.bin(z);
          if (bb != rb) {
            if (run) atomicAdd(hist + rb, (unsigned)run);
            rb = bb;
            run = 0;
          }
          ++run;
        });
        if (run) atomicAdd(hist + rb, (unsigned)run);
      }
      double lower;
      have = s.cluster_sum(sp_block_sum(have), lower);
      if ((double)k < have) {
        const int b = s.border(SP_COUNT, (double)k, 0, 0);
        s.refine(false, s.edge_low(b), s.edge_high(b), b, -1, (double)k - sh.found[0], 0, tk, ti);
        s.cut = true;
      }
    }
    if (s.cut) {
      s.ck = tk;
      s.ci = ti;
    }
  }

  int b = SP_BINS;                              // top-p: kept are the bins before b and a part of b
  double above = 0.0;
  SpWide wd;
  if (N == 8 && use_p) {
    // C: counts by value, down to where V tokens hold less than 2^-14 of the 1 - top_p of the maximum alone
    const double x = (double)s.zmax - (14.0 - log2(0.99 * (1.0 - fmax(top_p, 0.0)) / p.V)) / s.c;
    const float low = x > (double)s.zlow ? __double2float_ru(x) : s.zlow;
    wd = SpWide(s.zmax, fminf(__bfloat162float(__float2bfloat16_ru(low)), s.zmax));
    s.wide_hist(wd);
    b = s.wide_border(true, fmax(top_p, 0.0), wd, p.V);
  } else if (use_p && pf > 0.f) {
    // C: every fourth vector's mass, to fp32: a lower bound of the row's
    float some = 0.f, part = 0.f;
    const float scale = -(float)s.c;
#pragma unroll 1
    for (int v = tid; v < s.nvec; v += 4 * SP_THREADS)
      s.template each<4>(v, [&](float z, int idx) { some += s.left(z, idx) ? tc::ex2((s.zmax - z) * scale) : 0.f; });
    double lower;
    const double bound = s.cluster_sum(sp_block_sum((double)some), lower);
    // what is lighter than `mean` stays out; the bins before the last cover the rest, with a bin to spare
    const float mean = (float)fmin(0.99 * (1.0 - top_p) * bound / p.V, 0.99);
    const float range = mean > 0x1p-63f ? -log2f(mean) : 63.f;   // octaves
    s.ybin = (float)fmin((SP_BINS - 3) * s.c / (double)range, 3e38);   // (clamped, the bins reach farther)
    const int far = SP_BINS - 2;
    const float low = s.edge_low(far), oct = s.octaves();
    unsigned* hist = s.clear_hist(SP_BINS);
#pragma unroll 1
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      unsigned run = 0;                         // equal neighbours in one atomic
      int rb = -1;
      s.template each<4>(v, [&](float z, int idx) {
        const bool in = s.left(z, idx);
        const float d = s.zmax - z;
        part += in ? tc::ex2(d * scale) : 0.f;
        if (!(z >= low) || !in) return;
        const float r = fmaf(d, s.ybin, SP_ONE);
        const int bb = __float_as_int(r) - 0x4B000000;
        if (bb > far) return;
        if (bb != rb) {
          if (run) atomicAdd(hist + rb, run);
          rb = bb;
          run = 0;
        }
        // 2^-(distance from the bin's middle), at most 2^(1/16), in 2^-15 units
        const float y = fmaf(d, s.ybin, SP_ONE - r);
        run += (unsigned)__float_as_int(fmaf(tc::ex2(y * -oct), 32768.f, SP_ONE)) - 0x4B000000u;
      });
      if (run) atomicAdd(hist + rb, run);
    }
    const double whole = sp_block_sum((double)part);
    if (tid == 0) sh.part = whole;
    b = s.border(SP_SHARE, top_p, 0, p.V > 125000 ? 2 : 0);   // 125000 2^(15 + 1/16) < 2^32
  } else if (use_p) {
    b = 0;                                      // top_p <= 0: one token
  }
  // D: the kept mass by stretches of 32 vectors
  const int nst = (s.nvec + 31) / 32;
  int kept = 0;
  bool done = false;
  if constexpr (N == 8) {
    // Where the bounds on the row's mass leave no doubt about the cut, only what stays is summed: the
    // bin is one value of weight w, a number of its ties stays, and few vectors hold any of it
    // (256 rows of 128256 with filters of all kinds: 164 -> 124 us).
    const float high = use_p ? fminf(wd.high(b), s.zmax) : 0.f;
    const double w = use_p ? s.weight(high) : 0.0, share = fmax(top_p, 0.0);
    const double least = sh.found[2] * (1.0 - 1e-12), most = sh.found[3] * (1.0 + 1e-12);   // beside fp64's own errors
    if (use_p && wd.single(b) && w > 0.0 && (most - least) * share <= 0.25 * w) {
      unsigned* count = sh.hist;
      double before_b = 0.0, same = 0.0;
      const typename SpVec<T>::Range front(high, INFINITY);
#pragma unroll 1
      for (int st = warp; st < nst; st += SP_WARPS) {
        const int v = st * 32 + lane;
        double mine = 0.0;
        int n = 0;
        if (v < s.nvec && front.any(slice[v]))
          s.template each<1>(v, [&](float z, int idx) {
            if (!(z >= high) || !s.left(z, idx)) return;
            if (z == high) {
              ++n;
              return;
            }
            const double x = sp_raw_weight(z, s.zmax, s.c);
            before_b += x;
            if (z >= zcut) {
              mine += x;
              ++kept;
            }
          });
        if (__any_sync(FULL, mine > 0.0)) mine = warp_sum_d(mine);
        n = __reduce_add_sync(FULL, n);
        if (lane == 0) {
          wsum[st] = mine;
          count[st] = (unsigned)n;
          same += n;
        }
      }
      before_b = sp_block_sum(before_b);
      same = sp_block_sum(same);
      s.exchange(before_b, same);
      double ties = 0.0, earlier = 0.0;
      above = 0.0;
#pragma unroll 1
      for (int r = 0; r < s.C; ++r) {
        if (r == s.rank) earlier = ties;
        above += s.got_d(r, 0);
        ties += s.got_d(r, 1);
      }
      double take = 1.0;                        // top_p <= 0: one token
      done = b == 0;
      if (pf > 0.f) {
        take = ceil((share * least - above) / w);
        done = take == ceil((share * most - above) / w) && take >= 1.0 && take <= ties;
      }
      if (done) {
        const int stay = (int)fmin(fmax(take - earlier, 0.0), same), all = (int)same;
        int ti = stay == all ? INT_MAX : -1;
        if (stay > 0 && stay < all) {
          s.find_tie(count, high, stay);
          __syncthreads();
          ti = sh.ifound[1];
        }
        if (high >= zcut && warp == 0) {
          int from = 0;
#pragma unroll 1
          for (int s0 = 0; s0 < nst; s0 += 32) {
            const int n = s0 + lane < nst ? (int)count[s0 + lane] : 0;
            const int inc = sp_warp_scan(n), mine = min(max(stay - from - (inc - n), 0), n);
            if (mine) wsum[s0 + lane] += (double)mine * w;
            from += __shfl_sync(FULL, inc, 31);
          }
          if (lane == 0) kept += stay;
        }
        // from here on `left` is the final cut, in this slice
        const uint32_t tk = sp_key(high, KS);
        s.ci = s.cut && tk == s.ck ? min(ti, s.ci) : ti;
        s.ck = tk;
        s.cut = true;
      }
    }
  }
  const float least_kept = use_p ? -INFINITY : fmaxf(zcut, s.cut ? sp_value<KS>(s.ck) : -INFINITY);
  const typename SpVec<T>::Range may_stay(least_kept, INFINITY);
  for (int moved = 0; !done;) {
    double sums[2] = {0.0, 0.0};                // all that is left, bins before b
    // bin(z) < b  <=>  not fma(zmax - z, ybin, 2^23) >= 2^23 + b; without top-p (NaN) everything is before
    const float rb = use_p ? SP_ONE + (float)b : __int_as_float(0x7fffffff);
    const float high = N == 8 && use_p ? fminf(wd.high(b), s.zmax) : -INFINITY;   // bf16: the bin's largest value
    auto in_front = [&](float z) { return N == 8 ? z > high : !(fmaf(s.zmax - z, s.ybin, SP_ONE) >= rb); };
    const bool plain = !s.cut && zcut == -INFINITY;
    kept = 0;
#pragma unroll 1
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      double mine = 0.0;
      if (v < s.nvec) {
        if (plain) {
          s.template each<4>(v, [&](float z, int) {
            const bool some = z >= s.zlow;
            const double x = sp_raw_weight(some ? z : s.zmax, s.zmax, s.c), w = some ? x : 0.0;
            sums[0] += w;
            if (in_front(z)) {
              mine += w;
              kept += z > -INFINITY;
            }
          });
        } else if (least_kept == -INFINITY || may_stay.any(slice[v])) {
          s.template each<4>(v, [&](float z, int idx) {
            const bool in = s.left(z, idx), some = in && z >= s.zlow;
            const double x = sp_raw_weight(some ? z : s.zmax, s.zmax, s.c), w = some ? x : 0.0;
            const bool before = in_front(z);
            const bool head = in && before && z >= zcut;   // kept for certain: before bin b, above the min-p cut
            kept += head;
            sums[0] += w;
            sums[1] += before ? w : 0.0;
            mine += head ? w : 0.0;
          });
        }
      }
      if (plain) sums[1] += mine;
      mine = warp_sum_d(mine);
      if (lane == 0) wsum[st] = mine;
    }
    if (!use_p) break;
    sums[0] = sp_block_sum(sums[0]);
    sums[1] = sp_block_sum(sums[1]);
    s.exchange(sums[0], sums[1]);
    double total = 0.0;
    above = 0.0;
#pragma unroll 1
    for (int r = 0; r < s.C; ++r) {
      total += s.got_d(r, 0);
      above += s.got_d(r, 1);
    }
    // the bin is right if the sum reaches top_p of the total inside it (b == 0: it starts there)
    const double goal = pf > 0.f ? top_p * total : 0.0;
    if (above >= goal && b > 0 && moved <= 0) {
      if constexpr (N == 8) {                   // back by the bins' own masses
        double x = above;
        do {
          --b;
          x -= (double)sh.total[b] * s.weight(fminf(wd.middle(b), s.zmax));
        } while (b > 0 && (x >= goal || sh.total[b] == 0));
      } else {
        --b;
      }
      moved = -1;
      continue;
    }
    // weights of the bin scaled by 2^e are at most 1: none is above that of `top` (past 2^-64 all are nothing)
    const float zl = N == 8 ? wd.low(b) : s.edge_low(b), top = N == 8 ? high : s.edge_high(b);
    const int e = (int)fmin(((double)s.zmax - (double)top) * s.c, 100.0);
    const int known = N == 8 && wd.single(b) ? (int)sh.total[b] : -1;
    uint32_t tk;
    int ti;
    if (!s.refine(true, zl, top, N == 8 ? -1 : b, known, fmax(ldexp(goal - above, 31 + e), 0.0), e, tk, ti)) {
      bool further = moved >= 0 && (N == 8 ? b + 1 < wd.n : b < SP_BINS - 2);
      if (N == 8 && further) {                  // on by the bins' own masses, if there is anything
        double x = above;
        int to = b, last = b;
        while (to + 1 < wd.n && (to == b || x < goal)) {
          x += (double)sh.total[to] * s.weight(fminf(wd.middle(to), s.zmax));
          ++to;
          if (sh.total[to]) last = to;
          if (sh.total[to] && x + (double)sh.total[to] * s.weight(fminf(wd.middle(to), s.zmax)) >= goal) break;
        }
        further = last != b;
        b = last;
      } else if (further) {
        ++b;
      }
      if (further) {
        moved = 1;
        continue;
      }
      // between two bins by the sums' last bits: all of this one stays
      tk = max(sp_key(zl, KS), sp_key(-INFINITY, KS) + 1u);
      ti = INT_MAX;
    }
    // the part of bin b that stays
    const float zt = sp_value<KS>(tk);
    const typename SpVec<T>::Range part(zt, top);
#pragma unroll 1
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      double mine = 0.0;
      if (v < s.nvec && part.any(slice[v]))
        s.template each<1>(v, [&](float z, int idx) {
          if (!(z >= zt && z <= top && z >= zcut) || (z == zt && idx > ti) || (N != 8 && s.bin(z) != b) || !s.left(z, idx)) return;
          mine += s.weight(z);
          ++kept;
        });
      if (!__any_sync(FULL, mine > 0.0)) continue;
      mine = warp_sum_d(mine);
      if (lane == 0) wsum[st] += mine;
    }
    // from here on `left` is the final cut
    s.ci = s.cut && tk == s.ck ? min(ti, s.ci) : ti;
    s.ck = tk;
    s.cut = true;
    break;
  }
  const double kk = sp_block_sum((double)kept);                              // also orders the stretches' sums before their use
  // E: the slices' masses, the slice, the stretch, the element
  const int q = (nst + 31) / 32;                // stretches a lane of the first warp
  double lane_sum = 0.0, lane_inc = 0.0;
  if (warp == 0) {
#pragma unroll 1
    for (int j = lane * q; j < min(nst, (lane + 1) * q); ++j) lane_sum += wsum[j];
    lane_inc = sp_warp_scan(lane_sum);
    if (lane == 31) sh.found[2] = lane_inc;
  }
  __syncthreads();
  double mass = 0.0, before = 0.0, chosen_before = 0.0;
  double kept_all = 0.0;
  int chosen = -1;
  s.exchange(sh.found[2], kk);
#pragma unroll 1
  for (int r = 0; r < s.C; ++r) {
    mass += s.got_d(r, 0);
    kept_all += s.got_d(r, 1);
  }
  // the first slice whose running sum passes u of the total (else, by rounding, the last with mass)
#pragma unroll 1
  for (int r = 0; r < s.C; ++r) {
    const double m = s.got_d(r, 0);
    if (m > 0.0 && (chosen < 0 || chosen_before + s.got_d(chosen, 0) <= (double)u * mass)) {
      chosen = r;
      chosen_before = before;
    }
    before += m;
  }
  const double goal = (double)u * mass;
  if (s.rank == chosen && warp == 0) {
    // the stretch whose running sum passes the goal, or the last one with mass
    const unsigned hit = __ballot_sync(FULL, chosen_before + lane_inc > goal && lane_sum > 0.0);
    const unsigned any = __ballot_sync(FULL, lane_sum > 0.0);
    const int l = hit ? __ffs(hit) - 1 : 31 - __clz(any);
    double run = chosen_before + __shfl_sync(FULL, lane_inc - lane_sum, l);
    int st = -1;
    double st_run = 0.0;
#pragma unroll 1
    for (int j = l * q; j < min(nst, (l + 1) * q); ++j) {
      const double w = wsum[j];
      if (w > 0.0) {
        st = j;
        st_run = run;
        if (run + w > goal) break;
      }
      run += w;
    }
    const int v = st * 32 + lane;
    double mine = 0.0;
    auto mass_of = [&](float z, int idx) { return s.left(z, idx) && z >= zcut ? s.weight(z) : 0.0; };
    if (v < s.nvec) s.template each<1>(v, [&](float z, int idx) { mine += mass_of(z, idx); });
    const double inc = sp_warp_scan(mine);
    const unsigned hit2 = __ballot_sync(FULL, st_run + inc > goal && mine > 0.0);
    const unsigned any2 = __ballot_sync(FULL, mine > 0.0);
    const int l2 = hit2 ? __ffs(hit2) - 1 : 31 - __clz(any2);
    if (lane == l2) {
      double r2 = st_run + inc - mine, tw = 1.0;
      int tok = -1;
      s.template each<1>(v, [&](float z, int idx) {
        const double w = mass_of(z, idx);
        if (w > 0.0 && (tok < 0 || r2 <= goal)) {
          tok = idx;
          tw = w;
        }
        r2 += w;
      });
      p.token[row] = tok;
      if (p.logprob) p.logprob[row] = (float)log(tw / mass);
      if (p.kept) p.kept[row] = (int)kept_all;
    }
  }
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  const int es = p.bf16 ? 2 : 4, vn = 16 / es;
  // the cluster.  Few rows: slices down to 4096, for short passes, up to 16 CTAs a row (more than 8 need
  // the non-portable size) while all rows fit the GPU at once.  Many rows: slices of up to 40960, two
  // CTAs an SM, so that a search's barriers are paid by fewer CTAs
  const int64_t n = p.n;
  const int most = n * 8 > 4 * num_sms() ? 40960 : 16384;
  int C = 1;
  while (C < 8 && (p.V + C - 1) / C > most) C <<= 1;
  while (C < SP_MAXC && p.V / C > 4096 && n * 2 * C <= num_sms()) C <<= 1;
  const int unit = 32 * vn;
  const int per = ((p.V + C - 1) / C + unit - 1) / unit * unit;
  const size_t smem = sizeof(SpShared) + (size_t)per * es + (size_t)(per / unit) * sizeof(double);
  const bool aligned = (uintptr_t)p.logits % 16 == 0 && (p.n == 1 || p.row_stride * es % 16 == 0);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(n * C));
  cfg.blockDim = dim3(SP_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  auto go = [&](auto kern) {
    cudaError_t e = allow_smem(kern);
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, p, per);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (p.bf16) return aligned ? go(sample_kernel<__nv_bfloat16, true>) : go(sample_kernel<__nv_bfloat16, false>);
  return aligned ? go(sample_kernel<float, true>) : go(sample_kernel<float, false>);
}

}  // namespace kvc
