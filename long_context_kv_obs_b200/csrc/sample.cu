// Token sampling: temperature, top-k, top-p, min-p and one given random number a row.
//
// Which tokens stay is decided on the row's order (logit down, index up): each filter keeps a
// head of it, so the outcome is one cut (key, index), and the token is found where the kept
// mass, summed in index order, passes u times its total.  No sort of the row.
//
// Masses.  A vocabulary of 10^5 flat probabilities puts borders 10^-5 apart, so fp32 sums
// (errors near 10^-7) would move a border once in a hundred rows.  Weights are formed in fp64:
// 2^t with t = (z - max) log2(e) / T split as t = k / 64 + f, |f| <= 1/128; 2^(k mod 64 / 64) from a
// table that the CUDA function exp2 fills, 2^f by the Taylor series of exp(f ln 2) to degree 4
// (relative error below 4e-14), and the exponent added.  Weights below 2^-64 of the largest count
// as nothing: all of them together are below 2^-46 of the mass.  Sums run in a fixed order.
//
// A row is a cluster of CTAs, each with a slice of it in shared memory, read from HBM once.
//   A  the maximum
//   B  top-k, few: the k-th largest of the threads' own maxima is a bound that k elements reach; what
//      reaches it goes to one CTA, which sorts it, sums it in that order for top-p, and again in
//      index order for the token
//   C  else the cut is searched: counts (top-k) or masses (top-p) by bins of 1/8 octave of weight below
//      the maximum (shared-memory integer atomics: order does not matter), summed over the
//      cluster through distributed shared memory; the bin that holds the border is searched
//      again by ranges of the key, until one key is left; of its ties the lowest indices stay.
//      512 bins: every CTA reads all histograms of the cluster, which at 2048 bins and 16 CTAs took
//      9.8k cycles.  Tokens whose weight is below (1 - top_p) of the mean are left out of the first
//      search of masses: together they hold less than the 1 - top_p that is cut.  Its bins hold
//      masses to 16 bits only: the exact sums of D decide whether the bin is the right one (else its
//      neighbour is taken), the later searches count in 2^-31 units of the bin's weights, or
//      exactly once a bin is one key.
//   D  fp64 sums of the kept weights by 32-vector stretches of a warp, in index order
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
constexpr int SP_MAXC = 16;
constexpr int SP_LIST = 4096;                   // candidates that one CTA sorts
constexpr float SP_ONE = 8388608.f;             // 2^23: adding it leaves the rounded integer in a float's low bits

struct alignas(16) SpShared {                   // the slice follows: its vectors are 16-byte aligned
  union {
    unsigned hist[2][2 * SP_BINS];              // two searches deep: counts or masses; two 16-bit limbs of a mass
    unsigned long long list[SP_LIST];
  };
  double table[64];                             // 2^(j / 64)
  double part[2];                               // beside a histogram: the mass of the slice, to fp32
  unsigned long long xch[2][SP_MAXC][4];        // values of every CTA of the cluster, two steps deep
  unsigned long long red[SP_WARPS][4];
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
};
template <> struct SpVec<float> {
  static constexpr int N = 4, KSHIFT = 0;
  __device__ __forceinline__ static uint4 clean(uint4 u) {
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]), -INFINITY) + 0.f);
    return u;
  }
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

// Sum of N values, pairwise.
template <int N>
__device__ __forceinline__ double sp_tree(const double (&v)[N]) {
  double a[N];
#pragma unroll
  for (int j = 0; j < N; ++j) a[j] = v[j];
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1)
#pragma unroll
    for (int j = 0; j < h; ++j) a[j] = a[2 * j] + a[2 * j + 1];
  return a[0];
}

template <typename T>
struct SpRow {
  static constexpr int N = SpVec<T>::N, KS = SpVec<T>::KSHIFT;
  cg::cluster_group cl;
  SpShared& sh;
  uint4* slice;                                 // this CTA's vectors; thread t owns t, t + SP_THREADS, ...
  double* wsum;                                 // kept mass of every 32-vector stretch
  int C, rank, nvec, i0;                        // cluster size, rank, vectors of the slice, its first index
  int step, search;
  float zmax, ybin;                             // bins below the maximum: (zmax - z) * ybin
  float zlow;                                   // weights below this one's, 2^-64 of the largest, are nothing
  double c;                                     // log2(e) / T
  bool cut;                                     // top-k left: key > ck, or key == ck and index <= ci
  uint32_t ck;
  int ci;

  __device__ __forceinline__ SpRow(SpShared& s) : cl(cg::this_cluster()), sh(s) {}

  // The values v of every CTA, which all its threads know: each CTA writes its own into every other's
  // shared memory (a store does not wait), and after the cluster barrier the reads are local.  A slot
  // is written again two steps later: by then its reader has passed the barrier between.
  template <int K, typename F>
  __device__ __forceinline__ void exchange(const unsigned long long (&v)[K], F&& use) {
    if ((int)threadIdx.x < C) {
      unsigned long long* o = cl.map_shared_rank(&sh.xch[step & 1][rank][0], threadIdx.x);
#pragma unroll
      for (int k = 0; k < K; ++k) o[k] = v[k];
    }
    cl.sync();
    for (int r = 0; r < C; ++r) {
      unsigned long long w[K];
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = sh.xch[step & 1][r][k];
      use(r, w);
    }
    ++step;
  }
  // Sums over the CTA, in a fixed order, known to every thread.
  template <int K, typename V>
  __device__ __forceinline__ void block_sum(V (&v)[K]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(FULL, v[k], o);
    }
    __syncthreads();
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) *reinterpret_cast<V*>(&sh.red[warp][k]) = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      V s = *reinterpret_cast<V*>(&sh.red[lane & (SP_WARPS - 1)][k]);
#pragma unroll
      for (int o = SP_WARPS / 2; o > 0; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
      v[k] = s;
    }
  }

  __device__ __forceinline__ void unpack(int v, float (&z)[N]) const { Vec<T>::unpack(slice[v], z); }
  // Monotone in z; the maximum is in bin 0, the last bin holds all that is farther.
  __device__ __forceinline__ int bin(float z) const {
    const float r = fmaf(zmax - z, ybin, SP_ONE);
    return min(__float_as_int(r) - 0x4B000000, SP_BINS - 1);
  }
  // For z >= zlow: weights of the others are nothing.
  __device__ __forceinline__ double raw_weight(float z) const {
    const double t = ((double)z - (double)zmax) * c;
    const double magic = 6755399441055744.0 / 64;   // 1.5 * 2^52 / 64: rounds t to a multiple of 1/64
    const double r = t + magic;
    const int k = __double2loint(r);
    const double f = t - (r - magic);
    // exp(f ln 2) = 1 + f ln2 + (f ln2)^2 / 2 + (f ln2)^3 / 6 + (f ln2)^4 / 24
    double p = fma(f, 9.618129107628477e-3, 5.550410866482158e-2);
    p = fma(f, p, 2.402265069591007e-1);
    p = fma(f, p, 6.931471805599453e-1);
    p = fma(f, p, 1.0);
    p *= sh.table[k & 63];
    return __hiloint2double(__double2hiint(p) + ((k >> 6) << 20), __double2loint(p));
  }
  __device__ __forceinline__ double weight(float z) const { return z >= zlow ? raw_weight(z) : 0.0; }
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

  // The histogram of this search, cleared for use (its words are used again two searches on).
  __device__ __forceinline__ unsigned* clear_hist(int words) {
    unsigned* h = sh.hist[search & 1];
    for (int j = threadIdx.x; j < words / 4; j += SP_THREADS) reinterpret_cast<uint4*>(h)[j] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    return h;
  }
  // The first bin at which the sum over the cluster's histograms reaches `target` (frac > 0: that
  // share of the cluster's `part`), or the last that holds something; the sum before it and the bin's
  // own value.  A bin's value is val(bin, words summed over the cluster); LIMBS: the histogram has a
  // second half, 2^16 times the first's unit.  Every CTA reads all histograms (a thread one bin, its
  // loads all in flight) and scans them for itself: one cluster barrier a search.  The next search
  // uses the other buffer, so a slow reader is not overtaken.
  template <bool LIMBS, typename F>
  __device__ __forceinline__ void border(double frac, double target, F&& val, int& b, double& above, double& value) {
    static_assert(SP_BINS == SP_THREADS, "a bin a thread");
    cl.sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long h = 0;
#pragma unroll 8
    for (int r = 0; r < C; ++r) {
      const unsigned* o = cl.map_shared_rank(&sh.hist[search & 1][0], r);
      h += o[threadIdx.x];
      if (LIMBS) h += (unsigned long long)o[SP_BINS + threadIdx.x] << 16;
    }
    if (frac > 0.0 && warp == 0) {
      double m = lane < C ? *cl.map_shared_rank(&sh.part[search & 1], lane) : 0.0;
      m = warp_sum_d(m);
      if (lane == 0) sh.found[3] = frac * m;
    }
    ++search;
    const double v = h ? val((int)threadIdx.x, (double)h) : 0.0;
    double inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) *reinterpret_cast<double*>(&sh.red[warp][0]) = inc;
    __syncthreads();
    if (frac > 0.0) target = sh.found[3];
    // sum of the warps before (lanes 0 .. 15 hold the warps' sums)
    double before = (lane & (SP_WARPS - 1)) < warp ? *reinterpret_cast<double*>(&sh.red[lane & (SP_WARPS - 1)][0]) : 0.0;
#pragma unroll
    for (int o = SP_WARPS / 2; o > 0; o >>= 1) before += __shfl_xor_sync(FULL, before, o);
    const unsigned some = __ballot_sync(FULL, v > 0.0);
    const unsigned hit = __ballot_sync(FULL, v > 0.0 && before + inc >= target);
    if (lane == 0) {
      sh.cand[warp][0] = hit ? warp * 32 + __ffs(hit) - 1 : INT_MAX;
      sh.cand[warp][1] = some ? warp * 32 + 31 - __clz(some) : -1;
    }
    __syncthreads();
    const int at = __reduce_min_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][0]);
    const int end = __reduce_max_sync(FULL, sh.cand[lane & (SP_WARPS - 1)][1]);
    b = at == INT_MAX ? max(end, 0) : at;
    if ((int)threadIdx.x == b) {
      sh.found[0] = before + inc - v;
      sh.found[1] = v;
    }
    __syncthreads();
    above = sh.found[0];
    value = sh.found[1];
  }

  // use(value, index) for every element of the slice with lo <= value <= hi; they are few
  template <typename F>
  __device__ __forceinline__ void in_range(float lo, float hi, F&& use) {
    for (int v = threadIdx.x; v < nvec; v += SP_THREADS) {
      float z[N];
      unpack(v, z);
      unsigned in = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) in |= (z[j] >= lo && z[j] <= hi ? 1u : 0u) << j;
      while (in) {
        const int j = __ffs(in) - 1;
        in &= in - 1;
        use((float)reinterpret_cast<const T*>(slice + v)[j], i0 + v * N + j);
      }
    }
  }

  // Within bin b0 (of the tokens left by top-k), the key at which the count (MASS: the mass, in units
  // of 2^-(31 + e)) reaches `need`, and the index of the last tie that stays.  False if the bin holds
  // less than that (then nothing else is set).
  template <bool MASS>
  __device__ __forceinline__ bool refine(int b0, double need, int e, uint32_t& tkey, int& tidx) {
    uint32_t hi = sp_key(edge_high(b0), KS), lo = max(sp_key(edge_low(b0), KS), sp_key(-INFINITY, KS) + 1u);
    double above = 0.0, value = 0.0;
    bool first_search = true;
    int shift = 0;
    while (((hi - lo) >> shift) >= SP_BINS) ++shift;
    while (true) {
      const bool limbs = MASS && shift > 0;
      unsigned* hist = clear_hist(limbs ? 2 * SP_BINS : SP_BINS);
      in_range(sp_value<KS>(lo), sp_value<KS>(hi), [&](float z, int idx) {
        if (bin(z) != b0 || !left(z, idx)) return;
        const uint32_t hb = (hi - sp_key(z, KS)) >> shift;
        if (limbs) {
          const unsigned long long q = (unsigned long long)__double2ll_rn(scalbn(weight(z), 31 + e));
          atomicAdd(hist + hb, (unsigned)(q & 0xffffu));
          atomicAdd(hist + SP_BINS + hb, (unsigned)(q >> 16));
        } else {
          atomicAdd(hist + hb, 1u);
        }
      });
      int hb;
      double ab;
      if (limbs) {
        border<true>(0.0, need - above, [](int, double n) { return n; }, hb, ab, value);
      } else if (MASS) {                        // a bin is one key: its weight times its count
        const uint32_t first = hi;
        border<false>(0.0, need - above,
                      [&](int i, double n) { return n * scalbn(weight(sp_value<KS>(first - (uint32_t)i)), 31 + e); }, hb, ab,
                      value);
      } else {
        border<false>(0.0, need - above, [](int, double n) { return n; }, hb, ab, value);
      }
      if (MASS && first_search && ab + value < need) return false;
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
    if (MASS) {
      const double w = scalbn(weight(sp_value<KS>(tkey)), 31 + e);
      take = w > 0.0 ? ceil(take / w) : 1.0;
      ties = w > 0.0 ? rint(value / w) : 1.0;
    }
    if (take < 1.0) take = 1.0;
    tidx = INT_MAX;
    if (take >= ties) return true;
    // ties of every 32-vector stretch, in the histogram words of the next search
    const int lane = threadIdx.x & 31, nst = (nvec + 31) / 32;
    const float zt = sp_value<KS>(tkey);
    unsigned* count = sh.hist[search & 1];
    int mine[1] = {0};
    for (int v0 = threadIdx.x - lane; v0 < nvec; v0 += SP_THREADS) {
      const int v = v0 + lane;
      int n = 0;
      if (v < nvec) {
        float z[N];
        unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) n += z[j] == zt && left(z[j], i0 + v * N + j);
      }
      n = __reduce_add_sync(FULL, n);
      if (lane == 0) {
        count[v0 >> 5] = (unsigned)n;
        mine[0] += n;
      }
    }
    block_sum<1>(mine);
    double before = 0.0;
    {
      unsigned long long x[1] = {(unsigned long long)mine[0]};
      exchange<1>(x, [&](int r, unsigned long long (&w)[1]) { before += r < rank ? (double)w[0] : 0.0; });
    }
    const bool here = before < take && take <= before + (double)mine[0];
    if (here && threadIdx.x < 32) {             // this slice holds the last tie that stays
      int want = (int)(take - before), st = 0;
      for (int s0 = 0; s0 < nst; s0 += 32) {
        const int n = s0 + lane < nst ? (int)count[s0 + lane] : 0;
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(FULL, inc, d);
          if (lane >= d) inc += y;
        }
        const unsigned hit = __ballot_sync(FULL, inc >= want);
        if (hit) {
          st = s0 + __ffs(hit) - 1;
          want -= __shfl_sync(FULL, inc - n, __ffs(hit) - 1);
          break;
        }
        want -= __shfl_sync(FULL, inc, 31);
      }
      const int v = st * 32 + lane;
      unsigned in = 0;
      if (v < nvec) {
        float z[N];
        unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) in |= (z[j] == zt && left(z[j], i0 + v * N + j) ? 1u : 0u) << j;
      }
      int inc = __popc(in);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(FULL, inc, d);
        if (lane >= d) inc += y;
      }
      int k = inc - __popc(in);
      while (in) {
        const int j = __ffs(in) - 1;
        in &= in - 1;
        if (++k == want) sh.ifound[1] = i0 + v * N + j;
      }
    }
    __syncthreads();
    unsigned long long y[1] = {(unsigned long long)(here ? sh.ifound[1] + 1 : 0)};
    int at = 0;
    exchange<1>(y, [&](int, unsigned long long (&w)[1]) { at = max(at, (int)w[0]); });
    tidx = at - 1;
    return true;
  }
};

// a[0, n) sorted downwards, n a power of two (bitonic merges).
__device__ __forceinline__ void sp_sort(unsigned long long* a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
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
  extern __shared__ __align__(16) uint8_t sp_raw[];
  SpShared& sh = *reinterpret_cast<SpShared*>(sp_raw);
  uint4* slice = reinterpret_cast<uint4*>(sp_raw + sizeof(SpShared));
  SpRow<T> s(sh);
  s.cl.barrier_arrive();                        // every CTA of the cluster runs before its shared memory is written
  s.C = (int)s.cl.num_blocks();
  s.rank = (int)s.cl.block_rank();
  const int row = blockIdx.x / s.C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  s.slice = slice;
  s.wsum = reinterpret_cast<double*>(slice + per_cta / N);
  s.i0 = s.rank * per_cta;
  s.nvec = max(0, min(per_cta, p.V - s.i0) + N - 1) / N;
  s.step = s.search = 0;
  s.cut = false;
  const T* z0 = reinterpret_cast<const T*>(p.logits) + row * p.row_stride;

  // A: the slice into shared memory and the maximum
  float best = -INFINITY;
#pragma unroll 4
  for (int v = tid; v < s.nvec; v += SP_THREADS) {
    const uint4 u = SpVec<T>::clean(sp_load<T, ALIGNED>(z0, s.i0 + (int64_t)v * N, p.V));
    slice[v] = u;
    float z[N];
    Vec<T>::unpack(u, z);
#pragma unroll
    for (int j = 0; j < N; ++j) best = fmaxf(best, z[j]);
  }
  if (tid < 64) sh.table[tid] = exp2((double)tid / 64.0);
  const float T_ = p.temperature ? p.temperature[row] : 1.f;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float pf = p.top_p ? p.top_p[row] : 1.f, mf = p.min_p ? p.min_p[row] : 0.f;
  {
    const float m = warp_max(best);
    if (lane == 0) sh.red[warp][0] = f2key(m);
    __syncthreads();
    unsigned long long x[1] = {0};
#pragma unroll
    for (int w = 0; w < SP_WARPS; ++w) x[0] = max(x[0], sh.red[w][0]);
    s.cl.barrier_wait();
    unsigned long long top = 0;
    s.exchange(x, [&](int, unsigned long long (&w)[1]) { top = max(top, w[0]); });
    s.zmax = key2f((uint32_t)top);
  }
  if (s.zmax == -INFINITY || !(T_ > 0.f)) {
    // nothing to take, or the first token of the order
    int at = INT_MAX;
    if (s.zmax > -INFINITY)
      s.in_range(s.zmax, s.zmax, [&](float, int idx) { at = min(at, idx); });
    at = __reduce_min_sync(FULL, at);
    __syncthreads();
    if (lane == 0) sh.red[warp][0] = (unsigned long long)at;
    __syncthreads();
    unsigned long long x[1] = {INT_MAX};
#pragma unroll
    for (int w = 0; w < SP_WARPS; ++w) x[0] = min(x[0], sh.red[w][0]);
    unsigned long long first = INT_MAX;
    s.exchange(x, [&](int, unsigned long long (&w)[1]) { first = min(first, w[0]); });
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
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      T* e = reinterpret_cast<T*>(slice + v);
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = (float)e[j] == INFINITY ? T(0.f) : T(-INFINITY);
    }
    best = best == INFINITY ? 0.f : -INFINITY;
    s.zmax = 0.f;
  }
  s.c = 1.4426950408889634 / (double)T_;
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
    const double x = (double)s.zmax + (mf < 1.f ? (double)T_ * log((double)mf) : 0.0);
    zcut = x > -3.4028234663852886e38 ? __double2float_ru(x) : -INFINITY;
  }
  float u = p.u[row];
  u = u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f;   // NaN and negatives: 0

  if (k > 0 && k < p.V) {
    double above, value;
    auto number = [](int, double n) { return n; };
    if (k <= s.C * (SP_THREADS / 4)) {
      // B: a bin that the k-th largest cannot lie beyond, from the threads' own maxima
      unsigned* hist = s.clear_hist(SP_BINS);
      if (best > -INFINITY) atomicAdd(hist + s.bin(best), 1u);
      int far;
      s.template border<false>(0.0, (double)k, number, far, above, value);
      const float low = above + value >= (double)k ? s.edge_low(far) : -INFINITY;
      const float floor_ = fmaxf(low, -3.4028234663852886e38f);   // never -infinity itself
      // what reaches it, first counted
      int n[1] = {0};
      s.in_range(floor_, INFINITY, [&](float, int) { ++n[0]; });
      s.block_sum(n);
      unsigned long long x[1] = {(unsigned long long)n[0]};
      int off = 0, m = 0;
      s.exchange(x, [&](int r, unsigned long long (&w)[1]) {
        off += r < s.rank ? (int)w[0] : 0;
        m += (int)w[0];
      });
      if (m <= SP_LIST) {
        // the candidates, to the first CTA (its histograms are read no more: all have passed the exchange)
        if (tid == 0) sh.nlist = off;
        __syncthreads();
        unsigned long long* list = s.cl.map_shared_rank(&sh.list[0], 0);
        s.in_range(floor_, INFINITY, [&](float z, int idx) {
          list[atomicAdd(&sh.nlist, 1)] = ((unsigned long long)f2key(z) << 32) | (unsigned)~idx;
        });
        s.cl.sync();
        if (s.rank != 0) return;                // the rest is the first CTA's own
        int np = 2;
        while (np < m) np <<= 1;
        for (int i = m + tid; i < np; i += SP_THREADS) sh.list[i] = 0ull;
        sp_sort(sh.list, np);
        const int kk = min(k, m);
        // weights in the order, eight a thread, and their running sum
        constexpr int Q = SP_LIST / SP_THREADS;
        double w[Q], sum = 0.0;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const int i = tid * Q + j;
          w[j] = i < kk ? s.weight(key2f((uint32_t)(sh.list[i] >> 32))) : 0.0;
          sum += w[j];
        }
        auto scan = [&](double mine, double& total) {   // sum of the threads before
          double inc = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const double y = __shfl_up_sync(FULL, inc, d);
            if (lane >= d) inc += y;
          }
          __syncthreads();
          if (lane == 31) *reinterpret_cast<double*>(&sh.red[warp][0]) = inc;
          __syncthreads();
          double b = 0.0;
          total = 0.0;
#pragma unroll
          for (int q = 0; q < SP_WARPS; ++q) {
            const double y = *reinterpret_cast<double*>(&sh.red[q][0]);
            b += q < warp ? y : 0.0;
            total += y;
          }
          return b + inc - mine;
        };
        double total;
        double run = scan(sum, total);
        int keep[1] = {0};
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const int i = tid * Q + j;
          if (i < kk) {
            const bool in = i == 0 || ((!use_p || run < top_p * total) && key2f((uint32_t)(sh.list[i] >> 32)) >= zcut);
            keep[0] += in;                      // a head of the order: both conditions only turn false
          }
          run += w[j];
        }
        s.block_sum(keep);
        // the kept ones in index order
        int nk = 2;
        while (nk < keep[0]) nk <<= 1;
        for (int i = tid; i < nk; i += SP_THREADS) {
          const unsigned long long x = sh.list[i];
          // sorted downwards: index up is ~index down; what is cut sinks
          sh.list[i] = i < keep[0] ? (x << 32) | (x >> 32) : 0ull;
        }
        sp_sort(sh.list, nk);
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const int i = tid * Q + j;
          w[j] = i < keep[0] ? s.weight(key2f((uint32_t)sh.list[i])) : 0.0;
          sum += w[j];
        }
        run = scan(sum, total);
        const double goal = (double)u * total;
        // the first whose running sum passes the goal (else, by rounding, the last with mass)
        int at = INT_MAX, last = -1;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          if (w[j] > 0.0) {
            last = tid * Q + j;
            if (at == INT_MAX && run + w[j] > goal) at = last;
          }
          run += w[j];
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
          if (p.logprob) p.logprob[row] = (float)log(s.weight(key2f((uint32_t)x)) / total);
          if (p.kept) p.kept[row] = keep[0];
        }
        return;
      }
    }
    // C: the k-th key by counts
    unsigned* hist = s.clear_hist(SP_BINS);
    int have[1] = {0};
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      float z[N];
      s.unpack(v, z);
      int run = 0, rb = -1;                     // equal neighbours in one atomic
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (!(z[j] > -INFINITY)) continue;
        ++have[0];
        const int bb = s.bin(z[j]);
        if (bb != rb) {
          if (run) atomicAdd(hist + rb, (unsigned)run);
          rb = bb;
          run = 0;
        }
        ++run;
      }
      if (run) atomicAdd(hist + rb, (unsigned)run);
    }
    s.block_sum(have);
    int total = 0;
    unsigned long long x[1] = {(unsigned long long)have[0]};
    s.exchange(x, [&](int, unsigned long long (&w)[1]) { total += (int)w[0]; });
    if (k < total) {
      int b, ti;
      uint32_t tk;
      s.template border<false>(0.0, (double)k, number, b, above, value);
      s.template refine<false>(b, (double)k - above, 0, tk, ti);
      s.cut = true;
      s.ck = tk;
      s.ci = ti;
    }
  }

  int b = SP_BINS;                              // top-p: kept are the bins before b and a part of b
  double above = 0.0;
  if (use_p && pf > 0.f) {
    // C: the slice's mass to fp32.  The whole row's is no smaller, so what is below (1 - top_p) of it
    // over V is below (1 - top_p) of the mean, and each CTA knows by itself what to leave out
    float part = 0.f;
    const float scale = s.ybin * (-1.f / 8.f);
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      float z[N];
      s.unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j) part += s.left(z[j], s.i0 + v * N + j) ? tc::ex2((s.zmax - z[j]) * scale) : 0.f;
    }
    double about[1] = {(double)part};
    s.block_sum(about);
    if (tid == 0) sh.part[s.search & 1] = about[0];
    const float mean = (float)(0.99 * (1.0 - top_p) * about[0] / p.V);
    // bins up to this one; the last bin is below 2^-63 of the maximum
    const int far = mean > 0.f ? min((int)(-8.f * log2f(mean)) + 1, SP_BINS - 2) : SP_BINS - 2;
    const float low = s.edge_low(far);
    unsigned* hist = s.clear_hist(SP_BINS);
    for (int v = tid; v < s.nvec; v += SP_THREADS) {
      float z[N];
      s.unpack(v, z);
      unsigned run = 0;                         // equal neighbours in one atomic
      int rb = -1;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (!(z[j] >= low) || !s.left(z[j], s.i0 + v * N + j)) continue;
        const float d = s.zmax - z[j], r = fmaf(d, s.ybin, SP_ONE);
        const int bb = __float_as_int(r) - 0x4B000000;
        if (bb > far) continue;
        if (bb != rb) {
          if (run) atomicAdd(hist + rb, run);
          rb = bb;
          run = 0;
        }
        // 2^-(distance from the bin's middle, in eighths), below 1.045, in 2^-15 units
        const float y = fmaf(d, s.ybin, SP_ONE - r);
        run += (unsigned)__float_as_int(fmaf(tc::ex2(y * (-1.f / 8.f)), 32768.f, SP_ONE)) - 0x4B000000u;
      }
      if (run) atomicAdd(hist + rb, run);
    }
    double value;
    s.template border<false>(top_p, 0.0,
                             [](int i, double n) { return n * (double)exp2f((float)i * (-1.f / 8.f)) * 0x1p-15; }, b,
                             above, value);
  } else if (use_p) {
    b = 0;                                      // top_p <= 0: one token
  }
  // D: the kept mass by stretches of 32 vectors
  const int nst = (s.nvec + 31) / 32;
  int kept = 0;
  for (int moved = 0;;) {
    double sums[2] = {0.0, 0.0};                // all that is left, bins before b
    const float rb = SP_ONE + (float)b;         // bin(z) < b  <=>  fma(zmax - z, ybin, 2^23) < 2^23 + b
    kept = 0;
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      double mine = 0.0;
      if (v < s.nvec) {
        float z[N];
        double w[N];
        s.unpack(v, z);
        unsigned head = 0;                      // kept for certain: in bins before b, above the min-p cut
#pragma unroll
        for (int j = 0; j < N; ++j) {           // no branches: the chains of the N weights interleave
          const bool in = s.left(z[j], s.i0 + v * N + j), some = in && z[j] >= s.zlow;
          const double x = s.raw_weight(some ? z[j] : s.zmax);
          w[j] = some ? x : 0.0;
          const bool before = fmaf(s.zmax - z[j], s.ybin, SP_ONE) < rb || !use_p;
          head |= (in && before && z[j] >= zcut ? 1u : 0u) << j;
          if (use_p) sums[1] += before ? w[j] : 0.0;
        }
        if (use_p) sums[0] += sp_tree<N>(w);
        kept += __popc(head);
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = (head >> j) & 1u ? w[j] : 0.0;
        mine = sp_tree<N>(w);
      }
      mine = warp_sum_d(mine);
      if (lane == 0) s.wsum[st] = mine;
    }
    if (!use_p) break;
    s.block_sum(sums);
    unsigned long long x[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) x[q] = (unsigned long long)__double_as_longlong(sums[q]);
    double total = 0.0;
    above = 0.0;
    s.exchange(x, [&](int, unsigned long long (&w)[2]) {
      total += __longlong_as_double((long long)w[0]);
      above += __longlong_as_double((long long)w[1]);
    });
    // the bin is right if the sum reaches top_p of the total inside it (b == 0: it starts there)
    const double goal = pf > 0.f ? top_p * total : 0.0;
    if (above >= goal && b > 0 && moved <= 0) {
      --b;
      moved = -1;
      continue;
    }
    // the bin's weights lie within 2^(-(b +- 1/2) / 8) of the maximum: scaled by 2^e they are at most 2^(1/16)
    const int e = b / 8;
    uint32_t tk;
    int ti;
    if (!s.template refine<true>(b, fmax(ldexp(goal - above, 31 + e), 0.0), e, tk, ti)) {
      if (moved >= 0 && b < SP_BINS - 2) {
        ++b;
        moved = 1;
        continue;
      }
      // between two bins by the sums' last bits: all of this one stays
      tk = sp_key(s.edge_low(b), KS);
      ti = INT_MAX;
    }
    // the part of bin b that stays
    const float zt = sp_value<KS>(tk), top = s.edge_high(b);
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      unsigned in = 0;
      float z[N];
      if (v < s.nvec) {
        s.unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) in |= (z[j] >= zt && z[j] <= top && z[j] >= zcut ? 1u : 0u) << j;
      }
      if (!__any_sync(FULL, in != 0)) continue;
      double mine = 0.0;
      if (in) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int idx = s.i0 + v * N + j;
          if (!((in >> j) & 1u) || (z[j] == zt && idx > ti) || s.bin(z[j]) != b || !s.left(z[j], idx)) continue;
          mine += s.weight(z[j]);
          ++kept;
        }
      }
      mine = warp_sum_d(mine);
      if (lane == 0) s.wsum[st] += mine;
    }
    // from here on `left` is the final cut
    s.ci = s.cut && tk == s.ck ? min(ti, s.ci) : ti;
    s.ck = tk;
    s.cut = true;
    break;
  }
  int kk[1] = {kept};
  s.block_sum(kk);                              // also orders the stretches' sums before their use
  // E: the slices' masses, the slice, the stretch, the element
  const int q = (nst + 31) / 32;                // stretches a lane of the first warp
  double lane_sum = 0.0, lane_inc = 0.0;
  if (warp == 0) {
    for (int j = lane * q; j < min(nst, (lane + 1) * q); ++j) lane_sum += s.wsum[j];
    lane_inc = lane_sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, lane_inc, d);
      if (lane >= d) lane_inc += y;
    }
    if (lane == 31) sh.found[2] = lane_inc;
  }
  __syncthreads();
  double mass = 0.0, before = 0.0, chosen_before = 0.0;
  int chosen = -1, kept_all = 0;
  {
    // twice over the slices' masses: the total, then the first slice whose running sum passes u of it
    unsigned long long x[2] = {(unsigned long long)__double_as_longlong(sh.found[2]), (unsigned long long)kk[0]};
    s.exchange(x, [&](int, unsigned long long (&w)[2]) {
      mass += __longlong_as_double((long long)w[0]);
      kept_all += (int)w[1];
    });
    for (int r = 0; r < s.C; ++r) {
      const double m = __longlong_as_double((long long)sh.xch[(s.step - 1) & 1][r][0]);
      if (m > 0.0 && (chosen < 0 || chosen_before + __longlong_as_double((long long)sh.xch[(s.step - 1) & 1][chosen][0]) <=
                                        (double)u * mass)) {
        chosen = r;                             // (else, by rounding, the last slice with mass)
        chosen_before = before;
      }
      before += m;
    }
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
    for (int j = l * q; j < min(nst, (l + 1) * q); ++j) {
      const double w = s.wsum[j];
      if (w > 0.0) {
        st = j;
        st_run = run;
        if (run + w > goal) break;
      }
      run += w;
    }
    const int v = st * 32 + lane;
    double w[N], mine = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] = 0.0;
    if (v < s.nvec) {
      float z[N];
      s.unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (s.left(z[j], s.i0 + v * N + j) && z[j] >= zcut) w[j] = s.weight(z[j]);
        mine += w[j];
      }
    }
    double inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned hit2 = __ballot_sync(FULL, st_run + inc > goal && mine > 0.0);
    const unsigned any2 = __ballot_sync(FULL, mine > 0.0);
    const int l2 = hit2 ? __ffs(hit2) - 1 : 31 - __clz(any2);
    if (lane == l2) {
      double r2 = st_run + inc - mine;
      int tok = -1;
      double tw = 1.0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (w[j] > 0.0 && (tok < 0 || r2 <= goal)) {
          tok = s.i0 + v * N + j;
          tw = w[j];
        }
        r2 += w[j];
      }
      p.token[row] = tok;
      if (p.logprob) p.logprob[row] = (float)log(tw / mass);
      if (p.kept) p.kept[row] = kept_all;
    }
  }
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  const int es = p.bf16 ? 2 : 4, vn = 16 / es;
  // the cluster.  Few rows: short slices, for short passes, up to 16 CTAs a row (more than 8 need the
  // non-portable size) while all rows fit the GPU at once.  Many rows: slices of up to 40960, two
  // CTAs an SM, so that a search's barriers are paid by fewer CTAs
  const bool many = p.n * 8 > 4 * num_sms();
  const int most = many ? 40960 : 16384;
  int C = 1;
  while (C < 8 && (p.V + C - 1) / C > most) C <<= 1;
  if (C == 8 && p.n * 16 <= num_sms()) C = 16;
  const int unit = 32 * vn;
  const int per = ((p.V + C - 1) / C + unit - 1) / unit * unit;
  const size_t smem = sizeof(SpShared) + (size_t)per * es + (size_t)(per / unit) * sizeof(double);
  const bool aligned = (uintptr_t)p.logits % 16 == 0 && (p.n == 1 || p.row_stride * es % 16 == 0);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.n * C));
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, p, per);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (p.bf16) return aligned ? go(sample_kernel<__nv_bfloat16, true>) : go(sample_kernel<__nv_bfloat16, false>);
  return aligned ? go(sample_kernel<float, true>) : go(sample_kernel<float, false>);
}

}  // namespace kvc
