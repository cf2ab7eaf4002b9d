// Token sampling: temperature, top-k, top-p, min-p and one given random number a row.
//
// Which tokens stay is decided on the row's order (logit down, index up): each filter keeps a
// head of it, so the outcome is one cut (key, index), and the token is found where the kept
// mass, summed in index order, passes u times its total.  No sort: the cut of top-k is the k-th
// key by counts, that of top-p the key at which the summed mass reaches top_p of the total.
//
// Masses.  A vocabulary of 10^5 flat probabilities puts borders 10^-5 apart, so fp32 sums
// (errors near 10^-7) would move a border once in a hundred rows.  Weights are formed in fp64:
// 2^t with t = (z - max) log2(e) / T split as t = k / 64 + f, |f| <= 1/128; 2^(k mod 64 / 64) from a
// table that the CUDA function exp2 fills, 2^f by the Taylor series of exp(f ln 2) to degree 4
// (relative error below 4e-14), and the exponent added.  Sums run in fp64 in a fixed order.
//
// A row is a cluster of CTAs, each with a slice of it in shared memory, read from HBM once.
//   A  the maximum and its first index
//   B  cut search: counts or masses by bins of 1/16 octave of weight below the maximum (shared-memory
//      integer atomics: order does not matter), combined over the cluster through distributed
//      shared memory; the bin that holds the border is searched again by ranges of the key, until
//      one key is left; of its ties the lowest indices stay.  In the first search of top-p the bins
//      hold masses to 16 bits only: the exact fp64 sums of pass C decide whether the bin is the
//      right one (else its neighbour is taken), the later searches count in 2^-40 units.
//   C  fp64 sums of the kept weights by 32-vector stretches of a warp, in index order
//   D  the stretch, lane and element where u * total falls
#include <cooperative_groups.h>

#include <climits>

#include "kernels.cuh"

namespace kvc {
namespace cg = cooperative_groups;

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_BINS = 2048;
constexpr int SP_MAXC = 8;

struct alignas(16) SpShared {                   // the slice follows: its vectors are 16-byte aligned
  unsigned long long hist[SP_BINS];             // u32 counts / 16-bit masses, or u64 in 2^-40 units
  double comb[SP_BINS];                         // this CTA's share of the bins, combined over the cluster
  double table[64];                             // 2^(j / 64)
  unsigned long long xch[2][4];                 // values exchanged over the cluster, two steps deep
  unsigned long long red[SP_WARPS][4];
  double found[2];
  int ifound[2];
};

template <typename T> struct SpVec;
template <> struct SpVec<__nv_bfloat16> {
  static constexpr int N = 8, KSHIFT = 16;      // keys differ in their upper 16 bits only
};
template <> struct SpVec<float> {
  static constexpr int N = 4, KSHIFT = 0;
};

__device__ __forceinline__ uint32_t sp_key(float z, int shift) { return f2key(z + 0.f) >> shift; }   // -0 counts as +0

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

template <typename T>
struct SpRow {
  static constexpr int N = SpVec<T>::N, KS = SpVec<T>::KSHIFT;
  cg::cluster_group cl;
  SpShared& sh;
  const uint4* slice;                           // this CTA's vectors
  double* wsum;                                 // kept mass of every 32-vector stretch
  int C, rank, nvec, i0;                        // cluster size, rank, vectors of the slice, its first index
  int step;
  float zmax, ybin;                             // bin = (zmax - z) * ybin
  double c;                                     // log2(e) / T
  // tokens left by top-k: key > ck, or key == ck and index <= ci
  uint32_t ck;
  int ci;
  double zcut;                                  // min-p: z >= zcut

  __device__ __forceinline__ SpRow(SpShared& s) : cl(cg::this_cluster()), sh(s) {}

  // value of every CTA's thread 0; slots are reused two steps later, with a barrier between
  template <int K, typename F>
  __device__ __forceinline__ void exchange(const unsigned long long (&v)[K], F&& use) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) sh.xch[step & 1][k] = v[k];
    }
    cl.sync();
    for (int r = 0; r < C; ++r) {
      const unsigned long long* o = cl.map_shared_rank(&sh.xch[step & 1][0], r);
      unsigned long long w[K];
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = o[k];
      use(r, w);
    }
    ++step;
  }
  // sum over the CTA, in a fixed order, known to every thread
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
      V s = V(0);
      for (int w = 0; w < SP_WARPS; ++w) s += *reinterpret_cast<V*>(&sh.red[w][k]);
      v[k] = s;
    }
  }

  __device__ __forceinline__ void unpack(int v, float (&z)[N]) const {
    Vec<T>::unpack(slice[v], z);
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] = fmaxf(z[j], -INFINITY);   // NaN counts as -infinity
  }
  // distance below the maximum in bins, monotone in z; infinite maxima and steps: only the maximum is at 0
  __device__ __forceinline__ float dist(float z) const { return z == zmax ? 0.f : (zmax - z) * ybin; }
  __device__ __forceinline__ int bin(float z) const {
    const float y = dist(z);
    return y < (float)(SP_BINS - 1) ? (int)y : SP_BINS - 1;      // NaN: the last
  }
  __device__ __forceinline__ double weight(float z) const {
    const double d = (double)z - (double)zmax;
    double t = z == zmax ? 0.0 : d * c;
    if (!(t > -1020.0)) return 0.0;             // below any sum's last bit; infinite distances too
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
  __device__ __forceinline__ bool left(uint32_t key, int idx) const { return key > ck || (key == ck && idx <= ci); }

  // The first bin at which the sum of comb reaches `target`, over the cluster's shares; `above`
  // receives the sum before it.  The shares were written before a cluster barrier.
  __device__ __forceinline__ void border(double share, double frac, double target, int& b, double& above) {
    const int per = SP_BINS / C;
    double tot[SP_MAXC], all = 0.0;
    unsigned long long x[1] = {(unsigned long long)__double_as_longlong(share)};
    exchange<1>(x, [&](int r, unsigned long long (&w)[1]) {
      tot[r & (SP_MAXC - 1)] = __longlong_as_double((long long)w[0]);
      all += tot[r & (SP_MAXC - 1)];
    });
    if (frac > 0.0) target = frac * all;
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      double before = 0.0;
      int r = 0, end = 0;                       // shares that hold something: the one that reaches target, else the last
      for (int x = 0; x < C; ++x)
        if (tot[x] > 0.0) end = x;
      while (r < end && (!(tot[r] > 0.0) || before + tot[r] < target)) before += tot[r++];
      // the share's bins, per / 32 a lane
      const double* o = cl.map_shared_rank(&sh.comb[0], r);
      const int q = per / 32;
      double s = 0.0;
      for (int j = 0; j < q; ++j) s += o[lane * q + j];
      double inc = s;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(FULL, inc, d);
        if (lane >= d) inc += y;
      }
      const unsigned hit = __ballot_sync(FULL, before + inc >= target && s > 0.0);
      const unsigned any = __ballot_sync(FULL, s > 0.0);
      const int at = hit ? __ffs(hit) - 1 : any ? 31 - __clz(any) : 31;   // none by rounding: the last that holds something
      if (lane == at) {
        double run = before + inc - s;
        int j = 0, last = 0;
        double last_run = run;
        for (; j < q; ++j) {
          const double w = o[lane * q + j];
          if (w > 0.0) {
            last = j;
            last_run = run;
            if (run + w >= target) break;
          }
          run += w;
        }
        sh.ifound[0] = r * per + lane * q + last;
        sh.found[0] = last_run;
      }
    }
    __syncthreads();
    b = sh.ifound[0];
    above = sh.found[0];
    __syncthreads();
  }
  // Every CTA's histogram summed into shares of the bins; returns this CTA's share's sum.
  // kind 0: counts, 1: 16-bit masses relative to the bin's upper edge, 2: u64.
  __device__ __forceinline__ double combine(int kind) {
    cl.sync();
    const int per = SP_BINS / C;
    double s[1] = {0.0};
    for (int j = threadIdx.x; j < per; j += SP_THREADS) {
      const int b = rank * per + j;
      unsigned long long h = 0;
      for (int r = 0; r < C; ++r) {
        if (kind == 2) h += cl.map_shared_rank(&sh.hist[0], r)[b];
        else h += reinterpret_cast<unsigned*>(cl.map_shared_rank(&sh.hist[0], r))[b];
      }
      double v = (double)h;
      if (kind == 1) v *= (double)exp2f(-(float)b * (1.f / 16.f));
      sh.comb[j] = v;
      s[0] += v;
    }
    block_sum<1>(s);
    return s[0];
  }
  __device__ __forceinline__ void clear_hist(int words) {
    for (int j = threadIdx.x; j < words; j += SP_THREADS) sh.hist[j] = 0ull;
    __syncthreads();
  }

  // Within bin b0 (of the tokens left by top-k when in_left), the key at which the count (MASS:
  // the mass, in units of 2^-(40 + e)) reaches `need`, and the index of the last tie that stays.
  template <bool MASS>
  __device__ __forceinline__ void refine(int b0, double need, int e, bool in_left, uint32_t& tkey, int& tidx) {
    // keys the bin can hold: its edges, a thousandth of a bin wider for the roundings of bin()
    uint32_t hi, lo;
    {
      const float w = ybin > 0.f ? 1.f / ybin : INFINITY;
      const float zh = b0 == 0 ? zmax : zmax - ((float)b0 - 0.001f) * w;
      const float zl = b0 == SP_BINS - 1 ? -INFINITY : zmax - ((float)b0 + 1.001f) * w;
      hi = min(sp_key(zh, KS) + 1u, sp_key(zmax, KS));
      lo = zl > -INFINITY ? sp_key(zl, KS) : 0u;
      lo = lo > 0u ? lo - 1u : 0u;
      lo = max(lo, sp_key(-INFINITY, KS) + 1u);
      if (!(zh > -INFINITY)) hi = sp_key(zmax, KS);
    }
    double above = 0.0;
    int shift = 0;
    while (((hi - lo) >> shift) >= SP_BINS) ++shift;
    while (true) {
      clear_hist(MASS ? SP_BINS : SP_BINS / 2);
      for (int v = threadIdx.x; v < nvec; v += SP_THREADS) {
        float z[N];
        unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t key = sp_key(z[j], KS);
          if (key < lo || key > hi || bin(z[j]) != b0) continue;
          if (in_left && !left(key, i0 + v * N + j)) continue;
          const uint32_t hb = (hi - key) >> shift;
          if (MASS) {
            const unsigned long long q = (unsigned long long)__double2ll_rn(scalbn(weight(z[j]), 40 + e));
            atomicAdd(&sh.hist[hb], q);
          } else {
            atomicAdd(reinterpret_cast<unsigned*>(sh.hist) + hb, 1u);
          }
        }
      }
      __syncthreads();
      const double share = combine(MASS ? 2 : 0);
      int hb;
      double ab;
      border(share, 0.0, need - above, hb, ab);
      above += ab;
      const uint32_t top = hi - ((uint32_t)hb << shift);
      const uint32_t span = (1u << shift) - 1u;
      lo = top - lo > span ? top - span : lo;
      hi = top;
      if (shift == 0) break;
      shift = shift > 11 ? shift - 11 : 0;
      if (((hi - lo) >> shift) >= SP_BINS) ++shift;
    }
    tkey = hi;
    // of the ties of tkey the first `take` in index order stay
    double take = need - above;
    if (MASS) {
      const double w = rint(scalbn(weight(sp_value<KS>(tkey)), 40 + e));
      take = w > 0.0 ? ceil(take / w) : 1.0;
    }
    if (take < 1.0) take = 1.0;
    int mine[1] = {0};
    for (int v = threadIdx.x; v < nvec; v += SP_THREADS) {
      float z[N];
      unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t key = sp_key(z[j], KS);
        mine[0] += key == tkey && (!in_left || left(key, i0 + v * N + j));
      }
    }
    block_sum<1>(mine);
    double before = 0.0, total = 0.0;
    unsigned long long x[1] = {(unsigned long long)mine[0]};
    exchange<1>(x, [&](int r, unsigned long long (&w)[1]) {
      if (r < rank) before += (double)w[0];
      total += (double)w[0];
    });
    tidx = INT_MAX;
    if (take < total) {
      // this slice holds the last tie that stays: walk its stretches in order
      if (before < take && take <= before + (double)mine[0] && threadIdx.x < 32) {
        int want = (int)(take - before);        // the want-th tie of the slice
        for (int s0 = 0; s0 < nvec; s0 += 32) {
          const int v = s0 + threadIdx.x;
          int n = 0;
          float z[N];
          if (v < nvec) {
            unpack(v, z);
#pragma unroll
            for (int j = 0; j < N; ++j) {
              const uint32_t key = sp_key(z[j], KS);
              n += key == tkey && (!in_left || left(key, i0 + v * N + j));
            }
          }
          int inc = n;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(FULL, inc, d);
            if ((int)threadIdx.x >= d) inc += y;
          }
          const int all = __shfl_sync(FULL, inc, 31);
          if (all >= want) {
            const unsigned hit = __ballot_sync(FULL, inc >= want);
            if ((int)threadIdx.x == __ffs(hit) - 1) {
              int k = inc - n;
#pragma unroll
              for (int j = 0; j < N; ++j) {
                const uint32_t key = sp_key(z[j], KS);
                if (key == tkey && (!in_left || left(key, i0 + v * N + j)) && ++k == want) sh.ifound[1] = i0 + v * N + j;
              }
            }
            break;
          }
          want -= all;
        }
      }
      __syncthreads();
      unsigned long long y[1] = {(unsigned long long)(before < take && take <= before + (double)mine[0] ? sh.ifound[1] + 1 : 0)};
      int at = 0;
      exchange<1>(y, [&](int, unsigned long long (&w)[1]) { at = max(at, (int)w[0]); });
      tidx = at - 1;
    }
  }
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(SP_THREADS) sample_kernel(SampleParams p, int per_cta) {
  constexpr int N = SpVec<T>::N, KS = SpVec<T>::KSHIFT;
  static_assert(sizeof(SpShared) % 16 == 0, "vectors follow");
  extern __shared__ __align__(16) uint8_t sp_raw[];
  SpShared& sh = *reinterpret_cast<SpShared*>(sp_raw);
  uint4* slice = reinterpret_cast<uint4*>(sp_raw + sizeof(SpShared));
  SpRow<T> s(sh);
  s.C = (int)s.cl.num_blocks();
  s.rank = (int)s.cl.block_rank();
  const int row = blockIdx.x / s.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  s.slice = slice;
  s.wsum = reinterpret_cast<double*>(slice + per_cta / N);
  s.i0 = s.rank * per_cta;
  s.nvec = max(0, min(per_cta, p.V - s.i0) + N - 1) / N;
  s.step = 0;
  const T* z0 = reinterpret_cast<const T*>(p.logits) + row * p.row_stride;

  // A: the slice into shared memory, the maximum and its first index
  float best = -INFINITY;
  int at = INT_MAX;
#pragma unroll 4
  for (int v = threadIdx.x; v < s.nvec; v += SP_THREADS) {
    const uint4 u = sp_load<T, ALIGNED>(z0, s.i0 + (int64_t)v * N, p.V);
    slice[v] = u;
    float z[N];
    Vec<T>::unpack(u, z);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (z[j] > best) {
        best = z[j];
        at = s.i0 + v * N + j;
      }
  }
  if (threadIdx.x < 64) sh.table[threadIdx.x] = exp2((double)threadIdx.x / 64.0);
  unsigned long long bk = at == INT_MAX ? 0ull : ((unsigned long long)f2key(best + 0.f) << 32) | (unsigned)~at;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bk = max(bk, __shfl_xor_sync(FULL, bk, o));
  if (lane == 0) sh.red[warp][0] = bk;
  __syncthreads();
  for (int w = 0; w < SP_WARPS; ++w) bk = max(bk, sh.red[w][0]);
  {
    unsigned long long x[1] = {bk};
    s.exchange(x, [&](int, unsigned long long (&w)[1]) { bk = max(bk, w[0]); });
  }
  const bool leader = s.rank == 0 && threadIdx.x == 0;
  const float T_ = p.temperature ? p.temperature[row] : 1.f;
  if (bk == 0ull || !(T_ > 0.f)) {
    if (leader) {
      p.token[row] = bk == 0ull ? -1 : (int)~(unsigned)bk;
      if (p.logprob) p.logprob[row] = bk == 0ull ? -INFINITY : 0.f;
      if (p.kept) p.kept[row] = bk != 0ull;
    }
    s.cl.sync();                                // no CTA leaves while another reads its shared memory
    return;
  }
  s.zmax = key2f((uint32_t)(bk >> 32));
  s.c = 1.4426950408889634 / (double)T_;
  s.ybin = (float)(16.0 * s.c);
  s.ck = sp_key(-INFINITY, KS);                 // everything above -infinity
  s.ci = -1;
  const int k = p.top_k ? p.top_k[row] : 0;
  const double top_p = p.top_p ? (double)p.top_p[row] : 1.0;
  double min_p = p.min_p ? (double)p.min_p[row] : 0.0;
  min_p = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;   // NaN: off
  // p_i >= min_p max p  <=>  z_i >= max z + T ln(min_p)
  s.zcut = min_p > 0.0 ? (double)s.zmax + (min_p < 1.0 ? (double)T_ * log(min_p) : 0.0) : -INFINITY;
  if (!(s.zcut <= (double)s.zmax)) s.zcut = (double)s.zmax;   // infinite maximum and temperature
  const bool use_k = k > 0 && k < p.V, use_p = top_p < 1.0;

  if (use_k) {
    // B: the k-th key by counts
    s.clear_hist(SP_BINS / 2);
    int have[1] = {0};
    for (int v = threadIdx.x; v < s.nvec; v += SP_THREADS) {
      float z[N];
      s.unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (z[j] > -INFINITY) {
          ++have[0];
          atomicAdd(reinterpret_cast<unsigned*>(sh.hist) + s.bin(z[j]), 1u);
        }
    }
    s.block_sum(have);
    int total = 0;
    unsigned long long x[1] = {(unsigned long long)have[0]};
    s.exchange(x, [&](int, unsigned long long (&w)[1]) { total += (int)w[0]; });
    if (k < total) {
      const double share = s.combine(0);
      int b;
      double above;
      s.border(share, 0.0, (double)k, b, above);
      uint32_t tk;
      int ti;
      s.template refine<false>(b, (double)k - above, 0, false, tk, ti);
      s.ck = tk;
      s.ci = ti;
    }
  }

  // C (and B for top-p): the kept mass by stretches of 32 vectors
  int b = SP_BINS;                              // top-p: kept are the bins before b and a part of b
  double above = 0.0;
  if (use_p && top_p > 0.0) {
    s.clear_hist(SP_BINS / 2);
    for (int v = threadIdx.x; v < s.nvec; v += SP_THREADS) {
      float z[N];
      s.unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (!s.left(sp_key(z[j], KS), s.i0 + v * N + j)) continue;
        const int bb = s.bin(z[j]);
        if (bb >= SP_BINS - 1) continue;        // below 2^-128 of the maximum
        const float y = s.dist(z[j]) - (float)bb;
        atomicAdd(reinterpret_cast<unsigned*>(sh.hist) + bb, (unsigned)(exp2f(y * (-1.f / 16.f)) * 65536.f));
      }
    }
    __syncthreads();
    const double share = s.combine(1);
    s.border(share, top_p, 0.0, b, above);
  } else if (use_p) {
    b = 0;                                      // top_p <= 0: one token
  }
  const int nst = (s.nvec + 31) / 32;
  double mass = 0.0, in_b = 0.0;
  int kept = 0, kept_all = 0;
  double total = 0.0;
  for (int moved = 0;;) {
    double sums[3] = {0.0, 0.0, 0.0};           // all that is left, bins before b, bin b
    kept = 0;
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      double mine = 0.0;
      if (v < s.nvec) {
        float z[N];
        s.unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (!s.left(sp_key(z[j], KS), s.i0 + v * N + j)) continue;
          const bool over = (double)z[j] >= s.zcut;
          if (!use_p && !over) continue;
          const double w = s.weight(z[j]);
          const int bb = use_p ? s.bin(z[j]) : 0;
          sums[0] += w;
          if (bb < b) {
            sums[1] += w;
            if (over) {
              mine += w;
              ++kept;
            }
          } else if (bb == b) {
            sums[2] += w;
          }
        }
      }
      mine = warp_sum_d(mine);
      if (lane == 0) s.wsum[st] = mine;
    }
    if (!use_p) break;
    s.block_sum(sums);
    unsigned long long x[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) x[q] = (unsigned long long)__double_as_longlong(sums[q]);
    total = above = in_b = 0.0;
    s.exchange(x, [&](int, unsigned long long (&w)[3]) {
      total += __longlong_as_double((long long)w[0]);
      above += __longlong_as_double((long long)w[1]);
      in_b += __longlong_as_double((long long)w[2]);
    });
    // the bin is right if the sum passes top_p of the total inside it
    const double goal = top_p * total;
    if (top_p <= 0.0) break;
    const int way = above >= goal && b > 0 ? -1 : above + in_b < goal && b < SP_BINS - 2 ? 1 : 0;
    if (way == 0 || way == -moved) break;       // right, or between two bins by the sums' last bits
    b += way;
    moved = way;
  }
  if (use_p) {
    const int e = b / 16;                       // the bin's weights lie in (2^(-e-1), 2^-e], about
    uint32_t tk;
    int ti;
    double need = ldexp(top_p * total - above, 40 + e);
    if (!(need > 0.0)) need = 0.0;
    s.template refine<true>(b, need, e, true, tk, ti);
    // the part of bin b that stays
    for (int st = warp; st < nst; st += SP_WARPS) {
      const int v = st * 32 + lane;
      double mine = 0.0;
      bool any = false;
      if (v < s.nvec) {
        float z[N];
        s.unpack(v, z);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t key = sp_key(z[j], KS);
          const int idx = s.i0 + v * N + j;
          if (key < tk || (key == tk && idx > ti) || s.bin(z[j]) != b || !s.left(key, idx) || (double)z[j] < s.zcut) continue;
          mine += s.weight(z[j]);
          ++kept;
          any = true;
        }
      }
      if (__any_sync(FULL, any)) {
        mine = warp_sum_d(mine);
        if (lane == 0) s.wsum[st] += mine;
      }
    }
    // from here on `left` is the final cut
    s.ci = tk == s.ck ? min(ti, s.ci) : ti;
    s.ck = tk;
  }
  int kk[1] = {kept};
  s.block_sum(kk);                              // also orders the stretches' sums before their use
  // D: the slices' masses, the slice, the stretch, the element
  if (warp == 0) {
    const int q = (nst + 31) / 32;
    double sum = 0.0;
    for (int j = lane * q; j < min(nst, (lane + 1) * q); ++j) sum += s.wsum[j];
    double inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sh.found[1] = inc;
  }
  __syncthreads();
  double before = 0.0, upto = 0.0;
  int chosen = -1, last = 0;
  mass = 0.0;
  {
    double cum[SP_MAXC];
    unsigned long long x[2] = {(unsigned long long)__double_as_longlong(sh.found[1]), (unsigned long long)kk[0]};
    s.exchange(x, [&](int r, unsigned long long (&w)[2]) {
      const double m = __longlong_as_double((long long)w[0]);
      if (m > 0.0) last = r;
      mass += m;
      cum[r & (SP_MAXC - 1)] = mass;
      kept_all += (int)w[1];
    });
    float u = p.u[row];
    u = u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f;   // NaN and negatives: 0
    upto = (double)u * mass;
    for (int r = 0; r < s.C; ++r)
      if (chosen < 0 && cum[r & (SP_MAXC - 1)] > upto) chosen = r;
    if (chosen < 0) chosen = last;
    before = chosen > 0 ? cum[(chosen - 1) & (SP_MAXC - 1)] : 0.0;
  }
  if (s.rank == chosen && warp == 0) {
    // the stretch whose running sum passes the goal, or the last one with mass
    const int q = (nst + 31) / 32;
    double sum = 0.0;
    for (int j = lane * q; j < min(nst, (lane + 1) * q); ++j) sum += s.wsum[j];
    double inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned hit = __ballot_sync(FULL, before + inc > upto && sum > 0.0);
    const unsigned any = __ballot_sync(FULL, sum > 0.0);
    const int l = hit ? __ffs(hit) - 1 : 31 - __clz(any);
    double run = before + __shfl_sync(FULL, inc - sum, l);
    int st = -1;
    double st_run = 0.0;
    for (int j = l * q; j < min(nst, (l + 1) * q); ++j) {
      const double w = s.wsum[j];
      if (w > 0.0) {
        st = j;
        st_run = run;
        if (run + w > upto) break;
      }
      run += w;
    }
    const int v = st * 32 + lane;
    float z[N];
    double w[N], mine = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) w[j] = 0.0;
    if (v < s.nvec) {
      s.unpack(v, z);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (s.left(sp_key(z[j], KS), s.i0 + v * N + j) && (double)z[j] >= s.zcut) w[j] = s.weight(z[j]);
        mine += w[j];
      }
    }
    inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned hit2 = __ballot_sync(FULL, st_run + inc > upto && mine > 0.0);
    const unsigned any2 = __ballot_sync(FULL, mine > 0.0);
    const int l2 = hit2 ? __ffs(hit2) - 1 : 31 - __clz(any2);
    if (lane == l2) {
      double r2 = st_run + inc - mine;
      int tok = -1;
      double tw = 1.0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (w[j] > 0.0 && (tok < 0 || r2 <= upto)) {
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
  s.cl.sync();
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  const int es = p.bf16 ? 2 : 4, vn = 16 / es;
  // the cluster: slices of at most 19456 elements for few rows, so that the passes over a slice are
  // short; of at most 32768 once the rows alone fill the GPU
  const int most = p.n * 8 >= 4 * num_sms() ? 32768 : 19456;
  int C = 1;
  while (C < SP_MAXC && (p.V + C - 1) / C > most) C <<= 1;
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
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, p, per);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (p.bf16) return aligned ? go(sample_kernel<__nv_bfloat16, true>) : go(sample_kernel<__nv_bfloat16, false>);
  return aligned ? go(sample_kernel<float, true>) : go(sample_kernel<float, false>);
}

}  // namespace kvc
