// Decode attention of a batch over a shared prompt and each sequence's own rows: how the work is
// cut, the general kernel, and the merge of the partial results.
//
//   o(b,l,h) = sum_i 2^(z_i - M) v_i / sum_i 2^(z_i - M),  z in log2 units, over the prompt's keys
//   (z_i = q k_i * qscale + alpha_c log2 R_i) and the sequence's own (no bias).
// Any cut of the keys into stretches gives partial (m, sum, o) records that combine exactly:
// M = max m, each record scaled by 2^(m - M).  The prompt's stretches are worked on for all rows
// of the batch at once (prefix_tc.cu: bf16, tensor cores; here: fp32 caches or queries, groups of 8
// query rows), the own ones row by row (prefix_own.cu, or here).
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "tc_sm100.cuh"

namespace kvc {

constexpr float PF_LN2 = 0.6931471805599453f;
constexpr int PG_THREADS = 128;
constexpr int PG_ROWS = 8;                      // query rows a CTA

// Four consecutive elements of a row.
__device__ __forceinline__ void ld4(const char* p, int bf16, float (&f)[4]) {
  if (bf16) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    f[0] = bf_lo(u.x); f[1] = bf_hi(u.x); f[2] = bf_lo(u.y); f[3] = bf_hi(u.y);
  } else {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  }
}

// General form: one CTA a (group of up to 8 query rows, stretch of keys).  D / 4 lanes share a key,
// four dimensions each.  Their parts of the 8 logits are summed by halves: at every step a lane keeps half of
// its rows and gives the other half away, so that it ends with one row's logit (9 shuffles at D = 128, where
// 8 sums over all lanes took 40) and has that row's maximum, sum and weight to itself; 8 shuffles bring the
// weights back to all.  Two keys at a time, and the next two are loaded meanwhile.  Bound by issue (7
// sequences x 4 heads x 8, d = 64, 4013 keys, 3 layers, fp32: 90 us a call before, 61 so).  The key groups are merged
// in shared memory.  OWN: the group is the G heads of a (sequence, layer, KV head) row over its own keys;
// else 8 of the B * G rows of (layer, KV head) over the prompt's.
template <int D, bool OWN>
__global__ void __launch_bounds__(PG_THREADS) prefix_generic_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int LPK = D / 4, KPW = 32 / LPK, NG = (PG_THREADS / 32) * KPW;   // lanes a key, keys a warp, key groups
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = lane % LPK, grp = warp * KPW + lane / LPK;
  const int item = blockIdx.x, split = blockIdx.y;
  int g, l, b = 0, n, R0 = 0, nr;
  const char *Kb, *Vb;
  int64_t kst, vst;
  const int32_t* trow = nullptr;
  const float* Rr = nullptr;
  if (OWN) {
    g = item % p.Hkv;
    l = item / p.Hkv % p.L;
    b = item / (p.Hkv * p.L);
    const int n0 = p.len[b * p.L + l];
    n = n0 < 0 ? 0 : min(n0, p.max_len);
    if (n != n0 && split == 0 && threadIdx.x == 0) flag(p.status, ST_BOUNDS);
    nr = p.G;
    if (p.table) trow = p.table + b * p.tsb + l * p.tsl;
    Kb = p.K + g * p.Ksh + (p.table ? 0 : b * p.Ksb + l * p.Ksl);
    Vb = p.V + g * p.Vsh + (p.table ? 0 : b * p.Vsb + l * p.Vsl);
    kst = p.Kst;
    vst = p.Vst;
  } else {
    const int rg = item % p.rgp;
    g = item / p.rgp % p.Hkv;
    l = item / (p.rgp * p.Hkv);
    const int n0 = p.len_p[l];
    n = n0 < 0 ? 0 : min(n0, p.max_p);
    if (n != n0 && split == 0 && threadIdx.x == 0) flag(p.status, ST_BOUNDS);
    R0 = rg * PG_ROWS;
    nr = min(PG_ROWS, p.B * p.G - R0);
    Kb = p.Kp + l * p.Kpl + g * p.Kph;
    Vb = p.Vp + l * p.Vpl + g * p.Vph;
    kst = p.Kpt;
    vst = p.Vpt;
    if (p.R) Rr = p.R + l * p.Rsl + g * p.Rsh;
  }
  const int sl = OWN ? p.slo : p.spl, ns = OWN ? p.nso : p.nsp;
  const int s0 = split * sl, s1 = min(n, s0 + sl);
  const PartialBuf& out = OWN ? p.po : p.pp;
  const int64_t rec0 = ((int64_t)item * ns + split) * (OWN ? p.G : PG_ROWS);
  tc::pdl_launch();
  if (s0 >= s1) {
    if ((int)threadIdx.x < nr) out.ml[rec0 + threadIdx.x] = make_float2(-INFINITY, 0.f);
    if (OWN) tc::pdl_wait();
    return;
  }
  float q[PG_ROWS][4], acc[PG_ROWS][4];
#pragma unroll
  for (int r = 0; r < PG_ROWS; ++r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[r][e] = acc[r][e] = 0.f;
    if (r < nr) {
      const int bb = OWN ? b : (R0 + r) / p.G, gg = OWN ? r : (R0 + r) % p.G;
      const int64_t off = (((int64_t)bb * p.L + l) * p.Hq + g * p.G + gg) * D + part * 4;
      ld4(reinterpret_cast<const char*>(p.q) + off * (p.qbf16 ? 2 : 4), p.qbf16, q[r]);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[r][e] *= p.qscale;
    }
  }
  const int esz = p.kbf16 ? 2 : 4;
  constexpr int UK = 2;                         // keys of a lane group at a time
  struct Key {
    float k[4], v[4], bias;
  };
  auto fetch = [&](int i, Key& x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x.k[e] = x.v[e] = 0.f;
    x.bias = -INFINITY;                         // behind the stretch: no weight
    if (i >= s1) return;
    x.bias = Rr ? p.alpha_c * log2f(__ldg(Rr + i)) : 0.f;
    const char *ka, *va;
    if (OWN && trow) {
      const int pg = __ldg(trow + (i >> p.shift)), off = i & ((1 << p.shift) - 1);
      if ((unsigned)pg >= (unsigned)p.n_pages) {
        flag(p.status, ST_BOUNDS);
        return;
      }
      ka = Kb + (int64_t)pg * p.Ksb + off * kst;
      va = Vb + (int64_t)pg * p.Vsb + off * vst;
    } else {
      ka = Kb + (int64_t)i * kst;
      va = Vb + (int64_t)i * vst;
    }
    ld4(ka + part * 4 * esz, p.kbf16, x.k);
    ld4(va + part * 4 * esz, p.kbf16, x.v);
  };
  float m = -INFINITY, ls = 0.f;                // of row part / (LPK / 8)
  Key cur[UK], nxt[UK];
#pragma unroll
  for (int u = 0; u < UK; ++u) fetch(s0 + u * NG + grp, cur[u]);
  for (int i0 = s0; i0 < s1; i0 += UK * NG) {
#pragma unroll
    for (int u = 0; u < UK; ++u) fetch(i0 + (UK + u) * NG + grp, nxt[u]);
    float x[UK];
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      float z[PG_ROWS];
#pragma unroll
      for (int r = 0; r < PG_ROWS; ++r) {
        z[r] = q[r][0] * cur[u].k[0];
#pragma unroll
        for (int e = 1; e < 4; ++e) z[r] = fmaf(q[r][e], cur[u].k[e], z[r]);
      }
#pragma unroll
      for (int h = PG_ROWS / 2, o = LPK / 2; h > 0; h >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int r = 0; r < h; ++r) {
          const float mine = up ? z[r + h] : z[r], theirs = up ? z[r] : z[r + h];
          z[r] = mine + __shfl_xor_sync(FULL, theirs, o);
        }
      }
#pragma unroll
      for (int o = LPK / 16; o > 0; o >>= 1) z[0] += __shfl_xor_sync(FULL, z[0], o);
      x[u] = z[0] + cur[u].bias;
    }
    const float top = fmaxf(x[0], x[1]);
    const bool grow = top > m + 8.f;
    if (__any_sync(FULL, grow)) {
      const float corr = grow ? exp2f(m - top) : 1.f;   // 0 while nothing was seen
      if (grow) m = top;
      ls *= corr;
#pragma unroll
      for (int r = 0; r < PG_ROWS; ++r) {
        const float cr = __shfl_sync(FULL, corr, r * (LPK / 8), LPK);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] *= cr;
      }
    }
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      const float w = x[u] == -INFINITY ? 0.f : exp2f(x[u] - m);
      ls += w;
#pragma unroll
      for (int r = 0; r < PG_ROWS; ++r) {
        const float wr = __shfl_sync(FULL, w, r * (LPK / 8), LPK);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = fmaf(wr, cur[u].v[e], acc[r][e]);
      }
      cur[u] = nxt[u];
    }
  }
  // merge the CTA's key groups
  __shared__ float sm_o[NG][PG_ROWS][D];
  __shared__ float2 sm_ml[NG][PG_ROWS];
  if (part % (LPK / 8) == 0) sm_ml[grp][part / (LPK / 8)] = make_float2(m, ls);
#pragma unroll
  for (int r = 0; r < PG_ROWS; ++r) {
    *reinterpret_cast<float4*>(&sm_o[grp][r][part * 4]) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
  __syncthreads();
  for (int t = threadIdx.x; t < nr * D; t += PG_THREADS) {
    const int r = t / D, e = t % D;
    float M = -INFINITY, v = 0.f, s = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) M = fmaxf(M, sm_ml[k][r].x);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float sc = M == -INFINITY ? 0.f : exp2f(sm_ml[k][r].x - M);
      v += sm_o[k][r][e] * sc;
      s += sm_ml[k][r].y * sc;
    }
    out.o[(rec0 + r) * D + e] = v;
    if (e == 0) out.ml[rec0 + r] = make_float2(M, s);
  }
  if (OWN) tc::pdl_wait();                      // done is done: the merge waits for this kernel alone
}

// Merge of the records, in a fixed order: CTAs of a (sequence, layer) and some of its heads.  Where the
// prompt's runs lie depends on every layer's length: the CTA sums them once.  Eight lanes share a
// record, D / 8 dimensions each, so it is D / 32 loads a lane, all in flight.  Many heads: eight lanes
// a head (65536 heads of 3 records 30 us; with a warp a head, and its chain of lengths, maxima and
// outputs, 57 us).  Few heads, whose prompt is cut into many runs: a warp a head, its four groups
// of lanes a quarter of the records each (512 heads of 35 records: 9 us against 21).  Records without
// weight (nothing seen) are not read, they may hold anything.
constexpr int PC_THREADS = 256;
constexpr int PC_MANY = 4096;                   // heads from which eight lanes a head are faster (6272: 13 us against 19)
template <int D, int GR>
__global__ void __launch_bounds__(PC_THREADS) prefix_combine_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int Q = D / 32;                     // float4s a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, grp = GR == 1 ? 0 : lane >> 3;
  const int bl = blockIdx.x, l = bl % p.L, b = bl / p.L;
  const int h0 = blockIdx.y * (PC_THREADS / (8 * GR)) + (int)threadIdx.x / (8 * GR);
  __shared__ int sums[3];                       // tiles of the layers before, of all, of this one
  if (p.Kp && p.tc) {
    if (warp == 0) {
      const int per = p.Hkv * p.mp;
      int before = 0, all = 0, T = 0;
      for (int x = lane; x < p.L; x += 32) {
        const int t = (prefix_len(p, x) + 127) / 128;
        all += t * per;
        if (x < l) before += t * per;
        if (x == l) T = t;
      }
      before = __reduce_add_sync(FULL, before);
      all = __reduce_add_sync(FULL, all);
      T = __reduce_add_sync(FULL, T);
      if (lane == 0) {
        sums[0] = before;
        sums[1] = all;
        sums[2] = T;
      }
    }
    __syncthreads();
  }
  const bool live = h0 < p.Hq;
  const int h = live ? h0 : p.Hq - 1;           // lanes past the last head repeat it and write nothing
  const int g = h / p.G, gg = h - g * p.G;
  int np = 0, pstep = 0;                        // prompt records, `pstep` apart from prec
  int64_t prec = 0;
  if (p.Kp && p.tc) {
    np = prefix_records(p, sums[0], sums[1], sums[2], l, g, b * p.G + gg, prec, pstep);
  } else if (p.Kp) {
    const int r = b * p.G + gg;
    np = p.nsp;
    pstep = PG_ROWS;
    prec = (((int64_t)l * p.Hkv + g) * p.rgp + r / PG_ROWS) * p.nsp * PG_ROWS + r % PG_ROWS;
  }
  tc::pdl_wait();                               // the records are complete
  const int nall = np + (p.K ? p.nso : 0);
  const int64_t orec = ((int64_t)bl * p.Hkv + g) * p.nso * p.G + gg;
  const int most = __reduce_max_sync(FULL, nall);
  float M = -INFINITY, lsum = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = grp * 8; i0 - grp * 8 < most; i0 += 8 * GR) {
    const int i = i0 + sub;
    float2 x = make_float2(-INFINITY, 0.f);
    if (i < nall) x = i < np ? p.pp.ml[prec + (int64_t)i * pstep] : p.po.ml[orec + (int64_t)(i - np) * p.G];
    float Mn = fmaxf(M, x.x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(FULL, Mn, o));
    const float ref = Mn == -INFINITY ? 0.f : Mn;
    const float old = tc::ex2(M - ref);         // 0 while nothing was seen
    M = Mn;
    const float w = tc::ex2(x.x - ref);         // 0 for a record without weight
    float s = w * x.y;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
    lsum = fmaf(lsum, old, s);
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] = make_float4(acc[q].x * old, acc[q].y * old, acc[q].z * old, acc[q].w * old);
    const int nn = min(8, most - (i0 - grp * 8));   // the same in all groups: the shuffles want every lane
    for (int j0 = 0; j0 < nn; j0 += 2) {        // two records at a time
      float4 v[2][Q];
      float wj[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        wj[j] = __shfl_sync(FULL, w, (lane & 24) + ((j0 + j) & 7));
        const int k = i0 + j0 + j;
        const float4* r = reinterpret_cast<const float4*>(k < np ? p.pp.o + (prec + (int64_t)k * pstep) * D
                                                                 : p.po.o + (orec + (int64_t)(k - np) * p.G) * D);
#pragma unroll
        for (int q = 0; q < Q; ++q) v[j][q] = wj[j] > 0.f ? r[q * 8 + sub] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          acc[q].x = fmaf(v[j][q].x, wj[j], acc[q].x);
          acc[q].y = fmaf(v[j][q].y, wj[j], acc[q].y);
          acc[q].z = fmaf(v[j][q].z, wj[j], acc[q].z);
          acc[q].w = fmaf(v[j][q].w, wj[j], acc[q].w);
        }
    }
  }
  if (GR > 1) {                                 // the groups' parts
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const float Mo = __shfl_xor_sync(FULL, M, o), Mn = fmaxf(M, Mo), ref = Mn == -INFINITY ? 0.f : Mn;
      const float a0 = tc::ex2(M - ref), a1 = tc::ex2(Mo - ref);
      lsum = lsum * a0 + __shfl_xor_sync(FULL, lsum, o) * a1;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        acc[q].x = acc[q].x * a0 + __shfl_xor_sync(FULL, acc[q].x, o) * a1;
        acc[q].y = acc[q].y * a0 + __shfl_xor_sync(FULL, acc[q].y, o) * a1;
        acc[q].z = acc[q].z * a0 + __shfl_xor_sync(FULL, acc[q].z, o) * a1;
        acc[q].w = acc[q].w * a0 + __shfl_xor_sync(FULL, acc[q].w, o) * a1;
      }
      M = Mn;
    }
    if (grp > 0) return;
  }
  if (!live) return;
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;   // (a NaN among the logits makes lsum NaN, and with it the row)
  const int64_t out = (int64_t)bl * p.Hq + h;
  float4* o = reinterpret_cast<float4*>(p.o + out * D);
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q * 8 + sub] = make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv);
  if (p.lse && sub == 0) p.lse[out * p.lse_stride] = lsum == 0.f ? -INFINITY : (M + log2f(lsum)) * PF_LN2;
}

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t plan_prefix(PrefixParams& p, void* ws) {
  const int sms = num_sms();
  size_t off = 0;
  auto place = [&](PartialBuf& b, int64_t recs) {
    b.ml = ws ? reinterpret_cast<float2*>((char*)ws + off) : nullptr;
    off += up256((size_t)recs * sizeof(float2));
    b.o = ws ? reinterpret_cast<float*>((char*)ws + off) : nullptr;
    off += up256((size_t)recs * p.d * sizeof(float));
  };
  if (p.Kp) {
    const int rows = p.B * p.G;
    p.mt = rows <= 128 ? 1 : 2;
    p.mp = (rows + p.mt * 128 - 1) / (p.mt * 128);
    p.grid = sms;
    p.tc = prefix_tc_supported(p);
    p.rgp = (rows + PG_ROWS - 1) / PG_ROWS;
    if (p.tc) {
      // one group pair a run and item it touches: items + runs bound them
      place(p.pp, ((int64_t)p.L * p.Hkv * p.mp + p.grid) * 2 * 128);
    } else {
      // enough CTAs for four waves, stretches of at least 64 keys
      const int64_t items = (int64_t)p.L * p.Hkv * p.rgp;
      int64_t ns = (sms * 4 * 4 + items - 1) / items;
      const int most = (p.max_p + 63) / 64;
      if (ns > most) ns = most;
      if (ns < 1) ns = 1;
      p.spl = (int)((p.max_p + ns - 1) / ns);
      p.nsp = (p.max_p + p.spl - 1) / p.spl;
      place(p.pp, items * p.nsp * PG_ROWS);
    }
  }
  if (p.K) {
    // items of at least 128 keys, about 12 a persistent CTA (two an SM): drawn one by one, the last ones leave
    // little imbalance.  The cut goes by the bound: one far above the rows' lengths makes their items few and long
    const int64_t rows = (int64_t)p.B * p.L * p.Hkv;
    int64_t ns = ((int64_t)sms * 2 * 12 + rows - 1) / rows;
    const int most = (p.max_len + 127) / 128;
    if (ns > most) ns = most;
    if (ns < 1) ns = 1;
    // (whole 64-key stages: a stage starts on a page's first token or a multiple of 64 inside it)
    p.slo = (int)(((p.max_len + ns - 1) / ns + 63) / 64 * 64);
    p.nso = (p.max_len + p.slo - 1) / p.slo;
    p.own_mma = prefix_own_mma_supported(p);
    place(p.po, rows * p.nso * p.G);
    if (p.own_mma) {
      p.counter = ws ? reinterpret_cast<int*>((char*)ws + off) : nullptr;
      off += 256;
      p.counter_zeroed = p.Kp && p.tc;
    }
  }
  return off;
}

cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t st) {
  cudaError_t e;
  if (p.Kp) {
    if (p.tc) {
      if ((e = launch_prefix_tc(p, st)) != cudaSuccess) return e;
    } else {
      const dim3 grid(p.L * p.Hkv * p.rgp, p.nsp);
      if (p.d == 128) prefix_generic_kernel<128, false><<<grid, PG_THREADS, 0, st>>>(p);
      else prefix_generic_kernel<64, false><<<grid, PG_THREADS, 0, st>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      count_launch();
    }
  }
  if (p.K) {
    if (p.own_mma) {
      if ((e = launch_prefix_own_mma(p, st)) != cudaSuccess) return e;
    } else {
      const dim3 grid(p.B * p.L * p.Hkv, p.nso);
      auto kern = p.d == 128 ? prefix_generic_kernel<128, true> : prefix_generic_kernel<64, true>;
      if ((e = launch_dependent(kern, grid, PG_THREADS, 0, st, p.Kp != nullptr, p)) != cudaSuccess) return e;
      count_launch();
    }
  }
  const bool many = (int64_t)p.B * p.L * p.Hq >= PC_MANY;
  const int per = PC_THREADS / (many ? 8 : 32);   // heads a CTA
  const dim3 grid(p.B * p.L, (p.Hq + per - 1) / per);
  auto kern = p.d == 128 ? (many ? prefix_combine_kernel<128, 1> : prefix_combine_kernel<128, 4>)
                         : (many ? prefix_combine_kernel<64, 1> : prefix_combine_kernel<64, 4>);
  e = launch_dependent(kern, grid, PC_THREADS, 0, st, true, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace kvc
