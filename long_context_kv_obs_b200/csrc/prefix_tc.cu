// Decode attention of a batch over a shared prompt on the 5th-generation tensor cores.
//
// For every layer l and KV head g the B * G query rows of the batch face the same len_prefix[l]
// keys:  S = Q K^T,  P = 2^(S * qscale + alpha_c log2 R - m),  O = P V, with a running maximum m
// and sum a row.  Every key and value is read once for the whole batch: 512 bytes (bf16,
// d = 128) serve B * G rows, so the arithmetic per byte grows with the batch.  Up to 128 rows (one M =
// 128 tile) the floor is HBM, and what bounds the pass is each warpgroup's chain S, maximum, weights,
// P V (56 rows: 94 us for 62 of HBM); above that the products, under the power limit.
//
// P is carried as a bf16 pair hi + lo (two products with V), about 16 bits of it, so that the
// fp32 output keeps fp32-level accuracy: with hi alone its error would be up to 2^-8 a weight.
// The accumulator in TMEM truncates: left to run over a whole prompt (13107 keys, 1640 products) O
// came out 3.4e-5 too small.  So a tile's P V starts afresh and the softmax warps add it to O in
// registers, rounding to nearest.
//
// Work: tiles of 128 keys.  All items (l, g, row block) laid end to end are cut into equal runs of
// tiles, one run a CTA, one CTA an SM (lengths differ by layer; a run may cover the end of
// one item and the start of the next).  A partial record (m, sum, O) leaves for every item a
// run touches; the item's runs are consecutive, so the combine kernel finds them by arithmetic.
// MT = 1 (B * G <= 128): the two softmax warpgroups take the even and the odd tiles of a run, each
// with its own running state.  A warp can read the TMEM lanes of its own quarter only, and the
// quarters are the SM's schedulers: for up to 64 rows the M = 128 tile holds them twice, the first
// warpgroup works on the lower copy and the second on the upper, so that all schedulers have a part
// (56 rows with R: 96 us with half of them idle, 92 so).  MT = 2: both take every tile, with 128 query
// rows each, so K and V are fetched once for 256 rows.
//
// Roles: warps 0-3 and 4-7 are the softmax warpgroups (a thread owns a query row, its TMEM lane),
// warp 8 loads K and V (TMA, 128B swizzle, separate rings), warps 9 and 10 issue the products.  TMEM: a
// warpgroup has 128 columns of S, overwritten by its P, and 128 of O.  Every wait is an mbarrier
// with a time limit, those among the softmax warps too, so an abort strands no warp.  While one warpgroup
// works on its S the tensor cores run the other's products.
// Measured: 64 sequences (256 rows, 32 layers x 8 heads, 13107 keys) 513 us, 0.58 TFLOP with both parts of
// P: 1.13 PFLOP/s, held by the power limit; 56 rows, 28 x 4 heads, 8200 keys with R 94 us, 4.3 TB/s.
#include "kernels.cuh"
#include "tc_sm100.cuh"

namespace kvc {
using namespace tc;

constexpr int PX_KEYS = 128;                    // keys a tile
constexpr int PX_THREADS = 384;                 // warp 11 only completes the third warpgroup
constexpr int PX_ATOM = PX_KEYS * 128;          // 128 rows x 64 bf16, 128B-swizzled (16 KB)
template <int D> constexpr int px_tile() { return (D / 64) * PX_ATOM; }
// Slots of the K and V rings.  MT = 1: even, and tile t goes to warpgroup t & 1, so that a slot is always the
// same warpgroup's: who waits by parity must see every phase of a barrier (with three slots a warpgroup saw
// every other one, and took a phase long past for the one it wanted when loads were late).
template <int D, int MT> constexpr int px_nk() { return D == 64 ? 4 : 2; }
template <int D, int MT> constexpr int px_nv() { return D == 64 || MT == 1 ? 4 : 3; }
struct PxCtl {
  uint64_t fullK[4], emptyK[4], fullV[4], emptyV[4];
  uint64_t s_ready[2], p_ready[2][2], o_ready[2], b_ready[2], q_ready, q_free, s_done, drain;
  uint32_t tmem;
  int abort;
  alignas(16) float bias[2][2][PX_KEYS];        // [warpgroup][buffer], read as float4
  int cum[PREFIX_TC_LAYERS + 1];                         // tiles of the layers before
};
template <int D, int MT> constexpr size_t px_smem() {
  return (size_t)MT * px_tile<D>() + (size_t)(px_nk<D, MT>() + px_nv<D, MT>()) * px_tile<D>() + sizeof(PxCtl);
}

// A run's next piece: tiles [t0, t0 + n) of item (l, g, mp).
struct PxSeg {
  int l, g, mp, t0, n, item;
};
struct PxRun {
  int cur, end, l;
  __device__ __forceinline__ bool next(const PrefixParams& p, const int* cum, PxSeg& s) {
    if (cur >= end) return false;
    while (cur >= cum[l + 1]) ++l;
    const int per = p.Hkv * p.mp, T = (cum[l + 1] - cum[l]) / per;
    const int x = cur - cum[l], it = x / T;
    s.l = l;
    s.g = it / p.mp;
    s.mp = it % p.mp;
    s.t0 = x % T;
    s.n = min(T - s.t0, end - cur);
    s.item = l * per + it;
    cur += s.n;
    return true;
  }
};

// Maximum of 32 products, biased and in log2 units when HAS_R.
template <bool HAS_R>
__device__ __forceinline__ float px_max(const uint32_t (&r)[32], const float* bias, float qscale, float mx) {
  float m0 = mx, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 bb = HAS_R ? *reinterpret_cast<const float4*>(bias + k + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[e] = __uint_as_float(r[k + e]);
      x[e + 1] = __uint_as_float(r[k + e + 1]);
      x[e + 2] = __uint_as_float(r[k + e + 2]);
      x[e + 3] = __uint_as_float(r[k + e + 3]);
      if (HAS_R) {
        x[e] = fmaf(x[e], qscale, bb.x);
        x[e + 1] = fmaf(x[e + 1], qscale, bb.y);
        x[e + 2] = fmaf(x[e + 2], qscale, bb.z);
        x[e + 3] = fmaf(x[e + 3], qscale, bb.w);
      }
    }
    m0 = fmaxf(m0, fmaxf(x[0], x[1]));
    m1 = fmaxf(m1, fmaxf(x[2], x[3]));
    m2 = fmaxf(m2, fmaxf(x[4], x[5]));
    m3 = fmaxf(m3, fmaxf(x[6], x[7]));
  }
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

// acc += the row's D columns of O in TMEM.
template <int D>
__device__ __forceinline__ void px_add_o(uint32_t tO, float (&acc)[D]) {
  uint32_t a[32], b[32];
  tmem_ld32_raw(tO, a);
#pragma unroll
  for (int q = 0; q < D / 32; q += 2) {
    tmem_wait_ld32(a);
    tmem_ld32_raw(tO + q * 32 + 32, b);
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[q * 32 + k] += __uint_as_float(a[k]);
    tmem_wait_ld32(b);
    if (q + 2 < D / 32) tmem_ld32_raw(tO + q * 32 + 64, a);
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[q * 32 + 32 + k] += __uint_as_float(b[k]);
  }
}

template <int D, int MT, bool HAS_R>
__global__ void __launch_bounds__(PX_THREADS, 1)
prefix_tc_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const __grid_constant__ PrefixParams p) {
  constexpr int TILE = px_tile<D>(), NK = px_nk<D, MT>(), NV = px_nv<D, MT>(), NA = D / 64;
  static_assert(MT == 2 || (NK % 2 == 0 && NV % 2 == 0), "a slot belongs to one warpgroup");
  extern __shared__ __align__(1024) uint8_t px_raw[];
  uint8_t* Qs = px_raw;
  uint8_t* Ks = Qs + MT * TILE;
  uint8_t* Vs = Ks + NK * TILE;
  PxCtl* c = reinterpret_cast<PxCtl*>(Vs + NV * TILE);
  volatile int* abort = &c->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c->fullK[i], 1);
      mbar_init(&c->emptyK[i], MT);
      mbar_init(&c->fullV[i], 1);
      mbar_init(&c->emptyV[i], MT);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&c->s_ready[w], 1);
      mbar_init(&c->p_ready[w][0], 4);
      mbar_init(&c->p_ready[w][1], 4);
      mbar_init(&c->o_ready[w], 1);
      mbar_init(&c->b_ready[w], 4);
    }
    mbar_init(&c->q_ready, 8);
    mbar_init(&c->q_free, 10);                  // the softmax warps, and the product warps, which have seen q_ready
    mbar_init(&c->s_done, 8);
    mbar_init(&c->drain, 2);
    c->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&c->tmem, 512);
  if (warp == 8) {
    if (lane == 0) {
      prefetch_map(&mapK);
      prefetch_map(&mapV);
    }
    prefix_tile_sums(p, c->cum);
    if (blockIdx.x == 0) {
      for (int l = lane; l < p.L; l += 32)
        if (prefix_len(p, l) != p.len_p[l]) flag(p.status, ST_BOUNDS);
      if (lane == 0 && p.counter) *p.counter = 0;   // for the own rows' kernel, next on the stream
    }
  }
  pdl_launch();                                 // it fills the SMs as they fall free
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = c->tmem;
  const int total = c->cum[p.L];
  const int W = max(1, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  PxRun run;
  run.cur = (int)min((long long)blockIdx.x * W, (long long)total);
  run.end = min(total, run.cur + W);
  run.l = 0;
  PxSeg sg;

  // registers: 3 x 168 a thread at launch = 2 x 232 + 40
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 8) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      uint32_t tc = 0, issued_k = 0, issued_v = 0;
      while (run.next(p, c->cum, sg)) {
        for (int i = 0; i < sg.n; ++i, ++tc) {
          const int key0 = (sg.t0 + i) * PX_KEYS;
          const int ks = tc % NK, vs = tc % NV;
          if (!mbar_wait(&c->emptyK[ks], ((tc / NK) & 1) ^ 1, abort, p.status)) goto load_done;
          mbar_expect_tx(&c->fullK[ks], TILE);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            tma_load_4d(Ks + ks * TILE + a * PX_ATOM, &mapK, a * 64, key0, sg.g, sg.l, &c->fullK[ks]);
          ++issued_k;
          if (!mbar_wait(&c->emptyV[vs], ((tc / NV) & 1) ^ 1, abort, p.status)) goto load_done;
          mbar_expect_tx(&c->fullV[vs], TILE);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            tma_load_4d(Vs + vs * TILE + a * PX_ATOM, &mapV, a * 64, key0, sg.g, sg.l, &c->fullV[vs]);
          ++issued_v;
        }
      }
    load_done:
      if (*abort) {                             // copies in flight end before shared memory is given up
        int none = 0;
        for (uint32_t j = issued_k > NK ? issued_k - NK : 0; j < issued_k; ++j)
          mbar_wait(&c->fullK[j % NK], (j / NK) & 1, &none, p.status);
        for (uint32_t j = issued_v > NV ? issued_v - NV : 0; j < issued_v; ++j)
          mbar_wait(&c->fullV[j % NV], (j / NV) & 1, &none, p.status);
      }
    }
  } else if (warp < 11) {
    // ------------------------------------------------------------ products
    // A warp for each softmax warpgroup: one for both waits for one's P while the other's lies ready
    // (7 heads a group: 104 us with one, 96 with two).  The whole warp runs the loop and one lane issues: addresses that are known
    // to be the same in all lanes live in uniform registers, where the products' descriptors are wanted
    // (issued by a lone thread each product took 80 to 150 cycles to issue for 53 of work).
      constexpr uint32_t idS = idesc_bf16(128, PX_KEYS);
      constexpr uint32_t idO = idesc_bf16(128, D) | IDESC_B_MN;
      const int w = __shfl_sync(FULL, warp - 9, 0);
      constexpr int di = MT == 1 ? 2 : 1;
      const uint32_t ts = __shfl_sync(FULL, tmem, 0) + w * 128, to = ts + 256;
      const uint32_t q0 = __shfl_sync(FULL, smem_u32(Qs), 0), k0 = q0 + MT * TILE, v0 = k0 + NK * TILE;
      const uint64_t dq = sw128_desc_at(q0 + (MT == 2 ? w : 0) * TILE, 16);
      uint32_t tc = 0, nseg = 0, pv = 0;        // tiles, pieces, and P V products so far
      bool ok = true;
      while (ok && run.next(p, c->cum, sg)) {
        ok = __all_sync(FULL, mbar_wait(&c->q_ready, nseg & 1, abort, p.status));
        ++nseg;
        if (lane == 0) mbar_arrive(&c->q_free);
        __syncwarp();
        const int n = __shfl_sync(FULL, sg.n, 0), i0 = MT == 1 ? (int)((w ^ tc) & 1) : 0;
        auto issue_s = [&](int i) {
          const uint32_t t = tc + i, ks = t % NK;
          if (!__all_sync(FULL, mbar_wait(&c->fullK[ks], (t / NK) & 1, abort, p.status))) return false;
          fence_after();
          const uint64_t dk = sw128_desc_at(k0 + ks * TILE, 16);
          if (elect_one()) {
            if constexpr (D == 128) mma_bf16_k128(ts, dq, dk, PX_ATOM >> 4, PX_ATOM >> 4, idS);
            else mma_bf16_k64(ts, dq, dk, idS, 0);
            mma_commit(&c->s_ready[w]);
            mma_commit(&c->emptyK[ks]);
          }
          __syncwarp();
          return true;
        };
        if (ok && i0 < n) ok = issue_s(i0);
        for (int i = i0; i < n && ok; i += di, ++pv) {
          const uint32_t t = tc + i, vs = t % NV;
          ok = __all_sync(FULL, mbar_wait(&c->fullV[vs], (t / NV) & 1, abort, p.status));
          const uint64_t dv = sw128_desc_at(v0 + vs * TILE, PX_ATOM);
#pragma unroll
          for (int h = 0; h < 2; ++h) {         // the keys' halves: the first, while P of the second is formed
            ok = ok && __all_sync(FULL, mbar_wait(&c->p_ready[w][h], pv & 1, abort, p.status));
            if (!ok) break;
            fence_after();
            if (elect_one()) {
              // P lo first: the tensor core truncates its fp32 accumulator at every product, and the lo
              // parts of the first half leave it small: 12 roundings a tile count, not 16 (see the head of the file)
              mma_bf16_ts_k64(to, ts + h * 64 + 8, dv + h * 512, idO, h);
              mma_bf16_ts_k64(to, ts + h * 64, dv + h * 512, idO, 1);
              if (h == 1) {
                mma_commit(&c->o_ready[w]);
                mma_commit(&c->emptyV[vs]);
              }
            }
            __syncwarp();
          }
          // the next S overwrites the P that these products read
          if (ok && i + di < n) ok = __all_sync(FULL, mbar_wait(&c->o_ready[w], pv & 1, abort, p.status)) && issue_s(i + di);
        }
        tc += n;
      }
      // every arrive issued above has landed before shared memory is given up
      int none = 0;
      if (elect_one()) mma_commit(&c->drain);
      __syncwarp();
      mbar_wait(&c->drain, 0, &none, p.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2;
    const uint32_t tS = tmem + w * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = tS + 256;
    const int rows = p.B * p.G;
    const bool twice = MT == 1 && rows <= 64;    // see the head of the file
    const int row0 = (warp & 3) * 32 - (twice ? w * 64 : 0);   // the warp's first row of a record
    const int wt = threadIdx.x & 127;
    uint32_t steps = 0, tc = 0, nseg = 0;
    bool ok = true;
    while (ok && run.next(p, c->cum, sg)) {
      const int len = prefix_len(p, sg.l);
      const int r0 = sg.mp * (MT * 128);
      // Q of the piece: all S products of the piece before are done (both warpgroups waited for theirs)
      if (nseg > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->q_free);
        ok = mbar_wait(&c->q_free, (nseg - 1) & 1, abort, p.status);
        if (!__all_sync(FULL, ok)) break;
      }
      ++nseg;
      {
        // a warp fills 32 (MT 1: 16) of its rows, whole rows by consecutive lanes
        constexpr int CH = D / 8, WR = 16 * MT;  // 16-byte chunks a row, rows a warp
#pragma unroll
        for (int x = lane; x < WR * CH; x += 32) {
          const int qr = warp * WR + x / CH, ch = x % CH, R = r0 + (twice ? qr & 63 : qr);
          const int b = R / p.G, gg = R - b * p.G;
          const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                   (((int64_t)b * p.L + sg.l) * p.Hq + sg.g * p.G + gg) * D;
          const uint4 v = R < rows ? ldg16(q + ch * 8) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(Qs + (qr >> 7) * TILE + (ch >> 3) * PX_ATOM + (qr & 127) * 128 +
                                    (((ch & 7) ^ (qr & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->q_ready);
      }
      const int Rw = r0 + (MT == 2 ? w * 128 : 0) + row0;   // the warp's first query row
      const bool live = Rw < rows && (!twice || ((warp & 3) >> 1) == w);
      float m = -INFINITY, lsum = 0.f;
      const float* Rr = HAS_R ? p.R + sg.l * p.Rsl + sg.g * p.Rsh : nullptr;
      const int i0 = MT == 1 ? (int)((w ^ tc) & 1) : 0, di = MT == 1 ? 2 : 1;
      float rnext = 1.f;
      if (HAS_R && i0 < sg.n) {
        const int k = (sg.t0 + i0) * PX_KEYS + wt;
        rnext = k < len ? __ldg(Rr + k) : 1.f;
      }
      int mine = 0;
      float acc[D];                             // O of the row
#pragma unroll
      for (int k = 0; k < D; ++k) acc[k] = 0.f;
      for (int i = i0; i < sg.n; i += di, ++mine) {
        const int key0 = (sg.t0 + i) * PX_KEYS, nk = min(PX_KEYS, len - key0);
        const float* bias = c->bias[w][mine & 1];
        if (HAS_R) {
          c->bias[w][mine & 1][wt] = p.alpha_c * log2f(rnext);
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->b_ready[w]);
          ok = mbar_wait(&c->b_ready[w], steps & 1, abort, p.status);
          if (!__all_sync(FULL, ok)) {
            ok = false;
            break;
          }
          const int k = key0 + di * PX_KEYS + wt;
          rnext = i + di < sg.n && k < len ? __ldg(Rr + k) : 1.f;
        }
        if (mine > 0) {
          // the tile before's P V, while the tensor cores work on this tile's S
          ok = mbar_wait(&c->o_ready[w], (steps - 1) & 1, abort, p.status);
          if (!__all_sync(FULL, ok)) {
            ok = false;
            break;
          }
          fence_after();
          if (live) px_add_o<D>(tO, acc);
        }
        ok = mbar_wait(&c->s_ready[w], steps & 1, abort, p.status);
        if (!__all_sync(FULL, ok)) {
          ok = false;
          break;
        }
        fence_after();
        if (nk < PX_KEYS) {
          // rows past the length may hold anything and 0 * NaN is NaN: zero them in V, each warpgroup
          // before its own products
          const uint32_t t = tc + i, vs = t % NV;
          ok = mbar_wait(&c->fullV[vs], (t / NV) & 1, abort, p.status);
          if (!__all_sync(FULL, ok)) {
            ok = false;
            break;
          }
          for (int x = nk * (D / 8) + wt; x < PX_KEYS * (D / 8); x += 128) {
            const int r = x / (D / 8), ch = x % (D / 8);
            *reinterpret_cast<uint4*>(Vs + vs * TILE + (ch >> 3) * PX_ATOM + r * 128 + ((ch & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (live) {
          if (nk < PX_KEYS) {
            // products of keys past the length: -infinity, before anything reads them
#pragma unroll 1
            for (int q4 = nk >> 5; q4 < 4; ++q4) {
              uint32_t x[32];
              tmem_ld32_raw(tS + q4 * 32, x);
              tmem_wait_ld32(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = q4 * 32 + k < nk ? x[k] : 0xff800000u;
              tmem_st32(tS + q4 * 32, x);
            }
            tmem_wait_st();
          }
          // TMEM loads run one chunk ahead of the arithmetic (a wait covers all loads before it)
          float mt = -INFINITY;
          uint32_t xa[16], xb[16], ua[16], ub[16];
          {
            uint32_t ra[32], rb[32];
            tmem_ld32_raw(tS, ra);
            tmem_wait_ld32(ra);
            tmem_ld32_raw(tS + 32, rb);
            mt = px_max<HAS_R>(ra, bias, p.qscale, mt);
            tmem_wait_ld32(rb);
            tmem_ld32_raw(tS + 64, ra);
            mt = px_max<HAS_R>(rb, bias + 32, p.qscale, mt);
            tmem_wait_ld32(ra);
            tmem_ld32_raw(tS + 96, rb);
            mt = px_max<HAS_R>(ra, bias + 64, p.qscale, mt);
            tmem_wait_ld32(rb);
            tmem_ld16_raw(tS, xa);
            mt = px_max<HAS_R>(rb, bias + 96, p.qscale, mt);
          }
          if (!HAS_R) mt *= p.qscale;           // qscale > 0: the maximum of the products
          // the running maximum moves only when it grows by more than 2^8: sums and O stay within
          // fp32 range and most tiles rescale nothing
          const bool grow = mt > m + 8.f;
          const bool rescale = __any_sync(FULL, grow);
          const float corr = grow ? ex2(m - mt) : 1.f;   // 0 while nothing was seen
          if (grow) m = mt;
          if (rescale) {
            lsum *= corr;
#pragma unroll
            for (int k = 0; k < D; ++k) acc[k] *= corr;
          }
          const float mref = m == -INFINITY ? 0.f : m;
          const uint64_t qs2 = pk2(p.qscale, p.qscale), nm2 = pk2(-mref, -mref), neg1 = pk2(-1.f, -1.f);
          uint64_t sum2 = 0;
          // chunk q: P of 16 keys from x to u, while the loads of chunk q + 1 go to xn and the store of
          // chunk q - 1 (un) is under way
          auto chunk = [&](int q, uint32_t (&x)[16], uint32_t (&xn)[16], uint32_t (&u)[16], uint32_t (&un)[16]) {
            tmem_wait_ld16(x);
            if (q + 1 < PX_KEYS / 16) tmem_ld16_raw(tS + q * 16 + 16, xn);
            if (q > 0 && q != PX_KEYS / 32) tmem_st16(tS + q * 16 - 16, un);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              uint64_t off = nm2;
              if (HAS_R) {
                const float2 bb = *reinterpret_cast<const float2*>(bias + q * 16 + k);
                off = add2(pk2(bb.x, bb.y), nm2);
              }
              const float2 y = upk2(fma2(pk2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), qs2, off));
              const float a = ex2(y.x), b = ex2(y.y);
              const uint64_t ab = pk2(a, b);
              sum2 = add2(sum2, ab);
              const uint32_t hi = pack_bf16x2(a, b);
              const float2 lo = upk2(fma2(pk2(bf_lo(hi), bf_hi(hi)), neg1, ab));
              u[k >> 1] = hi;
              u[8 + (k >> 1)] = pack_bf16x2(lo.x, lo.y);
            }
          };
#pragma unroll
          for (int q = 0; q < PX_KEYS / 16; q += 2) {
            chunk(q, xa, xb, ua, ub);
            chunk(q + 1, xb, xa, ub, ua);
            if (q + 2 == PX_KEYS / 32) {        // the first half is there
              tmem_st16(tS + PX_KEYS / 2 - 16, ub);
              tmem_wait_st();
              fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&c->p_ready[w][0]);
            }
          }
          tmem_st16(tS + PX_KEYS - 16, ub);
          const float2 s2 = upk2(sum2);
          lsum += s2.x + s2.y;
          tmem_wait_st();
        } else {
          __syncwarp();                         // all lanes' zeros in V
          if (lane == 0) mbar_arrive(&c->p_ready[w][0]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->p_ready[w][1]);
        ++steps;
      }
      if (!ok) break;
      tc += sg.n;
      // the piece's record of this warpgroup
      const int64_t group = 2 * (int64_t)(sg.item + blockIdx.x) + w;
      const int64_t rec = group * 128 + row0 + lane;
      // its rows go to memory through the Q area: all S products of the piece are done first
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->s_done);
      ok = mbar_wait(&c->s_done, (nseg - 1) & 1, abort, p.status);
      if (!__all_sync(FULL, ok)) {
        ok = false;
        break;
      }
      if (mine > 0) {
        ok = mbar_wait(&c->o_ready[w], (steps - 1) & 1, abort, p.status);
        if (!__all_sync(FULL, ok)) {
          ok = false;
          break;
        }
        fence_after();
        if (live) {
          p.pp.ml[rec] = make_float2(m, lsum);
          px_add_o<D>(tO, acc);
          // (a lane that stores its own row, 16 bytes here and there, cost one layer 1.8 of 12.3 us)
          constexpr int CC = D / 4;              // dimensions at a time
          uint8_t* stage = Qs + warp * (32 * CC * 4);
          float* dst = p.pp.o + group * 128 * D + (int64_t)row0 * D;
#pragma unroll
          for (int d0 = 0; d0 < D; d0 += CC) {
#pragma unroll
            for (int k = 0; k < CC / 4; ++k)
              *reinterpret_cast<float4*>(stage + lane * CC * 4 + ((k ^ (lane & (CC / 4 - 1))) << 4)) =
                  make_float4(acc[d0 + 4 * k], acc[d0 + 4 * k + 1], acc[d0 + 4 * k + 2], acc[d0 + 4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int x = lane; x < 32 * (CC / 4); x += 32) {
              const int r = x / (CC / 4), k = x % (CC / 4);
              const float4 v = *reinterpret_cast<const float4*>(stage + r * CC * 4 + ((k ^ (r & (CC / 4 - 1))) << 4));
              *reinterpret_cast<float4*>(dst + (int64_t)r * D + d0 + 4 * k) = v;
            }
            __syncwarp();
          }
        }
        fence_before();
      } else if (live) {
        p.pp.ml[rec] = make_float2(-INFINITY, 0.f);
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side
// Byte strides (token, head, layer) of the 4-D map below.  A dimension of extent 1 gets the stride its
// inner neighbour implies (any legal value works).
static bool px_strides(int64_t (&s)[3], int64_t sl, int64_t sh, int64_t st, const PrefixParams& p) {
  const int64_t dims[4] = {p.d, p.max_p, p.Hkv, p.L};
  s[0] = dims[1] == 1 ? p.d * 2 : st;
  s[1] = dims[2] == 1 ? s[0] * dims[1] : sh;
  s[2] = dims[3] == 1 ? s[1] * dims[2] : sl;
  for (int i = 0; i < 3; ++i)
    if (s[i] <= 0 || s[i] % 16 || s[i] >= (1LL << 40)) return false;
  return true;
}

// 4-D map (dim, token, KV head, layer) with 64 x 128-token boxes, 128B swizzle.
static bool px_map(CUtensorMap* m, const char* base, int64_t sl, int64_t sh, int64_t st, const PrefixParams& p) {
  int64_t s[3];
  if (!px_strides(s, sl, sh, st, p)) return false;
  cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.max_p, (cuuint64_t)p.Hkv, (cuuint64_t)p.L};
  cuuint64_t strides[3] = {(cuuint64_t)s[0], (cuuint64_t)s[1], (cuuint64_t)s[2]};
  cuuint32_t box[4] = {64, PX_KEYS, 1, 1};
  return bf16_map(m, base, 4, dims, strides, box);
}

// bf16 queries and keys, at most 128 layers, and cache layouts a TMA map can describe.
bool prefix_tc_supported(const PrefixParams& p) {
  if (!p.qbf16 || !p.kbf16 || (p.d != 64 && p.d != 128) || p.L > PREFIX_TC_LAYERS) return false;
  if (((uintptr_t)p.q | (uintptr_t)p.Kp | (uintptr_t)p.Vp) % 16) return false;
  int64_t s[3];
  return px_strides(s, p.Kpl, p.Kph, p.Kpt, p) && px_strides(s, p.Vpl, p.Vph, p.Vpt, p);
}

template <int D, int MT, bool HAS_R>
static cudaError_t launch_px(const PrefixParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  auto kern = prefix_tc_kernel<D, MT, HAS_R>;
  cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, PX_THREADS, px_smem<D, MT>(), st>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_prefix_tc(const PrefixParams& p, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!px_map(&mk, p.Kp, p.Kpl, p.Kph, p.Kpt, p) || !px_map(&mv, p.Vp, p.Vpl, p.Vph, p.Vpt, p))
    return cudaErrorInvalidValue;
#define KVC_PX(DV, MTV) return p.R ? launch_px<DV, MTV, true>(p, mk, mv, st) : launch_px<DV, MTV, false>(p, mk, mv, st)
  if (p.d == 128) {
    if (p.mt == 1) KVC_PX(128, 1);
    KVC_PX(128, 2);
  }
  if (p.mt == 1) KVC_PX(64, 1);
  KVC_PX(64, 2);
#undef KVC_PX
}

}  // namespace kvc
