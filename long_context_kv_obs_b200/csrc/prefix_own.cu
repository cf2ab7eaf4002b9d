// Decode attention of every sequence over its own rows, in pages or contiguous, on mma.sync.
//
// A (sequence, layer, KV head) row has G <= 8 query rows against len[b][l] keys of its own, so each
// key is used G times and the pass is bound by HBM: 512 bytes a key (bf16, d = 128).  The query
// rows fill half of the 16 rows of an m16n8k16 A operand; the tensor pipe has room for that
// (a 128-row tcgen05 tile would be 94 % padding here):
//   S = Q K^T   B = K rows by ldmatrix;   O += P V   P as a bf16 pair hi + lo (about 16 bits, so the
//   fp32 output keeps its accuracy), B = V rows by ldmatrix.trans; the softmax runs online.
//
// A producer warp fills a ring of 64-key stages by TMA (128B swizzle); four consumer warps take 16
// keys of a stage each, with a running state of their own, and are merged in shared memory at the
// end of an item, a stretch of at most slo keys of one row.  Persistent CTAs, two an SM; the producer
// runs ahead across items, so short rows (a few hundred keys) still keep the ring full.  It draws
// the items from a counter and hands them on through a short queue: rows differ in length, and dealt
// out in turn the longest share took a quarter more than the mean (0.078 -> 0.063 ms for 896 rows of
// up to 1400 keys).  Who computes an item does not change it.  The first item of a
// CTA is its number: it is loaded while the prompt's kernel, which zeroes the counter, still runs
// elsewhere.  Merging the prompt's records here too, in place of a kernel of its own, doubled the
// time: the consumers wait for those loads while the ring is full.  Every wait is an mbarrier with a
// time limit.  Measured: 16384 rows of 175 keys on average, 1.47 GB in 260 us (5.7 TB/s); 896 rows, 270 MB, 57 us.
// Pages: a stage is four boxes of 16 tokens, the smallest page, each at the place its page's table entry
// says.  The producer's lanes hold 32 entries of the row's table at a time and four of them issue a
// box each.  A page id outside the pool becomes a coordinate past the map, whose box reads
// as zeros.  Boxes wholly behind the row's end are not loaded.
#include "kernels.cuh"
#include "mma_sync.cuh"
#include "tc_sm100.cuh"

namespace kvc {
using namespace tc;

constexpr int PO_KEYS = 64;                     // keys a stage, 16 a consumer warp
constexpr int PO_CW = 4;
constexpr int PO_THREADS = 32 * (1 + PO_CW);
constexpr int PO_ATOM = PO_KEYS * 128;          // 64 rows x 64 bf16 (8 KB)
constexpr int PO_PER_SM = 2;
template <int D> constexpr int po_stage() { return 2 * (D / 64) * PO_ATOM; }

constexpr int PO_Q = 4;                         // items handed on at a time
constexpr int PO_BOX = 16;                      // tokens of a box
constexpr int PO_NB = PO_KEYS / PO_BOX;         // boxes a stage (per K / V atom)

struct PoArgs {
  PrefixParams p;
  int nitems, nst;
};
struct PoCtl {
  uint64_t full[6], empty[6];
  uint64_t q_full[PO_Q], q_empty[PO_Q], upper, second, merged;
  int item[PO_Q], len[PO_Q];                    // an item and its row's length; its queries lie behind
  int abort;
};

template <int D>
__global__ void __launch_bounds__(PO_THREADS, PO_PER_SM)
prefix_own_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                  const __grid_constant__ PoArgs a) {
  constexpr int NA = D / 64, STAGE = po_stage<D>(), REC = D + 2;
  const PrefixParams& p = a.p;
  const int NST = a.nst;
  extern __shared__ __align__(1024) uint8_t po_raw[];
  uint8_t* ring = po_raw;
  PoCtl* c = reinterpret_cast<PoCtl*>(ring + (size_t)NST * STAGE);
  uint8_t* qbuf = ring + (size_t)NST * STAGE + ((sizeof(PoCtl) + 127) & ~(size_t)127);   // [PO_Q][G][D]
  float* dsm = reinterpret_cast<float*>(qbuf + (size_t)PO_Q * p.G * D * 2);              // [2][G][REC]
  uint64_t *full = c->full, *empty = c->empty;
  volatile int* abort = &c->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], PO_CW);
    }
    for (int q = 0; q < PO_Q; ++q) {
      mbar_init(&c->q_full[q], 1);
      mbar_init(&c->q_empty[q], PO_CW);
    }
    mbar_init(&c->upper, 2);
    mbar_init(&c->second, 1);
    mbar_init(&c->merged, 1);
    c->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_map(&mapK);
    prefetch_map(&mapV);
  }
  pdl_launch();
  __syncthreads();
  auto row_len = [&](int bl) {
    const int n = p.len[bl];
    return n < 0 ? 0 : min(n, p.max_len);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool paged = p.table != nullptr;
    uint32_t chunk = 0, nq = 0;
    bool ok = true;
    int drawn = blockIdx.x;
    while (ok) {
      const int item = __shfl_sync(FULL, drawn, 0);
      const bool last = item >= a.nitems;
      const int row = last ? 0 : item / p.nso, split = item - row * p.nso;
      const int bl = row / p.Hkv, g = row - bl * p.Hkv, b = bl / p.L, l = bl - b * p.L;
      const int n = row_len(bl);
      if (lane == 0) {
        // the item, its length and its queries (G rows, one after the other) to the consumers
        const int q = nq % PO_Q;
        ok = mbar_wait(&c->q_empty[q], ((nq / PO_Q) & 1) ^ 1, abort, p.status);
        if (ok) {
          const uint32_t bytes = p.G * D * 2;
          c->item[q] = item;
          c->len[q] = n;
          if (last) {
            mbar_arrive(&c->q_full[q]);
          } else {
            // the next one, while this one is loaded
            if (nq > 0) drawn = (int)gridDim.x + atomicAdd(p.counter, 1);
            mbar_expect_tx(&c->q_full[q], bytes);
            bulk_load(qbuf + q * bytes, reinterpret_cast<const char*>(p.q) + ((int64_t)bl * p.Hq + g * p.G) * D * 2, bytes,
                      &c->q_full[q]);
          }
        }
      }
      ++nq;
      ok = __shfl_sync(FULL, (int)ok, 0) != 0;
      if (!ok || last) break;
      const int s0 = split * p.slo, s1 = min(n, s0 + p.slo);
      const int32_t* trow = paged ? p.table + b * p.tsb + l * p.tsl : nullptr;
      int ent = 0, ent0 = -1;                   // entries ent0 .. ent0 + 31 of the table, one a lane
      for (int i0 = s0; i0 < s1; i0 += PO_KEYS, ++chunk) {
        const int s = chunk % NST;
        const int tok = i0 + lane * PO_BOX;     // this lane's box, lane < PO_NB
        const bool box = lane < PO_NB && tok < s1;
        int pg = 0, off = 0;
        if (paged) {
          const int first = i0 >> p.shift;      // the stage's entries: at most 4 from here
          if (ent0 < 0 || first + 3 >= ent0 + 32) {
            ent0 = first;
            const int e = ent0 + lane, last = (n - 1) >> p.shift;
            ent = e <= last ? __ldg(trow + e) : 0;
            if ((unsigned)ent >= (unsigned)p.n_pages) {
              flag(p.status, ST_BOUNDS);
              ent = p.n_pages;                  // past the map: reads as zeros
            }
          }
          pg = __shfl_sync(FULL, ent, min(31, ((box ? tok : i0) >> p.shift) - ent0));
          off = tok & ((1 << p.shift) - 1);
        }
        const unsigned boxes = __ballot_sync(FULL, box);
        if (lane == 0) {
          ok = mbar_wait(&empty[s], ((chunk / NST) & 1) ^ 1, abort, p.status);
          if (ok) mbar_expect_tx(&full[s], (uint32_t)__popc(boxes) * PO_BOX * 128 * 2 * NA);
        }
        ok = __shfl_sync(FULL, (int)ok, 0) != 0;
        if (!ok) break;
        if (box) {
          uint8_t* st = ring + (size_t)s * STAGE + (size_t)lane * PO_BOX * 128;
          const int c1 = paged ? off : tok, c3 = paged ? pg : l, c4 = paged ? 0 : b;
#pragma unroll
          for (int x = 0; x < NA; ++x) {
            tma_load_5d(st + x * PO_ATOM, &mapK, x * 64, c1, g, c3, c4, &full[s]);
            tma_load_5d(st + (NA + x) * PO_ATOM, &mapV, x * 64, c1, g, c3, c4, &full[s]);
          }
        }
      }
      if (nq == 1) {                            // the first is under way
        pdl_wait();
        if (lane == 0) drawn = (int)gridDim.x + atomicAdd(p.counter, 1);
      }
    }
    pdl_wait();
    if (*abort && lane == 0) {                  // copies in flight end before shared memory is given up
      int none = 0;
      const uint32_t issued = chunk, sent = nq;
      for (uint32_t j = sent > PO_Q ? sent - PO_Q : 0; j < sent; ++j)
        mbar_wait(&c->q_full[j % PO_Q], (j / PO_Q) & 1, &none, p.status);
      for (uint32_t j = issued > (uint32_t)NST ? issued - NST : 0; j < issued; ++j)
        mbar_wait(&full[j % NST], (j / NST) & 1, &none, p.status);
    }
    return;
  }
  // -------------------------------------------------------------- consumers
  const int cw = warp - 1;
  const int gid = lane >> 2, tig = lane & 3;    // accumulator row (query head) and column pair
  const int G = p.G;
  uint32_t chunk = 0, merges = 0;
  for (uint32_t nq = 0;; ++nq) {
    const int q = nq % PO_Q;
    if (nq == 1) pdl_wait();                    // as the producer does: the time limits are for what runs here, not the prompt
    bool fine = mbar_wait(&c->q_full[q], (nq / PO_Q) & 1, abort, p.status);
    if (!__all_sync(FULL, fine)) break;
    const int item = c->item[q], n = c->len[q];
    if (item >= a.nitems) break;
    const int row = item / p.nso, split = item - row * p.nso;
    const int s0 = split * p.slo, s1 = min(n, s0 + p.slo);
    // an item of one stage is one warp's, without a hand-over: the others go on to the next items (5624 rows
    // of at most 68 keys, the whole call: 104 -> 92 us)
    const bool alone = s1 - s0 <= PO_KEYS, idle = alone && cw != (int)(nq & 3);
    uint32_t qa[D / 16][2];
    if (!idle) {
      const uint8_t* qr = qbuf + (size_t)q * G * D * 2 + (size_t)gid * D * 2;
#pragma unroll
      for (int kc = 0; kc < D / 16; ++kc) {
        qa[kc][0] = gid < G ? *reinterpret_cast<const uint32_t*>(qr + (kc * 16 + 2 * tig) * 2) : 0u;
        qa[kc][1] = gid < G ? *reinterpret_cast<const uint32_t*>(qr + (kc * 16 + 8 + 2 * tig) * 2) : 0u;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->q_empty[q]);
    if (cw == 0 && lane == 0 && split == 0 && n != p.len[row / p.Hkv]) flag(p.status, ST_BOUNDS);
    const int64_t rec0 = ((int64_t)row * p.nso + split) * G;
    if (s0 >= s1) {                             // nothing here: records of no weight
      if (cw == 0 && lane < G) p.po.ml[rec0 + lane] = make_float2(-INFINITY, 0.f);
      continue;
    }
    if (idle) {                                 // (a slot's barriers want every warp, once it is filled)
      const int s = chunk % NST;
      fine = !*abort && mbar_wait(&full[s], (chunk / NST) & 1, abort, p.status);
      if (!__all_sync(FULL, fine)) break;
      if (lane == 0) mbar_arrive(&empty[s]);
      ++chunk;
      continue;
    }
    float O[D / 8][4];
#pragma unroll
    for (int t = 0; t < D / 8; ++t) O[t][0] = O[t][1] = O[t][2] = O[t][3] = 0.f;
    float m = -INFINITY, lsum = 0.f;
    for (int i0 = s0; i0 < s1; i0 += PO_KEYS, ++chunk) {
      const int s = chunk % NST;
      const bool ok = !*abort && mbar_wait(&full[s], (chunk / NST) & 1, abort, p.status);
      if (!__all_sync(FULL, ok)) {
        fine = false;
        break;
      }
      uint8_t* st = ring + (size_t)s * STAGE;
      const uint32_t kb = smem_u32(st), vb = kb + NA * PO_ATOM;
#pragma unroll 1
      for (int r0 = alone ? 0 : cw * 16; r0 < (alone ? PO_KEYS : cw * 16 + 16); r0 += 16) {   // this warp's keys
        const int nk = min(PO_KEYS, s1 - i0) - r0;   // valid ones of the 16
        if (nk <= 0) break;
        if (nk < 16) {
          // rows past the end may hold anything: zero V there (P is 0 for them, but 0 * NaN is not)
          for (int i = nk * (D / 8) + lane; i < 16 * (D / 8); i += 32) {
            const int r = r0 + i / (D / 8), ch = i % (D / 8);
            *reinterpret_cast<uint4*>(st + (NA + (ch >> 3)) * PO_ATOM + r * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        float S[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
          const int r = r0 + nt * 8 + (lane & 7);
#pragma unroll
          for (int kc2 = 0; kc2 < D / 32; ++kc2) {
            const int d0 = kc2 * 32 + (lane >> 3) * 8;
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kb + (d0 >> 6) * PO_ATOM + sw_off(r, (d0 & 63) >> 3), b0, b1, b2, b3);
            mma_rows8(S[nt], qa[2 * kc2][0], qa[2 * kc2][1], b0, b1);
            mma_rows8(S[nt], qa[2 * kc2 + 1][0], qa[2 * kc2 + 1][1], b2, b3);
          }
        }
        float x[2][2], mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = nt * 8 + 2 * tig + j;
            x[nt][j] = key < nk ? S[nt][j] * p.qscale : -INFINITY;
            mx = fmaxf(mx, x[nt][j]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        if (mx > m + 8.f) {
          const float corr = ex2(m - mx);
          lsum *= corr;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            O[t][0] *= corr;
            O[t][1] *= corr;
          }
          m = mx;
        }
        float pr[2][2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            pr[nt][j] = x[nt][j] == -INFINITY ? 0.f : ex2(x[nt][j] - m);
            lsum += pr[nt][j];
          }
        const uint32_t h0 = pack_bf16(pr[0][0], pr[0][1]), h2 = pack_bf16(pr[1][0], pr[1][1]);
        const uint32_t l0 = pack_bf16(pr[0][0] - bf_lo(h0), pr[0][1] - bf_hi(h0));
        const uint32_t l2 = pack_bf16(pr[1][0] - bf_lo(h2), pr[1][1] - bf_hi(h2));
        const int r = r0 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int dt2 = 0; dt2 < D / 16; ++dt2) {
          const int d0 = dt2 * 16 + (lane >> 4) * 8;
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(vb + (d0 >> 6) * PO_ATOM + sw_off(r, (d0 & 63) >> 3), b0, b1, b2, b3);
          mma_rows8(O[2 * dt2], h0, h2, b0, b1);
          mma_rows8(O[2 * dt2], l0, l2, b0, b1);
          mma_rows8(O[2 * dt2 + 1], h0, h2, b2, b3);
          mma_rows8(O[2 * dt2 + 1], l0, l2, b2, b3);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    if (!fine) break;
    lsum += __shfl_xor_sync(FULL, lsum, 1);
    lsum += __shfl_xor_sync(FULL, lsum, 2);
    auto record = [&]() {
      if (gid < G) {
        if (tig == 0) p.po.ml[rec0 + gid] = make_float2(m, lsum);
        float* o = p.po.o + (rec0 + gid) * D + 2 * tig;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) *reinterpret_cast<float2*>(o + t * 8) = make_float2(O[t][0], O[t][1]);
      }
    };
    if (alone) {
      record();
      continue;
    }
    // warps 2 and 3 hand their state to 0 and 1, warp 1 its own to 0, which writes the record; the
    // others go on to the next item
    auto hand = [&](int slot) {
      if (gid < G) {
        float* r = dsm + ((size_t)slot * G + gid) * REC;
        if (tig == 0) *reinterpret_cast<float2*>(r + D) = make_float2(m, lsum);
#pragma unroll
        for (int t = 0; t < D / 8; ++t) *reinterpret_cast<float2*>(r + t * 8 + 2 * tig) = make_float2(O[t][0], O[t][1]);
      }
      __syncwarp();
    };
    auto take = [&](int slot) {
      if (gid < G) {
        const float* r = dsm + ((size_t)slot * G + gid) * REC;
        const float2 x = *reinterpret_cast<const float2*>(r + D);
        const float M = fmaxf(m, x.x), ref = M == -INFINITY ? 0.f : M, a0 = ex2(m - ref), a1 = ex2(x.x - ref);
        m = M;
        lsum = lsum * a0 + x.y * a1;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          const float2 y = *reinterpret_cast<const float2*>(r + t * 8 + 2 * tig);
          O[t][0] = O[t][0] * a0 + y.x * a1;
          O[t][1] = O[t][1] * a0 + y.y * a1;
        }
      }
      __syncwarp();
    };
    if (cw >= 2) {
      // the slots of the item before have been read
      if (merges > 0) fine = mbar_wait(&c->merged, (merges - 1) & 1, abort, p.status);
      if (!__all_sync(FULL, fine)) break;
      hand(cw - 2);
      if (lane == 0) mbar_arrive(&c->upper);
    } else {
      fine = mbar_wait(&c->upper, merges & 1, abort, p.status);
      if (!__all_sync(FULL, fine)) break;
      take(cw);
      if (cw == 1) {
        hand(1);
        if (lane == 0) mbar_arrive(&c->second);
      } else {
        fine = mbar_wait(&c->second, merges & 1, abort, p.status);
        if (!__all_sync(FULL, fine)) break;
        take(1);
        if (lane == 0) mbar_arrive(&c->merged);
        record();
      }
    }
    ++merges;
  }
}

// ---------------------------------------------------------------- host side
// Byte strides of the 5-D map below; a dimension of extent 1 gets its inner neighbour's.
static bool po_strides(int64_t (&s)[4], int64_t sb, int64_t sl, int64_t sh, int64_t st, const PrefixParams& p) {
  const bool paged = p.table != nullptr;
  const int64_t dims[5] = {p.d, paged ? 1 << p.shift : p.max_len, p.Hkv, paged ? p.n_pages : p.L, paged ? 1 : p.B};
  const int64_t in[4] = {st, sh, paged ? sb : sl, sb};
  for (int i = 0; i < 4; ++i) {
    s[i] = dims[i + 1] > 1 ? in[i] : i ? s[i - 1] : p.d * 2;
    if (s[i] <= 0 || s[i] % 16 || s[i] >= (1LL << 40)) return false;
  }
  return true;
}

// 5-D map: (dim, token, KV head, layer, sequence), or (dim, token of the page, KV head, page, 1).
static bool po_map(CUtensorMap* m, const char* base, int64_t sb, int64_t sl, int64_t sh, int64_t st,
                   const PrefixParams& p) {
  int64_t s[4];
  if (!po_strides(s, sb, sl, sh, st, p)) return false;
  const bool paged = p.table != nullptr;
  cuuint64_t dims[5] = {(cuuint64_t)p.d, (cuuint64_t)(paged ? 1 << p.shift : p.max_len), (cuuint64_t)p.Hkv,
                        (cuuint64_t)(paged ? p.n_pages : p.L), (cuuint64_t)(paged ? 1 : p.B)};
  cuuint64_t strides[4] = {(cuuint64_t)s[0], (cuuint64_t)s[1], (cuuint64_t)s[2], (cuuint64_t)s[3]};
  cuuint32_t box[5] = {64, PO_BOX, 1, 1, 1};
  return bf16_map(m, base, 5, dims, strides, box);
}

bool prefix_own_mma_supported(const PrefixParams& p) {
  if (!p.qbf16 || !p.kbf16 || (p.d != 64 && p.d != 128) || p.G > 8) return false;
  if (((uintptr_t)p.q | (uintptr_t)p.K | (uintptr_t)p.V) % 16) return false;
  int64_t s[4];
  return po_strides(s, p.Ksb, p.Ksl, p.Ksh, p.Kst, p) && po_strides(s, p.Vsb, p.Vsl, p.Vsh, p.Vst, p);
}

template <int D>
static cudaError_t launch_po(const PrefixParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  PoArgs a{};
  a.p = p;
  a.nitems = p.B * p.L * p.Hkv * p.nso;
  int dev = 0, smem_sm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  // two CTAs an SM, as many stages (at most 6) as fit beside the queries and merge records (1 KB a CTA is
  // the runtime's)
  const size_t fixed = ((sizeof(PoCtl) + 127) & ~(size_t)127) + (size_t)PO_Q * p.G * D * 2 + (size_t)2 * p.G * (D + 2) * 4;
  const long long room = (long long)smem_sm / PO_PER_SM - 1024 - (long long)fixed;
  a.nst = (int)(room / po_stage<D>());
  if (a.nst > 6) a.nst = 6;
  if (a.nst < 2) return cudaErrorInvalidConfiguration;
  const size_t smem = fixed + (size_t)a.nst * po_stage<D>();
  auto kern = prefix_own_kernel<D>;
  cudaError_t e = allow_smem(kern);
  if (e != cudaSuccess) return e;
  int grid = PO_PER_SM * num_sms();
  if (!p.counter_zeroed && (e = cudaMemsetAsync(p.counter, 0, sizeof(int), st)) != cudaSuccess) return e;
  if (grid > a.nitems) grid = a.nitems;
  e = launch_dependent(kern, dim3(grid), PO_THREADS, smem, st, p.counter_zeroed != 0, mk, mv, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_prefix_own_mma(const PrefixParams& p, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!po_map(&mk, p.K, p.Ksb, p.Ksl, p.Ksh, p.Kst, p) || !po_map(&mv, p.V, p.Vsb, p.Vsl, p.Vsh, p.Vst, p))
    return cudaErrorInvalidValue;
  return p.d == 128 ? launch_po<128>(p, mk, mv, st) : launch_po<64>(p, mk, mv, st);
}

}  // namespace kvc
