// Page tables, slot maps and the append into pages.
//
// page_tables_kernel.  Row r holds len tokens in ceil(len / page) pages and is to hold
// len_new: take(r) = max(0, need - have) pages leave the ring of free pages at its head,
// free(r) = max(0, have - need) join it at its tail, and max(0, len_new - len) slots are
// written.  Where a row's pages and slots go depends on the sums of take, free and new tokens
// over the rows before it, and whether anything may be written at all on the sums over all
// rows.  Every CTA forms those sums itself from the two length arrays (8 bytes a row, out of
// L2), a thread to a run of rows and one scan over the threads: no CTA waits for another and
// one launch does it all.  The price is grid * rows * 8 bytes of L2 reads.  Bound by latency: 224 rows 5
// us, 2048 prompts with 1.0 M slots 8.5, 8192 rows with 1.8 M words to write 13.7.
// What there is to write is one sequence of elements, row after row: the row's own entry
// (slot_start, len_out), its pages, its slots.  A warp serves an equal share of that sequence,
// not of the rows: the rows of a new prompt are neighbours, and shares of rows left a few
// CTAs with nearly all slots.
// Taken pages come from ring places [head, head + taken), freed ones go to
// [head + count, ...): the two ranges never meet, because only pages that were free before
// the call are taken.  So no place of the ring is read and written in one call.
// When len_out or state_out is the input array itself, a CTA that is done must not overwrite
// what another still sums: the verdict goes to the workspace and page_commit_kernel, one
// more launch, writes the lengths and the state.
//
// page_append_kernel.  Token t's K and V rows are copied to slot slots[t] in 16-byte pieces;
// a thread carries two pieces of K and two of V, so four loads are in flight before the first
// store.  Bound by HBM: 4 * T * Hkv * row bytes read and written (65536 tokens of 8 heads of 128,
// bf16: 537 MB in 84 us, 6.4 TB/s).
#include "kernels.cuh"

namespace kvc {

constexpr int PT_THREADS = 1024;
constexpr int PT_WARPS = PT_THREADS / 32;

struct RowWork {
  int have, need, take, free, add;
  bool bad;
};

__device__ __forceinline__ RowWork row_work(int a, int z, int shift, int cap_tok) {
  RowWork w;
  w.bad = a < 0 || z < 0 || a > cap_tok || z > cap_tok;
  if (w.bad) a = z = 0;
  const int m = (1 << shift) - 1;
  w.have = (int)(((unsigned)a + m) >> shift);
  w.need = (int)(((unsigned)z + m) >> shift);
  w.take = max(0, w.need - w.have);
  w.free = max(0, w.have - w.need);
  w.add = max(0, z - a);
  return w;
}

// Rows of at most so many elements in a warp's share are served together, longer ones in turn.
constexpr int PT_SHORT = 64;

__global__ void __launch_bounds__(PT_THREADS) page_tables_kernel(PageTablesParams p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = p.shift, page = 1 << shift;
  const int cap_tok = (int)min((long long)p.max_pages << shift, 0x7fffffffLL);

  // this thread's rows [r0, r1), a multiple of four of them, and their sums of take, free, add
  const int run = (((p.rows + PT_THREADS - 1) / PT_THREADS) + 3) & ~3;
  const int r0 = (int)min((long long)p.rows, (long long)tid * run), r1 = min(p.rows, r0 + run);
  const bool vec = (((uintptr_t)p.len | (uintptr_t)p.len_new) & 15) == 0;
  const int head = p.state[0], count = p.state[1];
  long long sum[3] = {0, 0, 0};
  int bad = 0;
  auto add_row = [&](int a, int z) {
    const RowWork w = row_work(a, z, shift, cap_tok);
    bad |= w.bad;
    sum[0] += w.take;
    sum[1] += w.free;
    sum[2] += w.add;
  };
  int r = r0;
  if (vec)
#pragma unroll 2
    for (; r + 4 <= r1; r += 4) {
      const int4 a = *reinterpret_cast<const int4*>(p.len + r), z = *reinterpret_cast<const int4*>(p.len_new + r);
      add_row(a.x, z.x);
      add_row(a.y, z.y);
      add_row(a.z, z.z);
      add_row(a.w, z.w);
    }
  for (; r < r1; ++r) add_row(p.len[r], p.len_new[r]);

  // Sums of the threads before this one, and of all.  They are taken modulo 2^32, and hold where
  // the whole is below it, which its fp64 sum (exact here) tells.
  __shared__ unsigned red[PT_WARPS][3];
  __shared__ double red_all[PT_WARPS];
  __shared__ int red_bad[PT_WARPS];
  __shared__ unsigned s_first[PT_THREADS], s_pre[3][PT_THREADS];   // of each thread's run: first element, sums before it
  unsigned pre[3], tot[3];
  double all = (double)(sum[0] + sum[1] + sum[2] + (r1 - r0));
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    unsigned v = (unsigned)sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(FULL, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) red[warp][k] = v;
    pre[k] = v - (unsigned)sum[k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(FULL, all, o);
  bad = __any_sync(FULL, bad);
  if (lane == 0) {
    red_all[warp] = all;
    red_bad[warp] = bad;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const unsigned x = lane < PT_WARPS ? red[lane][k] : 0;
    tot[k] = __reduce_add_sync(FULL, x);
    pre[k] += __reduce_add_sync(FULL, lane < warp ? x : 0);
  }
  all = lane < PT_WARPS ? red_all[lane] : 0.;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(FULL, all, o);
  const unsigned with_slots = p.slots ? 1u : 0u;
  s_first[tid] = (unsigned)r0 + pre[0] + pre[1] + with_slots * pre[2];
#pragma unroll
  for (int k = 0; k < 3; ++k) s_pre[k][tid] = pre[k];
  bad = __any_sync(FULL, lane < PT_WARPS && red_bad[lane]);

  const bool ok = !bad && all < 4294967296. && head >= 0 && head < p.n_pages && count >= 0 && count <= p.n_pages &&
                  tot[0] <= (unsigned)count && (long long)count + tot[1] <= p.n_pages &&
                  (!p.slots || (long long)tot[2] <= p.slots_cap) && tot[2] <= 0x7fffffffu;
  const unsigned np = (unsigned)p.n_pages;
  auto wrap = [&](unsigned x) { return x >= np ? x - np : x; };           // of a sum of two places, below 2^32
  const int new_head = ok ? (int)wrap((unsigned)head + tot[0]) : head;
  const int new_count = ok ? (int)((unsigned)count - tot[0] + tot[1]) : count;
  const int gtid = blockIdx.x * PT_THREADS + tid, gthreads = gridDim.x * PT_THREADS;
  if (gtid == 0) {
    if (!ok) flag(p.status, ST_BOUNDS);
    if (p.commit) {                           // page_commit_kernel writes the state
      p.commit[0] = ok;
      p.commit[1] = new_head;
      p.commit[2] = new_count;
    } else {
      p.state_out[0] = new_head;
      p.state_out[1] = new_count;
    }
    if (p.slot_start) p.slot_start[p.rows] = ok ? (int)tot[2] : 0;
  }
  // the tail of the slot map
  if (p.slots)
    for (long long i = (ok ? (long long)tot[2] : 0) + gtid; i < p.slots_cap; i += gthreads) p.slots[i] = -1;
  if (!ok) {
    for (long long r = gtid; r < p.rows; r += gthreads) {
      if (p.slot_start) p.slot_start[r] = 0;
      if (p.len_out && !p.commit) p.len_out[r] = p.len[r];
    }
    return;
  }
  const unsigned tail = wrap((unsigned)head + (unsigned)count);
  __syncthreads();

  // this warp's share [c0, c1) of the elements, from the run of rows that holds c0 on
  const unsigned n_all = (unsigned)p.rows + tot[0] + tot[1] + with_slots * tot[2];
  const unsigned long long share = ((unsigned long long)n_all + gridDim.x * PT_WARPS - 1) / (gridDim.x * PT_WARPS);
  const unsigned long long at = ((share + 31) & ~31ull) * ((unsigned long long)blockIdx.x * PT_WARPS + warp);
  if (at >= n_all) return;
  const unsigned c0 = (unsigned)at, c1 = (unsigned)min((unsigned long long)n_all, at + ((share + 31) & ~31ull));
  const int grp = 31 - __clz(__ballot_sync(FULL, s_first[lane * 32] <= c0));       // (an empty run's is n_all)
  const int t = grp * 32 + 31 - __clz(__ballot_sync(FULL, s_first[grp * 32 + lane] <= c0));
  unsigned off = s_first[t], base[3] = {s_pre[0][t], s_pre[1][t], s_pre[2][t]};

  struct Row {
    int r, a, have, more;                     // more: pages to come (to go where negative)
    unsigned pages, add;                      // the row's first place among all pages taken (freed), its first slot's
  };
  // Element g of row q behind its own entry: what goes where.  What is loaded here is not written
  // in this call, so a thread may load for several elements before it stores.
  auto element = [&](const Row& q, int g, int& val) -> int32_t* {
    int32_t* trow = p.table + (int64_t)q.r * p.table_row;
    if (q.more < 0) {                         // a shrinking row has freed pages alone
      val = trow[q.have + q.more + g];
      if ((unsigned)val >= np) flag(p.status, ST_BOUNDS);
      return p.ring + wrap(tail + q.pages + g);                  // count + all freed pages <= n_pages
    }
    const int x = g - q.more, tok = q.a + x;
    const int pg = x < 0 ? q.have + g : tok >> shift;
    const int id = pg < q.have ? trow[pg] : p.ring[wrap((unsigned)head + q.pages + (pg - q.have))];
    const bool in = (unsigned)id < np;
    if (!in) flag(p.status, ST_BOUNDS);
    val = x < 0 ? id : in ? (id << shift) + (tok & (page - 1)) : -1;
    return x < 0 ? trow + pg : p.slots + q.add + x;
  };
  for (int rb = t * run; rb < p.rows && off < c1; rb += 32) {
    const bool valid = rb + lane < p.rows;
    Row q{rb + lane, valid ? p.len[rb + lane] : 0, 0, 0, 0, 0};
    const int z = valid ? p.len_new[q.r] : 0;
    const RowWork w = row_work(q.a, z, shift, cap_tok);
    unsigned v[4] = {(unsigned)w.take, (unsigned)w.free, (unsigned)w.add,
                     valid ? 1 + w.take + w.free + with_slots * w.add : 0u};
    const unsigned n = v[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned y = __shfl_up_sync(FULL, v[k], o);
        if (lane >= o) v[k] += y;
      }
    }
    q.have = w.have;
    q.more = w.need - w.have;
    q.pages = w.free ? base[1] + v[1] - w.free : base[0] + v[0] - w.take;
    q.add = base[2] + v[2] - w.add;
    const unsigned mine = off + v[3] - n, end = min(mine + n, c1);
    int g0 = 0, g1 = 0;
    if (mine < end && end > c0) {
      if (mine >= c0) {
        if (p.slot_start) p.slot_start[q.r] = (int)q.add;
        if (p.len_out && !p.commit) p.len_out[q.r] = z;
      } else {
        g0 = (int)(c0 - mine - 1);
      }
      g1 = (int)(end - mine - 1);
    }
    // Short rows together, an element to a lane, which finds its row in the scan of their lengths:
    // one by one, each waits for its loads (8192 rows of ~30 elements: 21.6 us, together 13.7).
    const int some = g1 - g0 <= PT_SHORT ? max(0, g1 - g0) : 0;
    int upto = some;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) upto += y;
    }
    const int n_short = __shfl_sync(FULL, upto, 31);
    for (int e = lane; e - lane < n_short; e += 64) {
      int32_t* dst[2];
      int val[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = e + 32 * k;
        int src = 0;                          // rows whose elements end at or before x
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(FULL, upto, src + o - 1) <= x) src += o;
        Row u;
        u.r = rb + src;
        u.a = __shfl_sync(FULL, q.a, src);
        u.have = __shfl_sync(FULL, q.have, src);
        u.more = __shfl_sync(FULL, q.more, src);
        u.pages = __shfl_sync(FULL, q.pages, src);
        u.add = __shfl_sync(FULL, q.add, src);
        const int g = __shfl_sync(FULL, g0 - upto + some, src) + x;
        if (x < n_short) dst[k] = element(u, g, val[k]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (e + 32 * k < n_short) *dst[k] = val[k];
    }
    for (unsigned left = __ballot_sync(FULL, g1 - g0 > PT_SHORT); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      Row u;
      u.r = rb + src;
      u.a = __shfl_sync(FULL, q.a, src);
      u.have = __shfl_sync(FULL, q.have, src);
      u.more = __shfl_sync(FULL, q.more, src);
      u.pages = __shfl_sync(FULL, q.pages, src);
      u.add = __shfl_sync(FULL, q.add, src);
      const unsigned last = __shfl_sync(FULL, g1, src);
      for (unsigned g = __shfl_sync(FULL, g0, src) + lane; g < last; g += 128) {
        int32_t* dst[4];
        int val[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (g + 32 * k < last) dst[k] = element(u, g + 32 * k, val[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (g + 32 * k < last) *dst[k] = val[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) base[k] += __shfl_sync(FULL, v[k], 31);
    off += __shfl_sync(FULL, v[3], 31);
  }
}

__global__ void __launch_bounds__(256) page_commit_kernel(const int32_t* commit, const int32_t* len,
                                                          const int32_t* len_new, int32_t* len_out, int rows,
                                                          int32_t* state_out) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i == 0) {
    state_out[0] = commit[1];
    state_out[1] = commit[2];
  }
  if (len_out && i < rows) len_out[i] = commit[0] ? len_new[i] : len[i];
}

cudaError_t launch_page_tables(const PageTablesParams& p, cudaStream_t st) {
  // one CTA to 512 rows and slots (their count is bounded by the slot map's length), one to an SM at most
  const long long most = num_sms();
  const int grid = (int)std::min(most, (p.rows + (p.slots ? (long long)p.slots_cap : 0) + 511) / 512);
  page_tables_kernel<<<grid, PT_THREADS, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  if (p.commit) {
    page_commit_kernel<<<(p.rows + 255) / 256, 256, 0, st>>>(p.commit, p.len, p.len_new, p.len_out, p.rows, p.state_out);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch();
  }
  return e;
}

// --------------------------------------------------------------------------- append
constexpr int PA_THREADS = 256;
constexpr int PA_ITEMS = 2;                    // 16-byte pieces of K (and of V) a thread

__global__ void __launch_bounds__(PA_THREADS) page_append_kernel(PageAppendParams p) {
  const int64_t total = (int64_t)p.T * p.Hkv * p.vr;
  const int64_t base = (int64_t)blockIdx.x * (PA_THREADS * PA_ITEMS) + threadIdx.x;
  const int nv = p.Hkv * p.vr;
  uint4 kk[PA_ITEMS], vv[PA_ITEMS];
  int64_t ko[PA_ITEMS], vo[PA_ITEMS];
#pragma unroll
  for (int i = 0; i < PA_ITEMS; ++i) {
    const int64_t x = base + (int64_t)i * PA_THREADS;
    ko[i] = -1;
    if (x < total) {
      const int t = total <= 0x7fffffff ? (int)x / nv : (int)(x / nv);
      const int c = (int)(x - (int64_t)t * nv), g = c / p.vr, v = c - g * p.vr;
      const int slot = __ldg(p.slots + t);
      if (slot >= 0) {
        const int pg = slot >> p.shift, off = slot & ((1 << p.shift) - 1);
        if (pg < p.n_pages) {
          kk[i] = ld_stream16(p.k + t * p.kst + g * p.ksh + v * 16);
          vv[i] = ld_stream16(p.v + t * p.vst + g * p.vsh + v * 16);
          ko[i] = pg * p.Ksp + g * p.Ksh + off * p.Kst + v * 16;
          vo[i] = pg * p.Vsp + g * p.Vsh + off * p.Vst + v * 16;
        } else if (c == 0) {
          flag(p.status, ST_BOUNDS);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PA_ITEMS; ++i)
    if (ko[i] >= 0) {
      *reinterpret_cast<uint4*>(p.K + ko[i]) = kk[i];
      *reinterpret_cast<uint4*>(p.V + vo[i]) = vv[i];
    }
}

cudaError_t launch_page_append(const PageAppendParams& p, cudaStream_t st) {
  const int64_t total = (int64_t)p.T * p.Hkv * p.vr;
  const int64_t per = PA_THREADS * PA_ITEMS;
  page_append_kernel<<<(unsigned)((total + per - 1) / per), PA_THREADS, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace kvc
