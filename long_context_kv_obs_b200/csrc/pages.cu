// Page tables, slot maps and the append into pages.
//
// page_tables_kernel.  Row r holds len tokens in ceil(len / page) pages and is to hold
// len_new: take(r) = max(0, need - have) pages leave the ring of free pages at its head,
// free(r) = max(0, have - need) join it at its tail, and max(0, len_new - len) slots are
// written.  Where a row's pages and slots go depends on the sums of take, free and new tokens
// over the rows before it, and whether anything may be written at all on the sums over all
// rows.  Every CTA forms those sums itself from the two length arrays (8 bytes a row, out of
// L2) and then serves its own range of rows: no CTA waits for another and one launch does
// it all.  The price is grid * rows * 8 bytes of L2 reads: 8192 rows on 148 CTAs read 9.7 MB.
// Taken pages come from ring places [head, head + taken), freed ones go to
// [head + count, ...): the two ranges never meet, because only pages that were free before
// the call are taken.  So no place of the ring is read and written in one call.
// When len_out or state_out is the input array itself, a CTA that is done must not overwrite
// what another still sums: the verdict goes to the workspace and page_commit_kernel, one
// more launch, writes the lengths and the state.
//
// page_append_kernel.  Token t's K and V rows are copied to slot slots[t] in 16-byte pieces;
// a thread carries two pieces of K and two of V, so four loads are in flight before the first
// store.  Bound by HBM: 4 * T * Hkv * row bytes read and written.
#include "kernels.cuh"

namespace kvc {

constexpr int PT_THREADS = 512;
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

__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// Inclusive scan of an int over the CTA (every thread calls it); total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* sm, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) sm[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int t = lane < PT_WARPS ? sm[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, t, o);
      if (lane >= o) t += x;
    }
    if (lane < PT_WARPS) sm[lane] = t;
  }
  __syncthreads();
  if (warp > 0) v += sm[warp - 1];
  total = sm[PT_WARPS - 1];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(PT_THREADS) page_tables_kernel(PageTablesParams p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = min((long long)p.rows, (long long)blockIdx.x * p.rows_per_cta), r1 = min(p.rows, r0 + p.rows_per_cta);
  const int shift = p.shift, page = 1 << shift;
  const int cap_tok = (int)min((long long)p.max_pages << shift, 0x7fffffffLL);

  // sums over all rows, and over the rows before this CTA's
  long long s[6] = {0, 0, 0, 0, 0, 0};
  int bad = 0;
  auto add_row = [&](int r, int a, int z) {
    const RowWork w = row_work(a, z, shift, cap_tok);
    bad |= w.bad;
    s[0] += w.take;
    s[1] += w.free;
    s[2] += w.add;
    if (r < r0) {
      s[3] += w.take;
      s[4] += w.free;
      s[5] += w.add;
    }
  };
  const bool vec = (((uintptr_t)p.len | (uintptr_t)p.len_new) & 15) == 0;
  const int nv = vec ? p.rows >> 2 : 0;
#pragma unroll 2
  for (int i = tid; i < nv; i += PT_THREADS) {
    const int4 a = *(reinterpret_cast<const int4*>(p.len) + i);
    const int4 z = *(reinterpret_cast<const int4*>(p.len_new) + i);
    add_row(4 * i, a.x, z.x);
    add_row(4 * i + 1, a.y, z.y);
    add_row(4 * i + 2, a.z, z.z);
    add_row(4 * i + 3, a.w, z.w);
  }
  for (int r = 4 * nv + tid; r < p.rows; r += PT_THREADS) add_row(r, p.len[r], p.len_new[r]);

  __shared__ long long red[PT_WARPS][6];
  __shared__ int red_bad[PT_WARPS];
  __shared__ int scan_sm[PT_WARPS];
  __shared__ int row_take[PT_THREADS], row_free[PT_THREADS], row_add[PT_THREADS];
#pragma unroll
  for (int k = 0; k < 6; ++k) s[k] = warp_sum_ll(s[k]);
  bad = __any_sync(FULL, bad);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < 6; ++k) red[warp][k] = s[k];
    red_bad[warp] = bad;
  }
  __syncthreads();
  bad = 0;
#pragma unroll
  for (int k = 0; k < 6; ++k) s[k] = 0;
  for (int w = 0; w < PT_WARPS; ++w) {
#pragma unroll
    for (int k = 0; k < 6; ++k) s[k] += red[w][k];
    bad |= red_bad[w];
  }
  const int head = p.state[0], count = p.state[1];
  bool ok = !bad && head >= 0 && head < p.n_pages && count >= 0 && count <= p.n_pages && s[0] <= count &&
            (long long)count + s[1] <= p.n_pages && (!p.slots || s[2] <= p.slots_cap) && s[2] <= 0x7fffffffLL;
  const int new_head = ok ? (int)((head + s[0]) % p.n_pages) : head;
  const int new_count = ok ? (int)(count - s[0] + s[1]) : count;
  if (blockIdx.x == 0 && tid == 0) {
    if (!ok) flag(p.status, ST_BOUNDS);
    if (p.commit) {                           // page_commit_kernel writes the state
      p.commit[0] = ok;
      p.commit[1] = new_head;
      p.commit[2] = new_count;
    } else {
      p.state_out[0] = new_head;
      p.state_out[1] = new_count;
    }
    if (p.slot_start) p.slot_start[p.rows] = ok ? (int)s[2] : 0;
  }
  // the tail of the slot map, spread over the grid
  if (p.slots) {
    const int t0 = ok ? (int)s[2] : 0;
    for (long long i = t0 + (long long)blockIdx.x * PT_THREADS + tid; i < p.slots_cap;
         i += (long long)gridDim.x * PT_THREADS)
      p.slots[i] = -1;
  }
  if (!ok) {
    for (int r = r0 + tid; r < r1; r += PT_THREADS) {
      if (p.slot_start) p.slot_start[r] = 0;
      if (p.len_out && !p.commit) p.len_out[r] = p.len[r];
    }
    return;
  }
  // this CTA's rows, PT_THREADS at a time: offsets by a scan, then a warp (or a share of the
  // warps) to a row
  int take0 = (int)s[3], free0 = (int)s[4], add0 = (int)s[5];
  for (int t0 = r0; t0 < r1; t0 += PT_THREADS) {
    const int nr = min(PT_THREADS, r1 - t0);
    const int r = t0 + tid;
    RowWork w{};
    if (tid < nr) {
      const int z = p.len_new[r];
      w = row_work(p.len[r], z, shift, cap_tok);
      if (p.len_out && !p.commit) p.len_out[r] = z;
    }
    int tt, ft, at;
    const int ti = block_scan(w.take, scan_sm, tt), fi = block_scan(w.free, scan_sm, ft),
              ai = block_scan(w.add, scan_sm, at);
    if (tid < nr) {
      row_take[tid] = take0 + ti - w.take;
      row_free[tid] = free0 + fi - w.free;
      row_add[tid] = add0 + ai - w.add;
      if (p.slot_start) p.slot_start[r] = add0 + ai - w.add;
    }
    __syncthreads();
    const int parts = nr >= PT_WARPS ? 1 : PT_WARPS / nr;   // warps to a row
    for (int job = warp; job < nr * parts; job += PT_WARPS) {
      const int i = job / parts, part = job % parts, rr = t0 + i;
      const int a = p.len[rr], z = p.len_new[rr];
      const RowWork q = row_work(a, z, shift, cap_tok);
      int32_t* trow = p.table + (int64_t)rr * p.table_row;
      const int first = part * 32 + lane, step = parts * 32;
      auto ring_at = [&](int j) {             // page id at place head + j of the ring, j < n_pages
        const int x = head + j;
        const int id = p.ring[x >= p.n_pages ? x - p.n_pages : x];
        if ((unsigned)id >= (unsigned)p.n_pages) flag(p.status, ST_BOUNDS);
        return id;
      };
      for (int j = first; j < q.take; j += step) trow[q.have + j] = ring_at(row_take[i] + j);
      for (int j = first; j < q.free; j += step) {
        const int id = trow[q.need + j];
        if ((unsigned)id >= (unsigned)p.n_pages) flag(p.status, ST_BOUNDS);
        int x = head + count;                 // count + all freed pages <= n_pages: one wrap at most
        x = (x >= p.n_pages ? x - p.n_pages : x) + row_free[i] + j;
        p.ring[x >= p.n_pages ? x - p.n_pages : x] = id;
      }
      if (p.slots) {
        int32_t* out = p.slots + row_add[i];
        for (int j = first; j < q.add; j += step) {
          const int t = a + j, pg = t >> shift;
          const int id = pg < q.have ? trow[pg] : ring_at(row_take[i] + (pg - q.have));
          const bool in = (unsigned)id < (unsigned)p.n_pages;
          if (!in) flag(p.status, ST_BOUNDS);
          out[j] = in ? (id << shift) + (t & (page - 1)) : -1;
        }
      }
    }
    __syncthreads();
    take0 += tt;
    free0 += ft;
    add0 += at;
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

cudaError_t launch_page_tables(const PageTablesParams& p0, cudaStream_t st) {
  PageTablesParams p = p0;
  // as many CTAs as give each at least four rows, two to an SM at most: few rows spread over
  // the SMs (a row's slots are written by one CTA), many rows do not repeat the sums too often
  const int most = 2 * num_sms();
  int grid = (p.rows + 3) / 4;
  if (grid > most) grid = most;
  p.rows_per_cta = (p.rows + grid - 1) / grid;
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
