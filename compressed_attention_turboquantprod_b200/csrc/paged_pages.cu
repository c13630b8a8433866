// Page management of the paged 8-bit cache: taking pages for new tokens, forking, copying,
// freeing and compacting.  Sequences are rows of a page table on the device, pages carry
// reference counts, and every decision is made on the device from that state, so the calls
// need no host copy of any length and replay in CUDA graphs.
//
// One CTA plans (a call names at most `slots` sequences; prefix sums over them and a walk
// over the reference counts for free pages, lowest first, so the result does not depend on
// timing), a grid then moves bytes.  A full page is never written again, so a fork shares
// it by its count; only the last, partly filled page and the exact tail are copied.
//
// Measured: 906 pages of 2 layers (238 MB) moved in 73 us, 6.5 TB/s of reads and writes, the copy peak; a
// plan takes 4-10 us (one CTA, latency).
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 16384;      // bytes a CTA moves per item

// Inclusive prefix sum over the CTA (kPlanThreads threads), `s` of 32 entries; every thread
// gets its own sum, *all the total.
template <typename I>
__device__ __forceinline__ I block_scan(I v, I* s, I* all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                     // s may still be read from the last call
  if (lane == 31) s[w] = v;
  __syncthreads();
  if (w == 0) {
    I t = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const I u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    s[lane] = t;
  }
  __syncthreads();
  *all = s[31];
  return v + (w ? s[w - 1] : 0);
}

// The `need` lowest free pages, in order: take(r, page) for the r-th.  The caller has
// checked that there are that many.  Each thread looks at four counts per round.
template <typename F>
__device__ void take_pages(const PGeom& g, int need, int* s, F take) {
  const int low = g.state->low;
  int got = 0, p0 = low & ~3, last = low;
  while (got < need && p0 < g.pages) {                     // uniform
    const int p = p0 + 4 * threadIdx.x;
    int f[4], c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = p + i >= low && p + i < g.pages && g.ref[p + i] == 0;
      c += f[i];
    }
    int all;
    int r = got + block_scan(c, s, &all) - c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (f[i]) {
        if (r < need) {
          g.ref[p + i] = 1;
          take(r, p + i);
        }
        ++r;
      }
    got += all;
    last = min(p0 + 4 * kPlanThreads, g.pages);
    p0 += 4 * kPlanThreads;
  }
  // every page below the last one looked at is in use, unless that round had more free
  // pages than were needed: then only those before its round are known to be
  __syncthreads();
  if (threadIdx.x == 0) {
    if (need > 0) g.state->low = got == need ? last : max(low, last - 4 * kPlanThreads);
    g.state->n_free -= need;
  }
}

// The index i in [0, n) with scan[i] <= x < scan[i + 1].
__device__ __forceinline__ int find_row(const int* scan, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (scan[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void k_paged_init(PGeom g) {
  pdl_wait();
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < g.slots; i += kPlanThreads) g.claim[i] = -1;
  if (threadIdx.x == 0) g.state->n_free = g.pages;
}

// ---------------------------------------------------------------- extend
// Row i appends cu[i + 1] - cu[i] tokens to slot slots[i] (slot -1: its tokens are left
// out).  All or nothing: any error, a row past the `total` input tokens (-1: not known) among them,
// sets a status bit and the plan stays empty.
__global__ void __launch_bounds__(kPlanThreads, 1) k_paged_extend(PGeom g, const int* slots, const int* cu, int n,
                                                                  int64_t total) {
  __shared__ int s_scan[32];
  __shared__ unsigned long long s_scan2[32];
  __shared__ int s_bad, s_need, s_items, s_end;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  if (tid == 0) {
    s_bad = 0;
    s_need = 0;
    s_items = 0;
    s_end = 0;
    g.state->n_rows = 0;
    g.state->n_items = 0;
  }
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, items = 0, bad = 0;
    if (i < n) {
      const int slot = slots[i], a = cu[i], b = cu[i + 1];
      int count = b - a, start = 0;
      if (a < 0 || b < a) {
        bad |= kPagedBadOffsets;
      } else if (slot == -1) {
        count = 0;
      } else if ((unsigned)slot >= (unsigned)g.slots || atomicCAS(&g.claim[slot], -1, i) != -1) {
        bad |= kPagedBadSlot;
      } else {
        start = g.len[slot];
        const int64_t end = (int64_t)start + count;
        if (end > (int64_t)g.max_pages * g.page) {
          bad |= kPagedTooLong;
        } else if (count > 0 && total >= 0 && b > total) {
          bad |= kPagedBadOffsets;
        } else if (count > 0) {
          const int first = start / g.page, stop = (int)((end + g.page - 1) / g.page);
          // held below 2^20 + 2 (the most pages a pool has), so that sums over 1024 rows
          // stay in 32 bits; a need past the pool's size is refused below
          need = min(stop - (start + g.page - 1) / g.page, g.pages + 1);
          items = min(stop - first, g.pages + 2);
          atomicMax(&s_end, b);
        }
      }
      if (bad) count = 0;
      g.rows[i] = PagedRow{slot, a, start, count, 0};
    }
    if (bad) atomicOr(&s_bad, bad);
    unsigned long long all;                      // both sums in one scan
    const unsigned long long r = block_scan((unsigned long long)need << 32 | (unsigned)items, s_scan2, &all);
    const int rn = (int)(r >> 32), ri = (int)(r & 0xffffffffu), all_n = (int)(all >> 32), all_i = (int)(all & 0xffffffffu);
    if (i < n) {
      g.scan[i] = s_need + rn - need;
      g.rows[i].item = s_items + ri - items;
    }
    __syncthreads();
    if (tid == 0) {
      s_need = min(s_need + all_n, g.pages + 1);
      s_items = min(s_items + all_i, 1 << 29);
    }
    __syncthreads();
  }
  for (int i = tid; i < n; i += kPlanThreads) {          // claims back to -1
    const int slot = slots[i];
    if ((unsigned)slot < (unsigned)g.slots) g.claim[slot] = -1;
  }
  if (tid == 0) {
    if (s_need > g.state->n_free) s_bad |= kPagedNoPages;
    if (s_bad) atomicOr(&g.state->status, s_bad);
    g.scan[n] = s_need;
  }
  __syncthreads();
  if (s_bad) return;
  const int need = s_need;
  if (need > 0)
    take_pages(g, need, s_scan, [&](int r, int page) {
      const int i = find_row(g.scan, n, r);
      const PagedRow w = g.rows[i];
      int* to = &g.table[(int64_t)w.slot * g.max_pages + (w.start + g.page - 1) / g.page + (r - g.scan[i])];
      if (TQ_CHECKED(to, 4, g.table, 4 * (int64_t)g.slots * g.max_pages, 445)) *to = page;
    });
  for (int i = tid; i < n; i += kPlanThreads) {
    const PagedRow w = g.rows[i];
    if (w.count > 0) g.len[w.slot] = w.start + w.count;
  }
  if (tid == 0) {
    g.state->n_rows = n;
    g.state->n_items = s_items;
    g.state->end = s_end;
  }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kMoveThreads) k_paged_free(PGeom g, const int* slots, int n) {
  __shared__ int s_len;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int slot = slots[i];
    __syncthreads();
    if (threadIdx.x == 0) {
      s_len = 0;
      if ((unsigned)slot < (unsigned)g.slots)
        s_len = atomicExch(&g.len[slot], 0);             // the same slot twice: the second finds 0
      else if (slot != -1)
        atomicOr(&g.state->status, kPagedBadSlot);
    }
    __syncthreads();
    const int np = (s_len + g.page - 1) / g.page;
    int freed = 0, low = g.pages;
    for (int p = threadIdx.x; p < np; p += kMoveThreads) {
      const int pid = g.table[(int64_t)slot * g.max_pages + p];
      if ((unsigned)pid >= (unsigned)g.pages) {
        atomicOr(&g.state->status, kPagedBadPage);
      } else if (atomicSub(&g.ref[pid], 1) == 1) {
        ++freed;
        low = min(low, pid);
      }
    }
    freed = __reduce_add_sync(0xffffffffu, freed);
    low = __reduce_min_sync(0xffffffffu, low);
    if ((threadIdx.x & 31) == 0 && freed) {
      atomicAdd(&g.state->n_free, freed);
      atomicMin(&g.state->low, low);
    }
  }
}

// ---------------------------------------------------------------- fork / copy
// Pair i takes sequence from[i] of `src` to the empty slot to[i] of `dst`.  The plan lists
// the pages to copy in dst.moves and sets the destinations' lengths and new table entries.
__global__ void __launch_bounds__(kPlanThreads, 1) k_paged_branch(PGeom src, PGeom dst, const int* from,
                                                                  const int* to, int n, int share) {
  __shared__ int s_scan[32];
  __shared__ int s_bad, s_need;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const bool same = src.base == dst.base;
  if (tid == 0) {
    s_bad = 0;
    s_need = 0;
    dst.state->n_moves = 0;
    dst.state->n_pairs = 0;
    dst.state->compacted = 0;
  }
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, bad = 0;
    if (i < n) {
      const int a = from[i], b = to[i];
      if ((unsigned)a >= (unsigned)src.slots || (unsigned)b >= (unsigned)dst.slots ||
          atomicCAS(&dst.claim[b], -1, i) != -1) {
        bad |= kPagedBadSlot;
      } else if (dst.len[b] != 0) {
        bad |= kPagedNotEmpty;
      } else {
        const int len = src.len[a];
        const int np = (len + src.page - 1) / src.page;
        need = share ? (len % src.page != 0) : min(np, dst.pages + 1);
        if (np > dst.max_pages) bad |= kPagedTooLong;
      }
    }
    if (bad) atomicOr(&s_bad, bad);
    int all;
    const int r = block_scan(need, s_scan, &all);
    if (i < n) dst.scan[i] = s_need + r - need;
    __syncthreads();
    if (tid == 0) s_need = min(s_need + all, dst.pages + 1);
    __syncthreads();
  }
  // a destination that is also a source of this call would be read while it is written
  if (same)
    for (int i = tid; i < n; i += kPlanThreads) {
      const int a = from[i];
      if ((unsigned)a < (unsigned)src.slots && dst.claim[a] != -1) atomicOr(&s_bad, kPagedBadSlot);
    }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int b = to[i];
    if ((unsigned)b < (unsigned)dst.slots) dst.claim[b] = -1;
  }
  if (tid == 0) {
    if (s_need > dst.state->n_free) s_bad |= kPagedNoPages;
    if (s_bad) atomicOr(&dst.state->status, s_bad);
    dst.scan[n] = s_need;
  }
  __syncthreads();
  if (s_bad) return;
  take_pages(dst, s_need, s_scan, [&](int r, int page) {
    const int i = find_row(dst.scan, n, r);
    const int p = share ? src.len[from[i]] / src.page : r - dst.scan[i];
    dst.table[(int64_t)to[i] * dst.max_pages + p] = page;
    dst.moves[r] = make_int2(src.table[(int64_t)from[i] * src.max_pages + p], page);
  });
  for (int i = tid; i < n; i += kPlanThreads) dst.len[to[i]] = src.len[from[i]];
  if (tid == 0) {
    dst.state->n_moves = s_need;
    dst.state->n_pairs = n;
  }
}

// ---------------------------------------------------------------- compact
// The live pages at or beyond the live count move into the free pages below it, both in
// ascending order: the fewest moves, no page is both read and written.
__global__ void __launch_bounds__(kPlanThreads, 1) k_paged_compact(PGeom g) {
  __shared__ int s_scan[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int live = g.pages - g.state->n_free;
  int holes = 0, high = 0;
  for (int p0 = 0; p0 < g.pages; p0 += 4 * kPlanThreads) {
    const int p = p0 + 4 * tid;
    int f[4], c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = p + i < g.pages && ((g.ref[p + i] == 0) == (p + i < live));
      c += f[i];
    }
    // low and high pages of one round are counted apart: the low ones in the low 16 bits
    int lowc = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) lowc += f[i] && p + i < live;
    int all;
    const int v = lowc | ((c - lowc) << 16);
    const int ex = block_scan(v, s_scan, &all) - v;
    int rl = holes + (ex & 0xffff), rh = high + (ex >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p + i < g.pages) g.remap[p + i] = p + i;
      if (!f[i]) continue;
      if (p + i < live) g.moves[rl++].y = p + i; else g.moves[rh++].x = p + i;
    }
    holes += all & 0xffff;
    high += all >> 16;
  }
  __syncthreads();
  for (int k = tid; k < holes; k += kPlanThreads) {
    const int2 m = g.moves[k];
    g.remap[m.x] = m.y;
    g.ref[m.y] = g.ref[m.x];
    g.ref[m.x] = 0;
  }
  if (tid == 0) {
    g.state->n_moves = holes;
    g.state->n_pairs = 0;
    g.state->compacted = 1;
    g.state->low = live;
  }
}

// ---------------------------------------------------------------- moving bytes
__device__ __forceinline__ void copy16(uint8_t* to, const uint8_t* from, int64_t bytes) {
  // four reads in flight a thread
  int64_t o = 16 * (int64_t)threadIdx.x;
  for (; o + 3 * 16 * kMoveThreads < bytes; o += 4 * 16 * kMoveThreads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(from + o + k * 16 * kMoveThreads);
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(to + o + k * 16 * kMoveThreads) = v[k];
  }
  for (; o < bytes; o += 16 * kMoveThreads) *reinterpret_cast<uint4*>(to + o) = *reinterpret_cast<const uint4*>(from + o);
}

// The moves of the last plan, in all layers; then, for a fork or copy, the exact tails and
// (fork) the shared table entries with their counts, or, for a compact, the renumbering of
// the page tables.
__global__ void __launch_bounds__(kMoveThreads) k_paged_move(PGeom src, PGeom dst, const int* from, const int* to,
                                                             int share) {
  pdl_wait();
  pdl_launch_dependents();
  const PagedState st = *dst.state;
  const int nch = (int)((dst.page_bytes + kMoveChunk - 1) / kMoveChunk);
  const int64_t items = (int64_t)st.n_moves * dst.layers * nch;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int ch = (int)(it % nch);
    const int64_t r = it / nch;
    const int layer = (int)(r % dst.layers);
    const int2 m = dst.moves[r / dst.layers];
    if ((unsigned)m.x >= (unsigned)src.pages || (unsigned)m.y >= (unsigned)dst.pages) {
      if (threadIdx.x == 0) atomicOr(&dst.state->status, kPagedBadPage);
      continue;
    }
    const int64_t o = (int64_t)ch * kMoveChunk;
    if (!TQ_CHECKED(dst.pool + ((int64_t)layer * dst.pages + m.y) * dst.page_bytes, dst.page_bytes, dst.base, dst.total, 441) ||
        !TQ_CHECKED(src.pool + ((int64_t)layer * src.pages + m.x) * src.page_bytes, src.page_bytes, src.base, src.total, 442))
      continue;
    copy16(dst.pool + ((int64_t)layer * dst.pages + m.y) * dst.page_bytes + o,
           src.pool + ((int64_t)layer * src.pages + m.x) * src.page_bytes + o,
           min((int64_t)kMoveChunk, dst.page_bytes - o));
  }
  if (st.compacted) {
    for (int slot = blockIdx.x; slot < dst.slots; slot += gridDim.x) {
      const int np = (dst.len[slot] + dst.page - 1) / dst.page;
      for (int p = threadIdx.x; p < np; p += kMoveThreads) {
        int* e = &dst.table[(int64_t)slot * dst.max_pages + p];
        if ((unsigned)*e < (unsigned)dst.pages) *e = dst.remap[*e];
      }
    }
    return;
  }
  const int es = paged_esize(dst.dtype);
  const int per = dst.layers * 2 * dst.Hkv;
  for (int64_t it = blockIdx.x; it < (int64_t)st.n_pairs * (per + 1); it += gridDim.x) {
    const int i = (int)(it / (per + 1)), k = (int)(it % (per + 1));
    const int a = from[i], b = to[i], len = dst.len[b];
    if (k < per) {
      const int layer = k / (2 * dst.Hkv), kvh = k % (2 * dst.Hkv);
      if (!TQ_CHECKED(paged_tail(dst, layer, b, 0, kvh), dst.tail_head, dst.base, dst.total, 443) ||
          !TQ_CHECKED(paged_tail(src, layer, a, 0, kvh), src.tail_head, src.base, src.total, 444))
        continue;
      copy16(paged_tail(dst, layer, b, 0, kvh), paged_tail(src, layer, a, 0, kvh),
             (int64_t)(len % dst.page) * dst.d * es);
    } else if (share) {
      for (int p = threadIdx.x; p < len / dst.page; p += kMoveThreads) {
        const int pid = src.table[(int64_t)a * src.max_pages + p];
        dst.table[(int64_t)b * dst.max_pages + p] = pid;
        if ((unsigned)pid < (unsigned)dst.pages) atomicAdd(&dst.ref[pid], 1);
      }
    }
  }
}

__global__ void k_paged_clear(PGeom g, int bits) {
  pdl_wait();
  atomicAnd(&g.state->status, ~bits);
}

// Rows of the page table, -1 where a sequence has no page.
__global__ void __launch_bounds__(kMoveThreads) k_paged_table(PGeom g, const int* slots, int n, int* out) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < (int64_t)n * g.max_pages;
       i += (int64_t)gridDim.x * kMoveThreads) {
    const int slot = slots[i / g.max_pages], p = (int)(i % g.max_pages);
    const int np = (paged_len(g, slot) + g.page - 1) / g.page;
    out[i] = p < np ? g.table[(int64_t)slot * g.max_pages + p] : -1;
  }
}

}  // namespace

cudaError_t paged_launch_init(const PGeom& g, cudaStream_t s) {
  // zero codes are finite in both formats: a masked token of a fresh page is harmless
  cudaError_t e = cudaMemsetAsync(g.base, 0, (size_t)g.total, s);
  return e != cudaSuccess ? e : launch_pdl(k_paged_init, dim3(1), dim3(kPlanThreads), 0, s, g);
}

cudaError_t paged_launch_extend(const PGeom& g, const int* slots, const int* cu, int n, int64_t total, cudaStream_t s) {
  return launch_pdl(k_paged_extend, dim3(1), dim3(kPlanThreads), 0, s, g, slots, cu, n, total);
}

cudaError_t paged_launch_free(const PGeom& g, const int* slots, int n, cudaStream_t s) {
  return launch_pdl(k_paged_free, dim3(n < 592 ? n : 592), dim3(kMoveThreads), 0, s, g, slots, n);
}

cudaError_t paged_launch_branch(const PGeom& src, const PGeom& dst, const int* from, const int* to, int n,
                                bool share, cudaStream_t s) {
  cudaError_t e = launch_pdl(k_paged_branch, dim3(1), dim3(kPlanThreads), 0, s, src, dst, from, to, n, (int)share);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_move, dim3(148 * 4), dim3(kMoveThreads), 0, s, src, dst, from, to, (int)share);
}

cudaError_t paged_launch_compact(const PGeom& g, cudaStream_t s) {
  cudaError_t e = launch_pdl(k_paged_compact, dim3(1), dim3(kPlanThreads), 0, s, g);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_move, dim3(148 * 4), dim3(kMoveThreads), 0, s, g, g, (const int*)nullptr,
                    (const int*)nullptr, 0);
}

cudaError_t paged_launch_clear(const PGeom& g, int bits, cudaStream_t s) {
  return launch_pdl(k_paged_clear, dim3(1), dim3(1), 0, s, g, bits);
}

cudaError_t paged_launch_table(const PGeom& g, const int* slots, int n, int* out, cudaStream_t s) {
  const int64_t c = ((int64_t)n * g.max_pages + kMoveThreads - 1) / kMoveThreads;
  return launch_pdl(k_paged_table, dim3((unsigned)(c < 1184 ? c : 1184)), dim3(kMoveThreads), 0, s, g, slots, n, out);
}

TQ_BOUNDS_READER(bounds_flag_paged_pages)

}  // namespace tq
