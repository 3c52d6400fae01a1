// Pages of a paged cache on sm_100a: growing, cutting and freeing sequences with
// copy on write, forks, compaction.  Integer bookkeeping plus copies of whole
// pages; the results are those of the sequential definition in the header
// whatever order the threads run in: lists are ranked by prefix sums; atomics add, or
// take a minimum or maximum of list positions.  Which slot of a resize's hash table a
// sequence claims depends on the order, but not what the slot comes to hold (the lowest
// entry that names it), and only that is read.
//
// Bound by latency for the bookkeeping (a few dependent passes over lists of some
// hundred entries and the reference counts), so the kernels of a call are launched
// with programmatic dependent launch: each is resident, with its lists read, when
// the one before it ends.  The copies are bound by memory (each byte read and
// written once): many small chunks in flight per SM.
// Measured, a call on a stream and on the device: fork of 24 sequences 8.6 and 3.9 us, of
// 192 8.5 and 6.4; compaction of 4096 pages (46 MB to move) 22.6 and 17.1 us, of 32768
// (372 MB) 142 and 139 us, 5.3 TB/s; resizes below.
#include <atomic>
#include <climits>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 128;
constexpr int kMoveChunk = 8192;                   // bytes of a page that a CTA copies at a time
constexpr int kSmallPage = 512;                    // pages up to this many bytes are copied by words
constexpr int kOwnPages = 49152;                   // pages whose counts a resize holds in shared memory
constexpr int kMaskWords = 4096;                   // pages / 32 whose masks fit in shared memory

// Programmatic dependent launch: let the next kernel of the call in; wait until the
// one before is through and its writes are visible.
__device__ __forceinline__ void next_kernel() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void last_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Exclusive prefix sum of one int per thread of the CTA; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                 // warp_sums may still be read by an earlier scan
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;                           // inclusive
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ int pages_of(int len, int page_size) {
  return len <= 0 ? 0 : static_cast<int>((static_cast<uint32_t>(len) + page_size - 1) / page_size);   // < 2^32
}

// to = from, four at a time where both are aligned (`i` of `step` threads).
__device__ __forceinline__ void copy_ints(int32_t* to, const int32_t* from, int64_t n, int64_t i, int64_t step) {
  int64_t done = 0;
  if (((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from)) & 15) == 0) {
    done = n / 4 * 4;
#pragma unroll 4
    for (int64_t k = i; k < n / 4; k += step)
      reinterpret_cast<int4*>(to)[k] = reinterpret_cast<const int4*>(from)[k];
  }
  for (int64_t k = done + i; k < n; k += step) to[k] = from[k];
}

// out = in, for the three arrays of a state; clears the status word.
__global__ void __launch_bounds__(256) copy_state_kernel(PagesParams p) {
  next_kernel();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  copy_ints(p.table_out, p.table_in, static_cast<int64_t>(p.num_seqs) * p.pages_per_seq, i, step);
  copy_ints(p.len_out, p.len_in, p.num_seqs, i, step);
  copy_ints(p.ref_out, p.ref_in, p.num_pages, i, step);
}

// The entry that the k-th unit of an exclusive prefix sum `start` [n] belongs to.
__device__ __forceinline__ int owner_of(const int32_t* start, int n, int k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= k)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// One CTA works out a resize: lengths and reference counts of `out`, which table entries
// are dropped and filled, and the page copies.  The pages that are dropped and taken are
// spread over the threads, whichever entries they belong to.  The table's changes are
// left to the kernel after it (patch_table), so that the grid's other CTAs can copy the
// table meanwhile.  With kOwn the counts of the pool are worked on in shared memory, and
// the state needs no launch of its own to be copied; larger pools have them in `out`,
// where the kernel before has copied them.  Bound by latency: some 25 dependent steps.
// On the device, with and without kOwn: 256 entries that drop 3500 and take 2800 of 24576
// pages 20.0 and 22.8 us; 64 entries of a decode step 8.8 and 7.9 us, but a launch more
// on the host (12 us a call against 13).
template <bool kOwn>
__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(PagesParams p) {
  extern __shared__ __align__(16) int32_t own_ref[];   // kOwn: [num_pages]
  __shared__ int sums[32];
  __shared__ int s_moves;
  __shared__ int s_seq[kPlanThreads], s_want[kPlanThreads], s_old[kPlanThreads], s_last[kPlanThreads];
  __shared__ int s_slot[2 * kPlanThreads];         // first a hash table, then two arrays
  int* const s_at = s_slot;
  int* const s_pos = s_slot + kPlanThreads;
  const int tid = threadIdx.x;
  next_kernel();
  if (blockIdx.x > 0) {
    copy_ints(p.table_out, p.table_in, static_cast<int64_t>(p.num_seqs) * p.pages_per_seq,
              static_cast<int64_t>(blockIdx.x - 1) * kPlanThreads + tid,
              static_cast<int64_t>(gridDim.x - 1) * kPlanThreads);
    return;
  }
  const int P = p.page_size, n = p.n;
  const int64_t top = static_cast<int64_t>(p.pages_per_seq) * P;
  int32_t* ref = kOwn ? own_ref : p.ref_out;
  auto count_of = [&](int pg) { return kOwn ? ref[pg] : __ldcg(&ref[pg]); };
  // The entries' working copies: in shared memory if a pass of the threads takes them all.
  const bool few = n <= kPlanThreads;
  const int32_t* seq = few ? s_seq : p.list_a;
  const int32_t* want = few ? s_want : p.list_b;
  int32_t* old_len = few ? s_old : p.old_len;      // -1: not valid
  int32_t* last_page = few ? s_last : p.last_page; // the partly filled page that an entry grows in, or -1
  int32_t* at = few ? s_at : p.drop_at;            // prefix sums of the entries' dropped pages
  int32_t* pos = few ? s_pos : p.drop_pos;         // table place of the k-th dropped page, minus k
  uint32_t flags = 0;
  if (tid == 0) {
    s_moves = 0;
    if (kOwn) *p.status = 0;
  }
  // An entry is valid if it is in range and the first that names its sequence.  Of few
  // entries the first ones are kept in a hash table in shared memory: a slot belongs to
  // one sequence and holds the lowest entry that names it.  (Comparing every entry with
  // those before it took 3.5 us of 256 entries.)
  auto probe = [&](int s, auto visit) {            // slots of a sequence in turn, until visit says stop
    for (uint32_t h = static_cast<uint32_t>(s) * 2654435761u >> 21; !visit(&s_slot[h & (2 * kPlanThreads - 1)]); ++h) {
    }
  };
  if (few) {
    s_seq[tid] = tid < n ? p.list_a[tid] : -1;
    s_want[tid] = tid < n ? p.list_b[tid] : 0;
    s_slot[tid] = s_slot[kPlanThreads + tid] = -1;
    __syncthreads();
    const int s = s_seq[tid];
    if (s >= 0)
      probe(s, [&](int* slot) {
        const int got = atomicCAS(slot, -1, tid);
        if (got >= 0 && s_seq[got] == s) atomicMin(slot, tid);
        return got < 0 || s_seq[got] == s;
      });
  } else {
    for (int i = tid; i < n; i += kPlanThreads) {
      const int s = p.list_a[i];
      if (s >= 0 && s < p.num_seqs) p.first[s] = INT_MAX;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) {
      const int s = p.list_a[i];
      if (s >= 0 && s < p.num_seqs) atomicMin(&p.first[s], i);
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = seq[i], to = want[i];
    bool ok = s >= 0 && s < p.num_seqs && to >= 0 && to <= top;
    int old = 0;
    if (ok) old = p.len_in[s];
    if (few) {
      int first = -1;
      if (ok)
        probe(s, [&](const int* slot) {
          first = *slot;
          return s_seq[first] == s;
        });
      ok = first == i;
    } else {
      ok = ok && __ldcg(&p.first[s]) == i;
    }
    ok = ok && old >= 0 && old <= top;
    old_len[i] = ok ? old : -1;
    if (!ok) flags |= DSA_DEV_BAD_QUERY;
    int pg = -1;
    if (ok && to > old && old % P != 0) {
      pg = p.table_in[static_cast<int64_t>(s) * p.pages_per_seq + old / P];
      if (pg < 0 || pg >= p.num_pages) {
        flags |= DSA_DEV_BAD_INDEX;
        pg = -1;
      } else {
        p.sharers[pg] = 0;
        p.last_sharer[pg] = -1;
      }
    }
    last_page[i] = pg;
  }
  if (kOwn) {
    // by the warps without an entry, if they are half of them or more
    const int first = n <= kPlanThreads / 2 ? (n + 31) / 32 * 32 : 0;
    if (tid >= first) {
      copy_ints(own_ref, p.ref_in, p.num_pages, tid - first, kPlanThreads - first);
      if (p.len_out != p.len_in) copy_ints(p.len_out, p.len_in, p.num_seqs, tid - first, kPlanThreads - first);
    }
  }
  last_kernel();
  __syncthreads();
  // the pages behind the new lengths of shrinking entries; who shares a last page
  int dropped = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int drop = 0;
    if (i < n && old_len[i] >= 0) {
      const int pg = last_page[i];
      if (want[i] <= old_len[i]) {
        drop = pages_of(old_len[i], P) - pages_of(want[i], P);
        p.len_out[seq[i]] = want[i];
      }
      if (pg >= 0) {
        atomicAdd(&p.sharers[pg], 1);
        atomicMax(&p.last_sharer[pg], i);
      }
    }
    int total;
    const int before = dropped + block_scan(drop, sums, total);
    if (i < n) {
      at[i] = p.drop_at[i] = before;
      pos[i] = p.drop_pos[i] = drop ? seq[i] * p.pages_per_seq + pages_of(want[i], P) - before : 0;
    }
    dropped += total;
  }
  __syncthreads();
  for (int64_t k0 = tid; k0 < dropped; k0 += 4 * kPlanThreads) {
    int pg[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t k = k0 + u * kPlanThreads;
      pg[u] = k < dropped ? p.table_in[pos[owner_of(at, n, static_cast<int>(k))] + k] : INT_MIN;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (pg[u] >= 0 && pg[u] < p.num_pages)
        atomicSub(&ref[pg[u]], 1);
      else if (k0 + u * kPlanThreads < dropped)
        flags |= DSA_DEV_BAD_INDEX;
    }
  }
  __syncthreads();
  // pages that each entry takes, and where its share of the free list begins.  Of the
  // growing sequences on a shared page all copy it, but for the last one if no one
  // else holds the page.
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int take = 0, copy = 0;
    if (i < n && old_len[i] >= 0 && want[i] > old_len[i]) {
      const int pg = last_page[i];
      if (pg >= 0) {
        const int r = count_of(pg);
        copy = r > 1 && !(r <= __ldcg(&p.sharers[pg]) && __ldcg(&p.last_sharer[pg]) == i);
      }
      take = copy + pages_of(want[i], P) - pages_of(old_len[i], P);
    }
    int total;
    const int before = need + block_scan(take, sums, total);
    if (i < n) {
      p.take_at[i] = before;
      p.take_pos[i] = take ? seq[i] * p.pages_per_seq + pages_of(old_len[i], P) - copy - before : 0;
      if (!copy) last_page[i] = -1;                // only the pages to be copied are left
    }
    need += total;
  }
  __syncthreads();
  // the lowest free pages, 16 words of 32 per warp and pass; they are taken as they are found
  constexpr int kWords = 16;
  const int lane = tid & 31;
  int found = 0;
  for (int64_t c0 = 0; c0 < p.num_pages && found < need; c0 += kWords * kPlanThreads) {
    const int64_t pg = c0 + (tid >> 5) * (kWords * 32) + lane;
    bool is_free[kWords];
#pragma unroll
    for (int u = 0; u < kWords; ++u)
      is_free[u] = pg + u * 32 < p.num_pages && count_of(static_cast<int>(pg + u * 32)) == 0;
    uint32_t mask[kWords];
    int mine = 0;
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      mask[u] = __ballot_sync(0xffffffffu, is_free[u]);
      mine += __popc(mask[u]);
    }
    int total;
    int k = found + __shfl_sync(0xffffffffu, block_scan(lane == 0 ? mine : 0, sums, total), 0);
    if (k < need) {
#pragma unroll
      for (int u = 0; u < kWords; ++u) {
        const int at_k = k + __popc(mask[u] & ((1u << lane) - 1));
        if ((mask[u] >> lane & 1) && at_k < need) {
          p.free_list[at_k] = static_cast<int>(pg) + u * 32;
          ref[pg + u * 32] = 1;
        }
        k += __popc(mask[u]);
      }
    }
    found += total;
  }
  __syncthreads();
  if (found < need) {                              // too few: none is taken
    if (tid == 0) set_status(p.status, DSA_DEV_NO_PAGES);
    for (int k = tid; k < found; k += kPlanThreads) ref[p.free_list[k]] = 0;
    need = 0;
  } else {
    for (int i = tid; i < n; i += kPlanThreads) {
      if (!(old_len[i] >= 0 && want[i] > old_len[i])) continue;
      p.len_out[seq[i]] = want[i];
      const int from = last_page[i];
      if (from >= 0) {
        const int m = atomicAdd(&s_moves, 1);
        p.move_src[m] = from;
        p.move_dst[m] = p.free_list[p.take_at[i]];
        atomicSub(&ref[from], 1);
      }
    }
  }
  if (flags) set_status(p.status, flags);
  __syncthreads();
  if (kOwn) copy_ints(p.ref_out, own_ref, p.num_pages, tid, kPlanThreads);
  if (tid == 0) {
    p.num_moves[0] = s_moves;
    p.num_moves[1] = dropped;
    p.num_moves[2] = need;
  }
}

// The table's changes of a resize: dropped entries become -1 (those outside the pool are
// left alone), taken ones get their pages, an entry's copied page first.
__device__ __forceinline__ void patch_table(const PagesParams& p) {
  __shared__ int at[2][kPlanThreads], pos[2][kPlanThreads];
  const int n = p.n;
  const int count[2] = {__ldcg(&p.num_moves[1]), __ldcg(&p.num_moves[2])};   // dropped, taken
  if (blockIdx.x * kMoveThreads >= max(count[0], count[1])) return;
  const bool few = n <= kPlanThreads;              // searched in shared memory
  if (few) {
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
      at[0][i] = p.drop_at[i];
      at[1][i] = p.take_at[i];
      pos[0][i] = p.drop_pos[i];
      pos[1][i] = p.take_pos[i];
    }
    __syncthreads();
  }
  for (int what = 0; what < 2; ++what) {
    const int32_t* a = few ? at[what] : what ? p.take_at : p.drop_at;
    const int32_t* b = few ? pos[what] : what ? p.take_pos : p.drop_pos;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; k < count[what];
         k += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
      const int64_t e = b[owner_of(a, n, static_cast<int>(k))] + k;
      if (what) {
        p.table_out[e] = p.free_list[k];
      } else {
        const int pg = p.table_in[e];
        if (pg >= 0 && pg < p.num_pages) p.table_out[e] = -1;
      }
    }
  }
}

// A CTA per pair: the pair is checked against the whole list.
__global__ void __launch_bounds__(256) fork_kernel(PagesParams p) {
  const int P = p.page_size;
  bool waited = false;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int src = p.list_a[i], dst = p.list_b[i];
    bool ok = src >= 0 && src < p.num_seqs && dst >= 0 && dst < p.num_seqs;
    int len = 0;
    if (ok) {
      len = p.len_in[src];
      ok = p.len_in[dst] == 0 && len >= 0 && len <= static_cast<int64_t>(p.pages_per_seq) * P;
    }
    bool clash = false;
    for (int j = threadIdx.x; j < p.n; j += blockDim.x)
      clash |= p.list_b[j] == src || (j < i && p.list_b[j] == dst);
    ok = !__syncthreads_or(clash) && ok;
    if (!waited) last_kernel();                    // `out` is written from here on
    waited = true;
    if (!ok) {
      if (threadIdx.x == 0) set_status(p.status, DSA_DEV_BAD_QUERY);
      continue;
    }
    const int have = pages_of(len, P);
    const int32_t* from = p.table_in + static_cast<int64_t>(src) * p.pages_per_seq;
    int32_t* to = p.table_out + static_cast<int64_t>(dst) * p.pages_per_seq;
    for (int j = threadIdx.x; j < p.pages_per_seq; j += blockDim.x) {
      const int pg = j < have ? from[j] : -1;
      to[j] = pg;
      if (j < have) {
        if (pg >= 0 && pg < p.num_pages)
          atomicAdd(&p.ref_out[pg], 1);
        else
          set_status(p.status, DSA_DEV_BAD_INDEX);
      }
    }
    if (threadIdx.x == 0) p.len_out[dst] = len;
  }
}

// One CTA: the map of the pages, their new reference counts and the list of moves.
// With L pages in use, the page in use at p >= L that has r pages in use between L and
// itself goes to the free page q < L that has r free pages below it.  A warp takes a
// stretch of words of 32 pages; the words' masks are kept, so the counts are read once.
// ref_out may be ref_in: the counts that move are read before they are written.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesParams p) {
  __shared__ int sums[32];
  __shared__ uint32_t s_masks[kMaskWords];
  __shared__ int s_before;                         // pages in use below page L
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (p.num_pages + 31) / 32;
  uint32_t* masks = words <= kMaskWords ? s_masks : reinterpret_cast<uint32_t*>(p.sharers);
  const int per = (words + 31) / 32;               // words per warp
  const int w0 = min(warp * per, words), w1 = min(w0 + per, words);
  next_kernel();
  if (tid == 0) *p.status = 0;
  int count = 0;
  for (int w = w0; w < w1; w += 4) {
    int r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int pg = (w + u) * 32 + lane;
      r[u] = w + u < w1 && pg < p.num_pages ? p.ref_in[pg] : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (w + u >= w1) break;
      const int pg = (w + u) * 32 + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, r[u] > 0);
      count += __popc(m);
      if (lane == 0) masks[w + u] = m;
      if (pg < p.num_pages) {
        p.map[pg] = r[u] > 0 ? pg : -1;
        if (p.ref_out != p.ref_in) p.ref_out[pg] = r[u];
      }
    }
  }
  int total;
  int before = block_scan(lane == 0 ? count : 0, sums, total);   // of lane 0: pages in use before the warp's
  before = __shfl_sync(0xffffffffu, before, 0);
  const int live = total;
  if (live < p.num_pages && live / 32 >= w0 && live / 32 < w1 && lane == 0) {
    int b = before;
    for (int w = w0; w < live / 32; ++w) b += __popc(masks[w]);
    s_before = b + __popc(masks[live / 32] & ((1u << (live & 31)) - 1));
  }
  if (live == p.num_pages && tid == 0) s_before = live;
  __syncthreads();
  const int base = s_before, moves = live - base;
  for (int w = w0; w < w1; ++w) {
    const uint32_t m = masks[w];
    const int pg = w * 32 + lane;
    const bool used = m >> lane & 1;
    const int at = before + __popc(m & ((1u << lane) - 1));
    if (used && pg >= live) p.move_src[at - base] = pg;
    if (!used && pg < live) p.move_dst[pg - at] = pg;
    before += __popc(m);
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kPlanThreads) {
    const int from = p.move_src[i], to = p.move_dst[i];
    p.map[from] = to;
    const int r = p.ref_in[from];
    p.ref_out[to] = r;
    p.ref_out[from] = 0;
  }
  if (tid == 0) *p.num_moves = moves;
}

// The table's changes of a compaction: entries in use follow the map; the rest is copied.
__device__ __forceinline__ void remap_table(const PagesParams& p) {
  const int64_t nt = static_cast<int64_t>(p.num_seqs) * p.pages_per_seq;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < nt; i += step) {
    const int64_t s = i / p.pages_per_seq;
    const int j = static_cast<int>(i - s * p.pages_per_seq);
    int pg = p.table_in[i];
    if (j < pages_of(p.len_in[s], p.page_size)) {
      if (pg >= 0 && pg < p.num_pages)
        pg = p.map[pg];
      else
        set_status(p.status, DSA_DEV_BAD_INDEX);
    }
    p.table_out[i] = pg;
  }
  if (p.len_out != p.len_in)
    for (int64_t i = i0; i < p.num_seqs; i += step) p.len_out[i] = p.len_in[i];
}

// Copies the listed pages in all buffers: large pages chunk by chunk, small ones a
// run of words over several pages.  Before that the changes of the table, of a resize or
// a compaction.
template <bool kResize>
__global__ void __launch_bounds__(kMoveThreads) move_pages_kernel(PagesParams p) {
  last_kernel();
  if (kResize)
    patch_table(p);
  else
    remap_table(p);
  const int64_t moves = __ldcg(p.num_moves);
  const int64_t items = moves * p.chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t m = it / p.chunks;
    int c = static_cast<int>(it - m * p.chunks);
    int b = 0;
    while (c >= p.buf_chunks[b]) c -= p.buf_chunks[b++];
    const int64_t pb = p.buf_bytes[b];
    const int64_t o = static_cast<int64_t>(c) * kMoveChunk;
    const int n = static_cast<int>(pb - o < kMoveChunk ? pb - o : kMoveChunk);
    const uint8_t* src = p.buf[b] + __ldcg(&p.move_src[m]) * pb + o;
    uint8_t* dst = p.buf[b] + __ldcg(&p.move_dst[m]) * pb + o;
    if (p.buf_vec[b]) {
      constexpr int kPer = kMoveChunk / 16 / kMoveThreads;
      uint4 v[kPer];
      const int nv = n / 16;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * kMoveThreads + static_cast<int>(threadIdx.x) < nv)
          v[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i * kMoveThreads + threadIdx.x);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * kMoveThreads + static_cast<int>(threadIdx.x) < nv)
          __stcs(reinterpret_cast<uint4*>(dst) + i * kMoveThreads + threadIdx.x, v[i]);
    } else {
      for (int i = threadIdx.x; i < n / 4; i += kMoveThreads)
        reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i];
    }
  }
  for (int b = 0; b < p.num_bufs; ++b) {
    if (p.buf_chunks[b]) continue;
    const int64_t pw = p.buf_bytes[b] / 4;
    uint32_t* base = reinterpret_cast<uint32_t*>(p.buf[b]);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kMoveThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < moves * pw; i += step) {
      const int64_t m = i / pw, w = i - m * pw;
      base[__ldcg(&p.move_dst[m]) * pw + w] = base[__ldcg(&p.move_src[m]) * pw + w];
    }
  }
}

// SMs of the current device, asked for once per device (a query costs a third of a launch).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool state_ok(const dsa_page_state* s) {
  return s && s->num_seqs >= 1 && s->num_pages >= 1 && s->page_size >= 1 && s->pages_per_seq >= 1;
}
// Sums of pages over all sequences, each with a copied page more, stay in 32 bits.
bool state_supported(const dsa_page_state* s) {
  constexpr int64_t most = int64_t{1} << 31;
  return s->page_size % 64 == 0 && static_cast<int64_t>(s->pages_per_seq) * s->page_size < most &&
         (static_cast<int64_t>(s->pages_per_seq) + 1) * s->num_seqs < most;
}

// Workspace: the status word, then the int32 arrays below.
PagesParams pages_params(const dsa_page_state* in, const dsa_page_state* out, int n, void* ws, size_t* bytes) {
  PagesParams p{};
  p.num_seqs = in->num_seqs;
  p.num_pages = in->num_pages;
  p.page_size = in->page_size;
  p.pages_per_seq = in->pages_per_seq;
  p.table_in = in->page_table;
  p.len_in = in->seq_len;
  p.ref_in = in->ref_count;
  p.table_out = out->page_table;
  p.len_out = out->seq_len;
  p.ref_out = out->ref_count;
  p.n = n;
  p.status = static_cast<uint32_t*>(ws);
  size_t off = kWsHeader;
  auto take = [&](size_t count) {
    int32_t* x = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + off);
    off += (count * sizeof(int32_t) + 255) / 256 * 256;
    return x;
  };
  const size_t pages = static_cast<size_t>(in->num_pages);
  p.num_moves = take(3);
  p.first = take(in->num_seqs);
  p.sharers = take(pages);
  p.last_sharer = take(pages);
  p.free_list = take(pages);
  p.map = take(pages);
  p.move_src = take(pages);
  p.move_dst = take(pages);
  p.old_len = take(n);
  p.last_page = take(n);
  p.drop_at = take(n);
  p.drop_pos = take(n);
  p.take_at = take(n);
  p.take_pos = take(n);
  *bytes = off;
  return p;
}

dsa_status check(const dsa_page_state* in, const dsa_page_state* out, int n, const void* a, const void* b, void* ws,
                 size_t ws_bytes, PagesParams& p) {
  if (!state_ok(in) || !state_ok(out) || n < 0 || !ws) return DSA_ERR_INVALID_ARGUMENT;
  if (!in->page_table || !in->seq_len || !in->ref_count || !out->page_table || !out->seq_len || !out->ref_count)
    return DSA_ERR_INVALID_ARGUMENT;
  if (n > 0 && (!a || !b)) return DSA_ERR_INVALID_ARGUMENT;
  if (in->num_seqs != out->num_seqs || in->num_pages != out->num_pages || in->page_size != out->page_size ||
      in->pages_per_seq != out->pages_per_seq)
    return DSA_ERR_INVALID_ARGUMENT;
  // in place, or apart
  const bool t = in->page_table == out->page_table, l = in->seq_len == out->seq_len,
             r = in->ref_count == out->ref_count;
  if (t != l || t != r) return DSA_ERR_INVALID_ARGUMENT;
  if (!state_supported(in)) return DSA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(ws) & 15u) return DSA_ERR_UNSUPPORTED;
  size_t bytes = 0;
  p = pages_params(in, out, n, ws, &bytes);
  return ws_bytes < bytes ? DSA_ERR_WORKSPACE_TOO_SMALL : DSA_OK;
}

dsa_status take_buffers(const dsa_page_buffers* bufs, PagesParams& p) {
  p.num_bufs = 0;
  p.chunks = 0;
  if (!bufs) return DSA_OK;
  if (bufs->num < 0 || bufs->num > DSA_MAX_PAGE_BUFFERS) return DSA_ERR_INVALID_ARGUMENT;
  for (int j = 0; j < bufs->num; ++j) {
    const int64_t pb = bufs->page_bytes[j];
    if (!bufs->base[j] || pb <= 0) return DSA_ERR_INVALID_ARGUMENT;
    const uintptr_t a = reinterpret_cast<uintptr_t>(bufs->base[j]);
    if (pb % 4 || a % 4 || pb > (int64_t{1} << 31)) return DSA_ERR_UNSUPPORTED;
    p.buf[j] = static_cast<uint8_t*>(bufs->base[j]);
    p.buf_bytes[j] = pb;
    p.buf_vec[j] = pb % 16 == 0 && a % 16 == 0;
    p.buf_chunks[j] = pb <= kSmallPage ? 0 : static_cast<int>((pb + kMoveChunk - 1) / kMoveChunk);
    p.chunks += p.buf_chunks[j];
  }
  p.num_bufs = bufs->num;
  return DSA_OK;
}

// Launches a kernel of a call; all but the first with programmatic dependent launch.
template <typename... Args>
cudaError_t launch_smem(void (*kernel)(Args...), int grid, int threads, size_t smem, cudaStream_t st, bool first,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = first ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), int grid, int threads, cudaStream_t st, bool first, Args... args) {
  return launch_smem(kernel, grid, threads, 0, st, first, args...);
}

// The shared memory of a resize that works on the counts there, once per device.
cudaError_t prepare_own() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(resize_plan_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(int32_t)) * kOwnPages);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

int grid_for(int64_t items) {
  const int64_t want = (items + 1023) / 1024, most = 8 * static_cast<int64_t>(sm_count());
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_copy_state(const PagesParams& p, cudaStream_t st) {
  return launch(copy_state_kernel, grid_for(static_cast<int64_t>(p.num_seqs) * p.pages_per_seq + p.num_pages), 256, st,
                true, p);
}

// The table's changes and copies of at most `most` pages.
template <bool kResize>
cudaError_t launch_moves(const PagesParams& p, int64_t most, cudaStream_t st) {
  const int64_t entries = kResize ? 0 : static_cast<int64_t>(p.num_seqs) * p.pages_per_seq / kMoveThreads + 1;
  const int64_t copies = p.num_bufs > 0 ? most * (p.chunks > 0 ? p.chunks : 1) : kResize ? most : 0;
  const int64_t items = copies > entries ? copies : entries, full = 16 * static_cast<int64_t>(sm_count());
  return launch(move_pages_kernel<kResize>, static_cast<int>(items < full ? items : full), kMoveThreads, st, false, p);
}

dsa_status status_of(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_pages_workspace_size(const dsa_page_state* state, int n) {
  if (!state_ok(state) || !state_supported(state) || n < 0) return 0;
  size_t bytes = 0;
  (void)pages_params(state, state, n, nullptr, &bytes);
  return bytes;
}

dsa_status dsa_pages_resize(const dsa_page_state* in, const dsa_page_state* out, int n, const int32_t* seqs,
                            const int32_t* new_len, const dsa_page_buffers* buffers, void* ws, size_t ws_bytes,
                            void* stream) {
  PagesParams p;
  dsa_status s = check(in, out, n, seqs, new_len, ws, ws_bytes, p);
  if (s == DSA_OK) s = take_buffers(buffers, p);
  if (s != DSA_OK) return s;
  p.list_a = seqs;
  p.list_b = new_len;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool apart = p.table_in != p.table_out;
  const bool own = p.num_pages <= kOwnPages;
  if (!own) {
    cudaError_t e = apart ? launch_copy_state(p, st) : cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st);
    if (e == cudaSuccess) e = launch(resize_plan_kernel<false>, 1, kPlanThreads, st, !apart, p);
    if (e == cudaSuccess && n > 0) e = launch_moves<true>(p, n, st);
    return status_of(e);
  }
  // the table goes by 8192 entries per CTA, one CTA per SM (they have the plan's shared memory too)
  const int64_t parts = (static_cast<int64_t>(p.num_seqs) * p.pages_per_seq + 8191) / 8192, most = sm_count() - 1;
  const int copiers = apart ? static_cast<int>(parts < most ? parts : most) : 0;
  cudaError_t e = prepare_own();
  if (e == cudaSuccess)
    e = launch_smem(resize_plan_kernel<true>, 1 + copiers, kPlanThreads, sizeof(int32_t) * p.num_pages, st, true, p);
  if (e == cudaSuccess && n > 0) e = launch_moves<true>(p, n, st);
  return status_of(e);
}

dsa_status dsa_pages_fork(const dsa_page_state* in, const dsa_page_state* out, int n, const int32_t* src_seqs,
                          const int32_t* dst_seqs, void* ws, size_t ws_bytes, void* stream) {
  PagesParams p;
  const dsa_status s = check(in, out, n, src_seqs, dst_seqs, ws, ws_bytes, p);
  if (s != DSA_OK) return s;
  p.list_a = src_seqs;
  p.list_b = dst_seqs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool apart = p.table_in != p.table_out;
  cudaError_t e = apart ? launch_copy_state(p, st) : cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st);
  if (e == cudaSuccess && n > 0) e = launch(fork_kernel, n < 4096 ? n : 4096, 256, st, !apart, p);
  return status_of(e);
}

dsa_status dsa_pages_compact(const dsa_page_state* in, const dsa_page_state* out, const dsa_page_buffers* buffers,
                             int32_t* page_map, void* ws, size_t ws_bytes, void* stream) {
  PagesParams p;
  dsa_status s = check(in, out, 0, nullptr, nullptr, ws, ws_bytes, p);
  if (s == DSA_OK) s = take_buffers(buffers, p);
  if (s != DSA_OK) return s;
  if (page_map) p.map = page_map;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch(compact_plan_kernel, 1, kPlanThreads, st, true, p);
  if (e == cudaSuccess) e = launch_moves<false>(p, p.num_pages, st);
  return status_of(e);
}

}  // extern "C"
