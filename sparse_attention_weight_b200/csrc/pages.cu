// Pages of a paged cache on sm_100a: growing, cutting and freeing sequences with
// copy on write, forks, compaction.  Integer bookkeeping plus copies of whole
// pages; the results are those of the sequential definition in the header
// whatever order the threads run in (lists are ranked by prefix sums; atomics
// only add, or take a maximum of list positions).
//
// Bound by latency for the bookkeeping (a few dependent passes over lists of some
// hundred entries and the reference counts) and by memory for the copies (each
// byte read and written once).
#include <climits>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 16384;                  // bytes of a page that a CTA copies at a time

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
  return static_cast<int>((static_cast<int64_t>(len) + page_size - 1) / page_size);
}

// out = in, for the three arrays of a state.
__global__ void __launch_bounds__(256) copy_state_kernel(PagesParams p) {
  const int64_t nt = static_cast<int64_t>(p.num_seqs) * p.pages_per_seq;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < nt; i += step) p.table_out[i] = p.table_in[i];
  for (int64_t i = i0; i < p.num_seqs; i += step) p.len_out[i] = p.len_in[i];
  for (int64_t i = i0; i < p.num_pages; i += step) p.ref_out[i] = p.ref_in[i];
}

// One CTA works out a resize on the state `out` (which holds the input's values)
// and lists the page copies.
__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(PagesParams p) {
  __shared__ int sums[32];
  __shared__ int s_moves;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = p.page_size, n = p.n;
  if (tid == 0) s_moves = 0;
  uint32_t flags = 0;
  // entry i is valid if it is the first that names its sequence
  auto in_range = [&](int s, int len) {
    return s >= 0 && s < p.num_seqs && len >= 0 &&
           len <= static_cast<int64_t>(p.pages_per_seq) * P && p.len_out[s] >= 0 &&
           p.len_out[s] <= static_cast<int64_t>(p.pages_per_seq) * P;
  };
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = p.list_a[i];
    if (s >= 0 && s < p.num_seqs) p.first[s] = INT_MAX;
    p.old_len[i] = s >= 0 && s < p.num_seqs ? p.len_out[s] : 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = p.list_a[i];
    if (s >= 0 && s < p.num_seqs) atomicMin(&p.first[s], i);
  }
  __syncthreads();
  auto valid = [&](int i) {
    const int s = p.list_a[i];
    return in_range(s, p.list_b[i]) && p.first[s] == i;
  };
  for (int i = tid; i < n; i += kPlanThreads) {
    const bool ok = valid(i);
    p.entry_ok[i] = ok;
    if (!ok) flags |= DSA_DEV_BAD_QUERY;
  }
  __syncthreads();
  // shrinking entries drop their pages
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    if (!p.entry_ok[i]) continue;
    const int s = p.list_a[i], want = pages_of(p.list_b[i], P), have = pages_of(p.old_len[i], P);
    int32_t* row = p.table_out + static_cast<int64_t>(s) * p.pages_per_seq;
    for (int j = want + lane; j < have; j += 32) {
      const int pg = row[j];
      if (pg >= 0 && pg < p.num_pages) {
        atomicSub(&p.ref_out[pg], 1);
        row[j] = -1;
      } else {
        flags |= DSA_DEV_BAD_INDEX;
      }
    }
    if (lane == 0 && p.list_b[i] <= p.old_len[i]) p.len_out[s] = p.list_b[i];
  }
  __syncthreads();
  // growing entries with a partly filled last page: how many share it, and the last of them
  auto last_page = [&](int i) {
    if (!p.entry_ok[i] || p.list_b[i] <= p.old_len[i] || p.old_len[i] % P == 0) return -1;
    const int pg = p.table_out[static_cast<int64_t>(p.list_a[i]) * p.pages_per_seq + p.old_len[i] / P];
    return pg >= 0 && pg < p.num_pages ? pg : -2;
  };
  for (int i = tid; i < n; i += kPlanThreads) {
    const int pg = last_page(i);
    if (pg == -2) flags |= DSA_DEV_BAD_INDEX;
    if (pg >= 0) {
      p.sharers[pg] = 0;
      p.last_sharer[pg] = -1;
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int pg = last_page(i);
    if (pg >= 0) {
      atomicAdd(&p.sharers[pg], 1);
      atomicMax(&p.last_sharer[pg], i);
    }
  }
  __syncthreads();
  // pages that each entry takes, and where its share of the free list begins
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int take = 0, copy = 0;
    if (i < n && p.entry_ok[i] && p.list_b[i] > p.old_len[i]) {
      const int pg = last_page(i);
      if (pg >= 0) {
        const int r = p.ref_out[pg];
        copy = r > 1 && !(r <= p.sharers[pg] && p.last_sharer[pg] == i);
      }
      take = copy + pages_of(p.list_b[i], P) - pages_of(p.old_len[i], P);
    }
    int total;
    const int at = block_scan(take, sums, total);
    if (i < n) {
      p.start[i] = need + at;
      p.copies[i] = copy;
    }
    need = need > INT_MAX - total ? INT_MAX : need + total;
  }
  // the lowest free pages
  int found = 0;
  for (int64_t c0 = 0; c0 < p.num_pages && found < need; c0 += kPlanThreads) {
    const int64_t pg = c0 + tid;
    const int is_free = pg < p.num_pages && p.ref_out[pg] == 0;
    int total;
    const int at = block_scan(is_free, sums, total);
    if (is_free && found + at < need) p.free_list[found + at] = static_cast<int>(pg);
    found += total;
  }
  __syncthreads();
  if (found < need) {
    if (tid == 0) set_status(p.status, DSA_DEV_NO_PAGES);
  } else {
    for (int i = warp; i < n; i += kPlanThreads / 32) {
      if (!p.entry_ok[i] || p.list_b[i] <= p.old_len[i]) continue;
      const int s = p.list_a[i], want = pages_of(p.list_b[i], P), have = pages_of(p.old_len[i], P);
      int32_t* row = p.table_out + static_cast<int64_t>(s) * p.pages_per_seq;
      const int copy = p.copies[i];
      const int* got = p.free_list + p.start[i];
      if (copy && lane == 0) {
        const int from = row[have - 1], to = got[0];
        const int m = atomicAdd(&s_moves, 1);
        p.move_src[m] = from;
        p.move_dst[m] = to;
        row[have - 1] = to;
        p.ref_out[to] = 1;
        atomicSub(&p.ref_out[from], 1);
      }
      for (int j = have + lane; j < want; j += 32) {
        const int pg = got[copy + j - have];
        row[j] = pg;
        p.ref_out[pg] = 1;
      }
      if (lane == 0) p.len_out[s] = p.list_b[i];
    }
  }
  if (flags) set_status(p.status, flags);
  __syncthreads();
  if (tid == 0) *p.num_moves = s_moves;
}

// A CTA per pair: the pair is checked against the whole list.
__global__ void __launch_bounds__(256) fork_kernel(PagesParams p) {
  const int P = p.page_size;
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
// ref_out may be ref_in, so the counts that move are read before they are written.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesParams p) {
  __shared__ int sums[32];
  const int tid = threadIdx.x;
  int live_count = 0;
  for (int64_t c0 = 0; c0 < p.num_pages; c0 += kPlanThreads) {
    const int64_t pg = c0 + tid;
    live_count += __syncthreads_count(pg < p.num_pages && p.ref_in[pg] > 0);
  }
  // k-th page in use at or above live_count -> k-th free page below it
  int up = 0, down = 0;
  for (int64_t c0 = 0; c0 < p.num_pages; c0 += kPlanThreads) {
    const int64_t pg = c0 + tid;
    const bool in = pg < p.num_pages;
    const bool live = in && p.ref_in[pg] > 0;
    const int is_up = live && pg >= live_count, is_down = in && !live && pg < live_count;
    int total;
    int at = block_scan(is_up, sums, total);
    if (is_up) p.move_src[up + at] = static_cast<int>(pg);
    up += total;
    at = block_scan(is_down, sums, total);
    if (is_down) p.move_dst[down + at] = static_cast<int>(pg);
    down += total;
    if (in) {
      p.map[pg] = live ? static_cast<int>(pg) : -1;
      if (p.ref_out != p.ref_in) p.ref_out[pg] = p.ref_in[pg];
    }
  }
  __syncthreads();
  for (int i = tid; i < up; i += kPlanThreads) {
    const int from = p.move_src[i], to = p.move_dst[i];
    p.map[from] = to;
    const int r = p.ref_in[from];
    p.ref_out[to] = r;
    p.ref_out[from] = 0;
  }
  if (tid == 0) *p.num_moves = up;
}

__global__ void __launch_bounds__(256) remap_kernel(PagesParams p) {
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

// Copies the listed pages in all buffers, chunk by chunk.
__global__ void __launch_bounds__(kMoveThreads) move_pages_kernel(PagesParams p) {
  const int moves = *p.num_moves;
  const int64_t items = static_cast<int64_t>(moves) * p.chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int m = static_cast<int>(it / p.chunks);
    int c = static_cast<int>(it - static_cast<int64_t>(m) * p.chunks);
    int b = 0;
    while (c >= p.buf_chunks[b]) c -= p.buf_chunks[b++];
    const int64_t pb = p.buf_bytes[b];
    const int64_t o = static_cast<int64_t>(c) * kMoveChunk;
    const int64_t n = pb - o < kMoveChunk ? pb - o : kMoveChunk;
    const uint8_t* src = p.buf[b] + p.move_src[m] * pb + o;
    uint8_t* dst = p.buf[b] + p.move_dst[m] * pb + o;
    if (p.buf_vec[b]) {
      constexpr int kPer = kMoveChunk / 16 / kMoveThreads;
      uint4 v[kPer];
      const int nv = static_cast<int>(n / 16);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * kMoveThreads + static_cast<int>(threadIdx.x) < nv)
          v[i] = reinterpret_cast<const uint4*>(src)[i * kMoveThreads + threadIdx.x];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i * kMoveThreads + static_cast<int>(threadIdx.x) < nv)
          reinterpret_cast<uint4*>(dst)[i * kMoveThreads + threadIdx.x] = v[i];
    } else {
      for (int i = threadIdx.x; i < n / 4; i += kMoveThreads)
        reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i];
    }
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

bool state_ok(const dsa_page_state* s) {
  return s && s->num_seqs >= 1 && s->num_pages >= 1 && s->page_size >= 1 && s->pages_per_seq >= 1;
}
bool state_supported(const dsa_page_state* s) {
  return s->page_size % 64 == 0 && static_cast<int64_t>(s->pages_per_seq) * s->page_size < (int64_t{1} << 31);
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
  p.num_moves = take(1);
  p.first = take(in->num_seqs);
  p.sharers = take(pages);
  p.last_sharer = take(pages);
  p.free_list = take(pages);
  p.map = take(pages);
  p.move_src = take(pages);
  p.move_dst = take(pages);
  p.old_len = take(n);
  p.entry_ok = take(n);
  p.start = take(n);
  p.copies = take(n);
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
    p.buf_chunks[j] = static_cast<int>((pb + kMoveChunk - 1) / kMoveChunk);
    p.chunks += p.buf_chunks[j];
  }
  p.num_bufs = bufs->num;
  return DSA_OK;
}

cudaError_t launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

cudaError_t launch_copy_state(const PagesParams& p, cudaStream_t st) {
  if (p.table_in == p.table_out) return cudaSuccess;
  const int64_t items = static_cast<int64_t>(p.num_seqs) * p.pages_per_seq + p.num_pages;
  const int64_t want = (items + 1023) / 1024, most = 8 * sm_count();
  copy_state_kernel<<<static_cast<int>(want < most ? want : most), 256, 0, st>>>(p);
  return launched();
}

cudaError_t launch_moves(const PagesParams& p, cudaStream_t st) {
  if (p.num_bufs == 0) return cudaSuccess;
  move_pages_kernel<<<8 * sm_count(), kMoveThreads, 0, st>>>(p);
  return launched();
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
  if (cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st) != cudaSuccess) return DSA_ERR_CUDA;
  cudaError_t e = launch_copy_state(p, st);
  if (e == cudaSuccess && n > 0) {
    resize_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
    e = launched();
    if (e == cudaSuccess) e = launch_moves(p, st);
  }
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
  if (cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st) != cudaSuccess) return DSA_ERR_CUDA;
  cudaError_t e = launch_copy_state(p, st);
  if (e == cudaSuccess && n > 0) {
    fork_kernel<<<n < 4096 ? n : 4096, 256, 0, st>>>(p);
    e = launched();
  }
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
  if (cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st) != cudaSuccess) return DSA_ERR_CUDA;
  compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  cudaError_t e = launched();
  if (e == cudaSuccess) {
    const int64_t items = static_cast<int64_t>(p.num_seqs) * p.pages_per_seq;
    const int64_t want = (items + 1023) / 1024, most = 8 * sm_count();
    remap_kernel<<<static_cast<int>(want < most ? want : most), 256, 0, st>>>(p);
    e = launched();
  }
  if (e == cudaSuccess) e = launch_moves(p, st);
  return status_of(e);
}

}  // extern "C"
