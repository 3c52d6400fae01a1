// Quantising append to the 8-bit latent cache on sm_100a.
//
// For each block of g = scale_block positions that receives tokens: need = the
// smallest power of two with 448 need >= the largest |entry| of its new rows,
// scale = need, or max(scale, need) where the block already held rows (which are
// re-encoded when the scale grows), codes = E4M3(kv / scale).  Powers of two make
// the division exact, so a stored value is rounded once, and re-encoding an
// earlier row only shifts its exponent (what falls below E4M3's smallest step is
// rounded again).
//
// Bound by memory: 1152 B read and 576 B written per row, once each.  One CTA
// (256 threads) takes a run of up to 64 new rows of one 64-position stretch (a
// page holds whole stretches, and a stretch whole blocks), holds all of it in
// registers between the maximum and the encoding (18 16-byte loads per thread, all
// in flight), so the rows are read once.  A CTA finds the runs that begin in its
// window of the token list by comparing neighbours.
#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kStretch = 64;                       // positions per run: divides every page, a multiple of every block
constexpr int kRowChunks = DSA_D_QK / 8;           // 16-byte chunks (8 bf16) of a row
constexpr int kWarpRows = kStretch / (kQuantThreads / 32);
constexpr int kPer = kWarpRows * kRowChunks / 32;  // chunks per thread
constexpr int kMinExp = -100, kMaxExp = 100;       // exponents of a scale

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Smallest e in [kMinExp, kMaxExp] with 448 * 2^e >= the bf16 magnitude `bits`
// (448 = 1.75 * 2^8).
__device__ __forceinline__ int need_exp(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return bits < 0x80u || e < kMinExp ? kMinExp : (e > kMaxExp ? kMaxExp : e);
}

__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint32_t v) {
  const uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  if (lo < 0x7f80u && lo > m) m = lo;
  if (hi < 0x7f80u && hi > m) m = hi;
  return m;
}

// Two bf16 (one word) times inv (a power of two: exact) -> two E4M3 codes.
__device__ __forceinline__ uint32_t encode2(uint32_t v, float inv) {
  const float2 f = make_float2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
  return static_cast<uint16_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ uint32_t reencode4(uint32_t v, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw x =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> (16 * h)), __NV_E4M3);
    const float2 y = __half22float2(__half2(x));
    r |= static_cast<uint32_t>(
             __nv_cvt_float2_to_fp8x2(make_float2(y.x * f, y.y * f), __NV_SATFINITE, __NV_E4M3))
         << (16 * h);
  }
  return r;
}

__global__ void __launch_bounds__(kQuantThreads) quantize_append_kernel(QuantParams p) {
  __shared__ uint32_t smax[kStretch];              // largest magnitude (bf16 bits) per scale block of the stretch
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = p.block;
  const int w0 = blockIdx.x * p.window;
  // runs that begin in the window (every warp finds the same mask)
  uint32_t starts;
  {
    const int t = w0 + lane;
    bool lead = false;
    if (lane < p.window && t < p.T) {
      const int s = p.q_seq[t], x = p.q_pos[t];
      lead = t == 0 || x % kStretch == 0 || p.q_seq[t - 1] != s || p.q_pos[t - 1] != x - 1;
    }
    starts = __ballot_sync(0xffffffffu, lead);
  }
  for (; starts; starts &= starts - 1) {
    const int t0 = w0 + __ffs(starts) - 1;
    const int seq = p.q_seq[t0], pos = p.q_pos[t0];
    const int first = pos & (kStretch - 1);        // row of the stretch that the run begins with
    bool ok = seq >= 0 && seq < p.num_seqs && pos >= 0 && pos < p.kv_len[seq];
    if (ok && t0 > 0) {
      const int ps = p.q_seq[t0 - 1];
      ok = seq > ps || (seq == ps && p.q_pos[t0 - 1] == pos - 1);
    }
    // rows of the run: consecutive tokens of the sequence within the stretch
    int n = 1;
    if (ok) {
      uint32_t same[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int l = lane + 32 * h, t = t0 + l;
        same[h] = __ballot_sync(0xffffffffu, t < p.T && l < kStretch - first && p.q_seq[t] == seq &&
                                                 p.q_pos[t] == pos + l);
      }
      n = same[0] == 0xffffffffu ? 32 + __ffs(~same[1]) - 1 : __ffs(~same[0]) - 1;
      if (same[0] == 0xffffffffu && same[1] == 0xffffffffu) n = 64;
    }
    uint32_t flag = ok ? 0u : DSA_DEV_BAD_QUERY;
    if (ok && n > p.kv_len[seq] - pos) {
      n = p.kv_len[seq] - pos;
      flag = DSA_DEV_BAD_QUERY;
    }
    int64_t row = 0;                               // cache row of the run's first token
    if (ok) {
      if (p.page_size == 0) {
        const int64_t off = p.kv_offset[seq];
        row = off + pos;
        if (off < 0 || off % g != 0) {
          ok = false;
          flag |= DSA_DEV_BAD_QUERY;
        } else if (row + n > p.kv_rows) {
          n = row < p.kv_rows ? static_cast<int>(p.kv_rows - row) : 0;
          flag |= DSA_DEV_BAD_INDEX;
        }
      } else {
        const int pg = pos / p.page_size < p.pages_per_seq
                           ? p.page_table[static_cast<int64_t>(seq) * p.pages_per_seq + pos / p.page_size]
                           : -1;
        row = static_cast<int64_t>(pg) * p.page_size + pos % p.page_size;
        if (pg < 0 || row >= p.kv_rows) {
          ok = false;
          flag |= DSA_DEV_BAD_INDEX;
        }
      }
    }
    if (flag && tid == 0) set_status(p.status, flag);
    if (!ok || n <= 0) continue;                   // uniform over the CTA

    // the run's rows: warp w holds rows 8w .. 8w + 7 of the stretch
    const uint4* src = reinterpret_cast<const uint4*>(p.kv + static_cast<int64_t>(t0) * DSA_D_QK);
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * 32 + lane, r = warp * kWarpRows + c / kRowChunks - first;
      v[i] = r >= 0 && r < n ? __ldg(src + static_cast<int64_t>(r) * kRowChunks + c % kRowChunks)
                             : make_uint4(0u, 0u, 0u, 0u);
    }
    if (tid < kStretch) smax[tid] = 0;
    // the scale of the block that the run begins within, if it held rows before
    const int b0 = first / g;
    const int64_t blk = (row - first % g) / g;     // physical block of the run's first row
    const bool held = first % g != 0;
    const float s_old = held ? p.scale[blk] : 0.f;
    const bool s_ok = s_old >= pow2f(kMinExp) && s_old <= pow2f(kMaxExp);
    if (held && !s_ok && tid == 0) set_status(p.status, DSA_DEV_BAD_SCALE);
    __syncthreads();
    if (g >= kWarpRows) {                          // a warp's rows lie in one block
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        m = max_finite(max_finite(max_finite(max_finite(m, v[i].x), v[i].y), v[i].z), v[i].w);
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0 && m) atomicMax(&smax[warp * kWarpRows / g], m);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t m = max_finite(max_finite(max_finite(max_finite(0, v[i].x), v[i].y), v[i].z), v[i].w);
        if (m) atomicMax(&smax[(warp * kWarpRows + (i * 32 + lane) / kRowChunks) / g], m);
      }
    }
    __syncthreads();
    // scale of a block of the stretch
    auto block_scale = [&](int b) {
      const float need = pow2f(need_exp(smax[b]));
      return b == b0 && s_ok ? fmaxf(need, s_old) : need;
    };
    // earlier rows of the first block, when its scale grows
    const float s0 = block_scale(b0);
    if (held && s_ok && s0 > s_old) {
      const float f = s_old / s0;
      uint4* dst = reinterpret_cast<uint4*>(p.kv8 + blk * g * DSA_D_QK);
      for (int i = tid; i < (first % g) * (DSA_D_QK / 16); i += kQuantThreads) {
        uint4 c = dst[i];
        c.x = reencode4(c.x, f);
        c.y = reencode4(c.y, f);
        c.z = reencode4(c.z, f);
        c.w = reencode4(c.w, f);
        dst[i] = c;
      }
    }
    // codes of the new rows
    uint8_t* out = p.kv8 + row * DSA_D_QK;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = i * 32 + lane, rs = warp * kWarpRows + c / kRowChunks, r = rs - first;
      if (r < 0 || r >= n) continue;
      const float inv = 1.f / block_scale(rs / g);
      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(r) * DSA_D_QK + (c % kRowChunks) * 8) =
          make_uint2(encode2(v[i].x, inv) | (encode2(v[i].y, inv) << 16),
                     encode2(v[i].z, inv) | (encode2(v[i].w, inv) << 16));
    }
    const int last = (first + n - 1) / g;
    if (tid >= b0 && tid <= last) p.scale[blk + tid - b0] = block_scale(tid);
    __syncthreads();                               // smax is reset by the next run
  }
}

}  // namespace

cudaError_t launch_quantize_append(const QuantParams& params, cudaStream_t stream) {
  if (params.T == 0) return cudaSuccess;
  QuantParams p = params;
  // A long list is mostly prompts (a run per 64 tokens), so a CTA looks at 16
  // tokens; in a short one every token may be a run of its own.
  p.window = p.T > 4096 ? 16 : 1;
  quantize_append_kernel<<<(p.T + p.window - 1) / p.window, kQuantThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dsa
