// Quantising append to the 8-bit latent cache on sm_100a.
//
// For each block of g = scale_block positions that receives tokens: need = the
// smallest power of two with 448 need >= the largest |entry| of its new rows,
// scale = need, or max(scale, need) where the block already held rows (which are
// re-encoded when the scale grows), codes = E4M3(kv / scale).  Powers of two make
// the division exact, so a stored value is rounded once, and re-encoding an
// earlier row only shifts its exponent (what falls below E4M3's smallest step is
// rounded again).  A block that was quantised elsewhere may hold any scale; its new rows
// then take a division, rounded once all the same.
//
// Bound by memory: 1152 B read and 576 B written per row, once each.  The work is
// cut into runs: the new rows of one 64-position stretch of one sequence (a page
// holds whole stretches, and a stretch whole blocks), up to 72 KB that lie together
// in the input.  A CTA (256 threads) brings a run into shared memory with one bulk
// copy, takes the maximum of each block and encodes from there, so the rows are read
// once; three CTAs per SM keep some 200 KB in flight.  Long token lists (prompts) are
// first searched for the places where runs begin; in short ones (decode steps, where
// nearly every token is a run) each token has its own CTA.
// Measured on the device: 61,000 prompt tokens in blocks of 64, 32 us with both kernels (106 MB, 3.3
// TB/s, half of a copy's rate): the 950 runs go round the 444 CTAs 2.2 times, so that the
// last round is nearly empty, and a CTA's copy, maxima and codes follow one another.  A
// decode step of 128 tokens, 6.5 us, is launch and latency.  With and
// without the search: 128 tokens in twos 8.2 and 6.2 us, 1024 in twos 10.3 and 8.2, 2000 of
// a prompt 10.3 and 10.5, 4000 10.3 and 14.3.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kWarps = kQuantThreads / 32;
constexpr int kStretch = 64;                       // positions per run: divides every page, a multiple of every block
constexpr int kRowBytes = DSA_D_QK * 2;
constexpr int kPieces = DSA_D_QK / 16;             // pieces of 16 entries of a row
constexpr int kMinExp = -100, kMaxExp = 100;       // exponents of a scale
constexpr int kShortList = 1024;                   // tokens up to which each has a CTA of its own
constexpr int kCtasPerSm = 3;

struct QuantSmem {
  uint4 rows[kStretch * kRowBytes / 16];
  uint32_t top[kStretch];                          // largest magnitude (bf16 bits) per scale block of the stretch
  float inv[kStretch];                             // 2^-e of its scale's exponent e
  uint64_t full;
};
static_assert((sizeof(QuantSmem) + 1024) * kCtasPerSm <= 228 * 1024, "three CTAs share an SM");

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }   // x >= 2^-126

// Smallest e in [kMinExp, kMaxExp] with 448 * 2^e >= the bf16 magnitude `bits`
// (448 = 1.75 * 2^8).
__device__ __forceinline__ int need_exp(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return bits < 0x80u || e < kMinExp ? kMinExp : (e > kMaxExp ? kMaxExp : e);
}

// Larger of two pairs of 16-bit magnitudes; with `finite`, infinite and NaN ones count as 0.
__device__ __forceinline__ uint32_t max2(uint32_t m, uint32_t v, bool finite) {
  v &= 0x7fff7fffu;
  if (finite) v &= __vcmpltu2(v, 0x7f807f80u);
  return __vmaxu2(m, v);
}

// Four bf16 (two words) times inv (a power of two: exact) -> four E4M3 codes.
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, float inv) {
  const float2 f = make_float2(inv, inv);
  const float2 x = mul2(make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)), f);
  const float2 y = mul2(make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)), f);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 16);
}

// A block's earlier scale may be any number, not only a power of two (a cache that was
// quantised elsewhere).  Quotients and products by one are rounded towards zero with the
// last bit set where anything was left (`rest`), so that the rounding to E4M3, of far fewer
// bits, is that of the exact value.  Beyond 512 (and for NaN) it saturates whatever the
// last bit.
__device__ __forceinline__ float to_odd(float y, float rest) {
  return rest != 0.f && fabsf(y) < 512.f ? __uint_as_float(__float_as_uint(y) | 1u) : y;
}
// x / m for m in [1, 2).
__device__ __forceinline__ float quotient(float x, float m) {
  const float y = __fdiv_rz(x, m);
  return to_odd(y, fmaf(-y, m, x));
}
__device__ __forceinline__ float product(float x, float f) {
  const float y = __fmul_rz(x, f);
  return to_odd(y, fmaf(x, f, -y));
}

// encode4 by any scale: inv = 2^-e and m = scale * 2^-e.
__device__ __noinline__ uint32_t encode4_any(uint32_t a, uint32_t b, float inv, float m) {
  const float2 x = make_float2(quotient(__uint_as_float(a << 16) * inv, m),
                               quotient(__uint_as_float(a & 0xffff0000u) * inv, m));
  const float2 y = make_float2(quotient(__uint_as_float(b << 16) * inv, m),
                               quotient(__uint_as_float(b & 0xffff0000u) * inv, m));
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3)) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3)) << 16);
}

__device__ __forceinline__ uint32_t reencode4(uint32_t v, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> (16 * h)), __NV_E4M3);
    const float2 y = __half22float2(__half2(x));
    r |= static_cast<uint32_t>(
             __nv_cvt_float2_to_fp8x2(make_float2(product(y.x, f), product(y.y, f)), __NV_SATFINITE, __NV_E4M3))
         << (16 * h);
  }
  return r;
}

// Whether token t begins a run.
__device__ __forceinline__ bool begins_run(const QuantParams& p, int t) {
  const int s = p.q_seq[t], x = p.q_pos[t];
  return t == 0 || x % kStretch == 0 || p.q_seq[t - 1] != s || p.q_pos[t - 1] != x - 1;
}

// Lists the tokens that begin runs (in any order: runs do not depend on one another).
__global__ void __launch_bounds__(256) find_runs_kernel(QuantParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x * blockDim.x + threadIdx.x, lane = threadIdx.x & 31;
  const bool lead = t < p.T && begins_run(p, t);
  const uint32_t m = __ballot_sync(0xffffffffu, lead);
  int at = 0;
  if (lane == 0 && m) at = atomicAdd(p.num_runs, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0);
  if (lead) p.runs[at + __popc(m & ((1u << lane) - 1))] = t;
}

__global__ void __launch_bounds__(kQuantThreads, kCtasPerSm) quantize_append_kernel(QuantParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  QuantSmem& S = *reinterpret_cast<QuantSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gl = p.block_log2, g = 1 << gl;
  if (tid == 0) {
    mbar_init(&S.full, 1);
    fence_mbar_init();
  }
  if (p.runs) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int runs = p.runs ? __ldcg(p.num_runs) : p.T;
  __syncthreads();
  uint32_t phase = 0;
  for (int run = blockIdx.x; run < runs; run += gridDim.x) {
    const int t0 = p.runs ? __ldcg(&p.runs[run]) : run;
    const int seq = p.q_seq[t0], pos = p.q_pos[t0];
    int ps = -1, pp = 0;
    if (t0 > 0) {
      ps = p.q_seq[t0 - 1];
      pp = p.q_pos[t0 - 1];
    }
    const bool follows = t0 > 0 && ps == seq && pp == pos - 1;
    if (!p.runs && follows && pos % kStretch != 0) continue;      // within another token's run
    const int first = pos & (kStretch - 1);        // row of the stretch that the run begins with
    // rows of the run: consecutive tokens of the sequence within the stretch
    uint32_t same[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int l = lane + 32 * h, t = t0 + l;
      same[h] = __ballot_sync(0xffffffffu,
                              t < p.T && l < kStretch - first && p.q_seq[t] == seq && p.q_pos[t] == pos + l);
    }
    int n = ~same[0] ? __ffs(~same[0]) - 1 : 32 + (~same[1] ? __ffs(~same[1]) - 1 : 32);
    bool ok = seq >= 0 && seq < p.num_seqs && pos >= 0 && (t0 == 0 || seq > ps || follows);
    // the rows are on their way while the place in the cache is looked up
    if (ok && tid == 0) {
      mbar_arrive_expect_tx(&S.full, n * kRowBytes);
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              smem_u32(S.rows)),
          "l"(p.kv + static_cast<int64_t>(t0) * DSA_D_QK), "r"(n * kRowBytes), "r"(smem_u32(&S.full))
          : "memory");
    }
    const bool loaded = ok;
    if (tid < kStretch) S.top[tid] = 0;
    uint32_t flag = ok ? 0u : DSA_DEV_BAD_QUERY;
    int64_t row = 0;                               // cache row of the run's first token
    if (ok) {
      const int len = p.kv_len[seq];
      if (p.page_size == 0) {
        const int64_t off = p.kv_offset[seq];
        row = off + pos;
        if (off < 0 || (off & (g - 1)) != 0) {
          n = 0;
          flag = DSA_DEV_BAD_QUERY;
        }
      } else {
        const int pg = pos / p.page_size < p.pages_per_seq
                           ? p.page_table[static_cast<int64_t>(seq) * p.pages_per_seq + pos / p.page_size]
                           : -1;
        row = pg < 0 ? p.kv_rows : static_cast<int64_t>(pg) * p.page_size + pos % p.page_size;
      }
      if (n > len - pos) {                         // tokens beyond their sequence
        n = max(len - pos, 0);
        flag |= DSA_DEV_BAD_QUERY;
      }
      if (n > 0 && row + n > p.kv_rows) {          // rows beyond the cache (with pages: all of them)
        n = row < p.kv_rows ? static_cast<int>(p.kv_rows - row) : 0;
        flag |= DSA_DEV_BAD_INDEX;
      }
      ok = n > 0;
    }
    if (flag && tid == 0) set_status(p.status, flag);
    // the scale of the block that the run begins within, if it held rows before
    const int b0 = first >> gl, last = (first + n - 1) >> gl;
    const int64_t blk = (row - (first & (g - 1))) >> gl;     // physical block of the run's first row
    const bool held = ok && (first & (g - 1)) != 0;
    const float s_old = held ? p.scale[blk] : 0.f;
    const bool s_ok = s_old >= pow2f(kMinExp) && s_old <= pow2f(kMaxExp);
    if (held && !s_ok && tid == 0) set_status(p.status, DSA_DEV_BAD_SCALE);
    bool done = true;
    if (loaded) {
      done = mbar_wait(&S.full, phase, p.status, nullptr);
      phase ^= 1;
    }
    // A copy that never landed: nothing is stored, and no other run is begun (a bulk copy
    // in flight keeps writing to this CTA's memory, so leave it one more wait).
    if (__syncthreads_or(!done)) {
      if (!done) mbar_wait(&S.full, phase ^ 1, p.status, nullptr);
      __syncthreads();
      return;
    }
    if (!ok) continue;
    // largest entries per block: warp w takes the run's rows w, w + 8, ...
    for (int i = warp; i < n; i += kWarps) {
      const uint4* src = S.rows + i * (kRowBytes / 16);
      auto largest = [&](bool finite) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const int c = u * 32 + lane;
          if (c < kRowBytes / 16) {
            const uint4 v = src[c];
            m = max2(max2(max2(max2(m, v.x, finite), v.y, finite), v.z, finite), v.w, finite);
          }
        }
        return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      };
      uint32_t m = largest(false);
      if (m >= 0x7f80u) m = largest(true);         // an infinity or NaN is among them
      if (lane == 0 && m) atomicMax(&S.top[(first + i) >> gl], m);
    }
    __syncthreads();
    float s0 = 0.f;                                // scale of the first block
    {
      const float need = pow2f(need_exp(S.top[b0]));
      s0 = s_ok ? fmaxf(need, s_old) : need;
    }
    if (tid >= b0 && tid <= last) {
      const float s = tid == b0 ? s0 : pow2f(need_exp(S.top[tid]));
      p.scale[blk + tid - b0] = s;
      S.inv[tid] = pow2f(-exponent(s));
    }
    // earlier rows of the first block, when its scale grows
    if (s_ok && s0 > s_old) {
      const float f = s_old / s0;
      uint4* dst = reinterpret_cast<uint4*>(p.kv8 + blk * g * DSA_D_QK);
      for (int i = tid; i < (first & (g - 1)) * (DSA_D_QK / 16); i += kQuantThreads) {
        uint4 c = dst[i];
        c.x = reencode4(c.x, f);
        c.y = reencode4(c.y, f);
        c.z = reencode4(c.z, f);
        c.w = reencode4(c.w, f);
        dst[i] = c;
      }
    }
    __syncthreads();
    // rows of the first block, where its scale is no power of two
    const int any = s0 != pow2f(exponent(s0)) ? min(n, ((b0 + 1) << gl) - first) : 0;
    if (any) {
      const float inv = S.inv[b0], m = s0 * inv;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(S.rows);
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.kv8 + row * DSA_D_QK);
      for (int c = tid; c < any * (DSA_D_QK / 4); c += kQuantThreads)
        dst[c] = encode4_any(src[2 * c], src[2 * c + 1], inv, m);
    }
    // codes of the new rows, 16 per thread and step
    uint4* out = reinterpret_cast<uint4*>(p.kv8 + row * DSA_D_QK);
    for (int c = any * kPieces + tid; c < n * kPieces; c += kQuantThreads) {
      const float inv = S.inv[(first + c / kPieces) >> gl];
      const uint4 a = S.rows[2 * c], b = S.rows[2 * c + 1];
      out[c] = make_uint4(encode4(a.x, a.y, inv), encode4(a.z, a.w, inv), encode4(b.x, b.y, inv),
                          encode4(b.z, b.w, inv));
    }
    __syncthreads();                               // the rows and tables are free for the next run
  }
}

}  // namespace

// The kernel's shared memory, once per device.
static cudaError_t prepare_device(size_t smem) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(quantize_append_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_quantize_append(const QuantParams& params, int sms, cudaStream_t stream) {
  if (params.T == 0) return cudaSuccess;
  QuantParams p = params;
  const size_t smem = sizeof(QuantSmem);
  cudaError_t e = prepare_device(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.blockDim = dim3(kQuantThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at = {};
  if (p.T <= kShortList) {
    p.runs = nullptr;
    cfg.gridDim = dim3(p.T);
  } else {
    find_runs_kernel<<<(p.T + 255) / 256, 256, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launches(1);
    const int most = kCtasPerSm * sms;
    cfg.gridDim = dim3(p.T < most ? p.T : most);
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
  }
  e = cudaLaunchKernelEx(&cfg, quantize_append_kernel, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dsa
