// Sparse (or dense) MLA over the 8-bit latent cache on sm_100a.
//
// For query t, head h and usable rows i with value c_i = s_i * code_i:
//   z_i = sm_scale q.c_i, p = softmax(z), out = sum_i p_i c_i[:512], lse = log sum exp z
//
// The cache's E4M3 codes are the tensor cores' operand as they lie in the cache: a
// row is gathered once (576 B) into shared memory and serves both products.  The
// bf16 side enters as a sum of two E4M3 numbers, hi + lo (8 significant bits, as
// many as bf16 has): x = hi + lo costs two FP8 MMAs, which run at twice the bf16
// rate, so a product takes the tensor time of the bf16 one with half the operand
// bytes and no decoding.  Everything is transposed, so that rows are the M
// dimension of the first product and the K dimension of the second:
//   S^T [128 rows, 64 hi | 64 lo] = codes [128, 576] . [Q_hi; Q_lo]^T     (N = 128)
//   O^T [512 dims, 64 heads]     += codes^T [512, 128] . (W_lo, then W_hi) (N = 64)
// with the weights w_ih = 2^(b_ih - m_h), b_ih = log2(e) z_ih + log2 s_i: the row's
// scale rides on its weight, and l_h = sum_i w_ih / s_i is the softmax denominator.
// The reference m_h puts the largest weight of the query's first tile at 2^5; E4M3
// holds up to 2^8.8, so m_h (and with it O and l) changes only when a later weight
// passes 2^8.5.  A weight has 8 significant bits down to 2^-7 of that largest one
// and an absolute error of at most 2^-15 of it below.
//
// One CTA per SM works through items (query, 64 heads, split of the row list).
// TMEM (512 columns): two S^T buffers of 128 columns, O^T as 4 x 64 columns.
// Shared memory (227 KB): Q 72 KB, two row tiles of 72 KB, W_lo 8 KB; W_hi lies over
// the row tile's RoPE part, which only the first product reads.  W_lo has one
// buffer, so the second product takes it first and gives it back half way.
// 20 warps: 0-3 and 4-7 softmax and output (one thread per row, 32 heads each), 8-15
// row gathers (16-byte cp.async) and the queries' hi/lo split, 16 issues S^T, 17 O^T.
// Registers: launched at 96 per thread, softmax 128, gathers 80, issuers 64.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kHT = 64;                            // heads per CTA
constexpr int kRows = 128;                         // rows per tile
constexpr int kSoftWarps = 8;
constexpr int kGatherWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kGatherWarps + 4);
constexpr int kLaunchRegs = 96, kSoftRegs = 128, kGatherRegs = 80, kIssueRegs = 64;
static_assert(32 * (kSoftWarps * kSoftRegs + kGatherWarps * kGatherRegs + 4 * kIssueRegs) == kThreads * kLaunchRegs,
              "the register split must add up to the launch allocation");
constexpr uint32_t kSCol = 0, kOCol = 256;         // TMEM columns
constexpr float kTop = 5.f;                        // log2 of the largest weight when m is set
constexpr float kLimit = 8.5f;                     // log2 of the weight that makes m move
constexpr int kMaxSplits = 64;
constexpr int kBarSoft = 1;                        // named barriers: 1, 2 softmax groups, 3 gathers
constexpr int kBarGather = 3;

struct Tile {                                      // 128 rows: latent as 4 x 128 B (SW128), RoPE 64 B (SW64)
  uint8_t lat[4][kRows * 128];
  uint8_t rope[kRows * 64];
};

struct Q8Smem {
  Tile q;                                          // rows 0-63: hi of head h, 64-127: lo
  Tile rows[2];
  uint8_t w_lo[kRows * 64];
  float s_row[2][kRows];                           // row scales, 0 = unused row
  float red[2][4][32];
  float qs[2][kHT];                                // 2^-e of each head's query
  float m[kHT];
  uint64_t rows_full[2], rows_empty[2], s_full[2], s_free[2], w_full, wlo_free, q_full, q_free, o_full, o_free,
      plan_full[2], plan_free[2], done;
  int plan[2];                                     // tiles of the item
  int last[kGatherWarps];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Q8Smem) <= 232448, "exceeds the 227 KB a CTA can have");

__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;   // descriptor version (sm_100)
  d |= 4ull << 61;   // SWIZZLE_64B
  return d;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Two fp32 -> E4M3 hi and lo with hi + lo = the value to 8 significant bits (low byte
// = a).  Through fp16, which holds 11 bits: |x| <= 448 and steps of 2^-24 near zero,
// both beyond what hi and lo can hold.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  uint32_t x, h, r;
  uint16_t hb, lb;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hb) : "r"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(hb));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(h));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lb) : "r"(r));
  hi = hb;
  lo = lb;
}

// Bounded wait that gives up at once when a thread of the CTA has given up.  Warps
// that meet on a named barrier leave their loops together: they agree on it there
// (bar_or), so none is left waiting.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* ab) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  return *ab == 0 && mbar_wait(bar, parity, status, ab);
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// v[0] of lane l = the reduction of v[l] over the warp's lanes.
template <bool kMax>
__device__ __forceinline__ float reduce_transposed(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// An item: query t, heads 64 hg .., entries [e0, e1) of its row list.
struct Item {
  int t, hg, sp;
  int seq, len;
  int64_t base;              // first cache row (contiguous)
  int e0, e1;
  bool ok;
};

__device__ __forceinline__ void item_place(const MlaQ8Params& p, int it, Item& I) {
  I.hg = it % p.groups;
  const int r = it / p.groups;
  I.sp = r % p.splits;
  I.t = r / p.splits;
}

__device__ __forceinline__ void item_list(const MlaQ8Params& p, Item& I) {
  I.seq = p.q_seq[I.t];
  const bool seq_ok = I.seq >= 0 && I.seq < p.num_seqs;
  I.len = seq_ok ? p.kv_len[I.seq] : 0;
  I.base = seq_ok && p.page_size == 0 ? p.kv_offset[I.seq] : 0;
  I.ok = seq_ok && I.len >= 0 &&
         (p.page_size == 0 ? I.base >= 0 && I.base + I.len <= p.kv_rows
                           : I.len <= static_cast<int64_t>(p.pages_per_seq) * p.page_size);
  int n = p.k;
  if (!p.idx) {
    const int pos = p.q_pos[I.t];
    I.ok = I.ok && pos >= 0 && pos < I.len;
    n = pos + 1;
  }
  I.e0 = I.sp * p.split_tiles * kRows;
  I.e1 = I.ok ? min(n, I.e0 + p.split_tiles * kRows) : I.e0;
}

__global__ void __launch_bounds__(kThreads, 1) mla_q8_kernel(MlaQ8Params p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Q8Smem& S = *reinterpret_cast<Q8Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* ab = &S.abort;
  if (tid == 0) {
    S.abort = 0;
    if (smem_u32(raw) & 1023u) {
      S.abort = 1;
      set_status(p.status, DSA_DEV_INTERNAL);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.rows_full[b], 32 * kGatherWarps + kGatherWarps);
      mbar_init(&S.rows_empty[b], 1);
      mbar_init(&S.s_full[b], 1);
      mbar_init(&S.s_free[b], kSoftWarps);
      mbar_init(&S.plan_full[b], 1);
      mbar_init(&S.plan_free[b], kSoftWarps + 2);
    }
    mbar_init(&S.w_full, kSoftWarps);
    mbar_init(&S.wlo_free, 1);
    mbar_init(&S.q_full, kGatherWarps);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_free, kSoftWarps);
    mbar_init(&S.done, 2);
    fence_mbar_init();
  }
  if (warp == kSoftWarps + kGatherWarps) tmem_alloc(&S.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int step = gridDim.x;

  if (warp < kSoftWarps) {
    // ================================================================ softmax and output
    setmaxnreg_inc<kSoftRegs>();
    const int grp = warp >> 2, quad = warp & 3;     // heads 32 grp .., rows 32 quad ..
    const int r = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const float c0 = p.sm_scale * 1.4426950408889634f;
    uint32_t g = 0, items_done = 0;                 // tiles and non-empty items so far
    bool bad = false;                               // a wait of this thread ran out
    for (int kk = 0, it = blockIdx.x; it < p.items; ++kk, it += step) {
      Item I;
      item_place(p, it, I);
      bad |= !wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab);
      const int tiles = S.plan[kk & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.plan_free[kk & 1]);
      const int h0 = I.hg * kHT + grp * 32;
      const float* qs = S.qs[items_done & 1] + grp * 32;
      float l[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) l[i] = 0.f;
      bool seen = false;                            // a usable row so far
      if (quad == 0) S.m[grp * 32 + lane] = 0.f;
      if (bar_or(kBarSoft + grp, 128, bad)) break;
      bool stop = false;
      for (int j = 0; j < tiles; ++j, ++g) {
        const int b = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        bad |= !wait(&S.rows_full[b], ph, p.status, ab) || !wait(&S.s_full[b], ph, p.status, ab);
        __syncwarp();
        tc_fence_after();
        const float s = S.s_row[b][r];
        const float c = c0 * s;
        const float sg = s > 0.f ? lg2_approx(s) : -INFINITY;
        const float inv = s > 0.f ? 1.f / s : 0.f;
        // x = b - m, the log2 of the weight
        float x[32];
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t hi[16], lo[16];
          tmem_ld16(tmem + lanes + kSCol + b * 128 + grp * 32 + q * 16, hi);
          tmem_ld16(tmem + lanes + kSCol + b * 128 + 64 + grp * 32 + q * 16, lo);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int h = q * 16 + i;
            const float2 sc = *reinterpret_cast<const float2*>(&qs[h]);
            const float2 mm = *reinterpret_cast<const float2*>(&S.m[grp * 32 + h]);
            const float2 d = make_float2(__uint_as_float(hi[i]) + __uint_as_float(lo[i]),
                                         __uint_as_float(hi[i + 1]) + __uint_as_float(lo[i + 1]));
            const float2 y = ffma2(d, make_float2(sc.x * c, sc.y * c), make_float2(sg - mm.x, sg - mm.y));
            x[h] = y.x;
            x[h + 1] = y.y;
            top = fmaxf(top, fmaxf(y.x, y.y));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.s_free[b]);
        const bool usable = s > 0.f;
        if (bar_or(kBarSoft + grp, 128, bad || (seen ? top > kLimit : usable))) {
          if ((stop = bar_or(kBarSoft + grp, 128, bad))) break;
          // move the reference of the heads that need it (all of them at the first usable rows)
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = usable ? x[i] : -INFINITY;
          S.red[grp][quad][lane] = reduce_transposed<true>(v, lane);
          named_bar_sync(kBarSoft + grp, 128);
          const float mx = fmaxf(fmaxf(S.red[grp][0][lane], S.red[grp][1][lane]),
                                 fmaxf(S.red[grp][2][lane], S.red[grp][3][lane]));
          const float up = (seen ? mx > kLimit : mx > -INFINITY) ? mx - kTop : 0.f;
          const float f = ex2_approx(-up);          // of head 32 grp + lane
          if (quad == 0) S.m[grp * 32 + lane] += up;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] -= __shfl_sync(0xffffffffu, up, i);
            l[i] *= seen ? __shfl_sync(0xffffffffu, f, i) : 1.f;
          }
          if (seen) {
            // O so far: wait for the product of the tile before this one
            bad |= !wait(&S.rows_empty[b ^ 1], ((g - 1) >> 1) & 1, p.status, ab);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
              const uint32_t at = tmem + lanes + kOCol + (q >> 1) * 64 + grp * 32 + (q & 1) * 16;
              uint32_t o[16];
              tmem_ld16(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, f, (q & 1) * 16 + i));
              tmem_st16(at, o);
            }
            tmem_st_wait();
          }
          seen = true;
          named_bar_sync(kBarSoft + grp, 128);      // m is set, red may be reused
        }
        // weights
        bad |= g > 0 && !wait(&S.wlo_free, (g - 1) & 1, p.status, ab);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t wh[4], wl[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, b0, a1, b1;
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2_approx(x[q * 16 + i * 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int h = q * 16 + i * 4 + e;
              const float2 y = ffma2(make_float2(w[e], w[e + 1]), make_float2(inv, inv), make_float2(l[h], l[h + 1]));
              l[h] = y.x;
              l[h + 1] = y.y;
            }
            split2(w[0], w[1], a0, b0);
            split2(w[2], w[3], a1, b1);
            wh[i] = a0 | (a1 << 16);
            wl[i] = b0 | (b1 << 16);
          }
          const uint32_t at = r * 64 + (((grp * 2 + q) ^ ((r >> 1) & 3)) << 4);
          *reinterpret_cast<uint4*>(&S.rows[b].rope[at]) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
          *reinterpret_cast<uint4*>(&S.w_lo[at]) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.w_full);
      }
      if (stop) break;
      // denominators: over the warp's rows, then over the four warps
      S.red[grp][quad][lane] = reduce_transposed<false>(l, lane);
      if (bar_or(kBarSoft + grp, 128, bad)) break;
      const float total = (S.red[grp][0][lane] + S.red[grp][1][lane]) + (S.red[grp][2][lane] + S.red[grp][3][lane]);
      const float inv_l = total == 0.f ? 0.f : 1.f / total;
      const int64_t row = p.splits == 1 ? static_cast<int64_t>(I.t) * p.H
                                        : (static_cast<int64_t>(I.t) * p.splits + I.sp) * p.H;
      if (quad == 0 && h0 + lane < p.H) {
        const float lse = total == 0.f ? -INFINITY : (S.m[grp * 32 + lane] + log2f(total)) * 0.6931471805599453f;
        if (p.splits > 1)
          p.part_lse[row + h0 + lane] = lse;
        else if (p.lse)
          p.lse[row + h0 + lane] = lse;
      }
      named_bar_sync(kBarSoft + grp, 128);          // red and m may be reused
      if (tiles > 0) {
        bad |= !wait(&S.o_full, items_done & 1, p.status, ab);
        __syncwarp();
        tc_fence_after();
        ++items_done;
      }
      if (p.splits > 1 && tiles == 0) continue;     // the combine skips parts of weight 0
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        const int mt = q >> 1, hc = (q & 1) * 16;
        uint32_t o[16];
        if (tiles > 0) {
          tmem_ld16(tmem + lanes + kOCol + mt * 64 + grp * 32 + hc, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y = __uint_as_float(o[i]) * __shfl_sync(0xffffffffu, inv_l, hc + i);
          const int h = h0 + hc + i;
          if (h < p.H) {
            const int64_t at = (row + h) * DSA_D_V + mt * 128 + r;
            if (p.splits > 1)
              p.part_o[at] = y;
            else
              p.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
          }
        }
      }
      if (tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_free);
      }
    }
  } else if (warp < kSoftWarps + kGatherWarps) {
    // ================================================================ queries and rows
    setmaxnreg_dec<kGatherRegs>();
    const int gw = warp - kSoftWarps, gt = tid - 32 * kSoftWarps;
    uint32_t g = 0, nq = 0;
    int prev_tiles = 0;                             // of the last non-empty item
    bool bad = false;                               // a wait of this thread ran out
    for (int kk = 0, it = blockIdx.x; it < p.items; ++kk, it += step) {
      Item I;
      item_place(p, it, I);
      item_list(p, I);
      if (!I.ok && gt == 0) set_status(p.status, DSA_DEV_BAD_QUERY);
      // tiles up to the last usable entry
      int tiles = I.e1 > I.e0 ? (I.e1 - I.e0 + kRows - 1) / kRows : 0;
      const int32_t* list = p.idx ? p.idx + static_cast<int64_t>(I.t) * p.k : nullptr;
      if (!list && __any_sync(0xffffffffu, bad)) break;
      if (list && tiles > 0) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = I.e0 + i * 256 + gt;
          v[i] = e < I.e1 ? __ldg(list + e) : -1;
        }
        int last = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (v[i] >= I.len) set_status(p.status, DSA_DEV_BAD_INDEX);
          if (v[i] >= 0 && v[i] < I.len) last = i * 256 + gt;
        }
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) S.last[gw] = last;
        if (bar_or(kBarGather, 32 * kGatherWarps, bad)) break;
#pragma unroll
        for (int i = 0; i < kGatherWarps; ++i) last = max(last, S.last[i]);
        tiles = last / kRows + (last >= 0 ? 1 : 0);
        named_bar_sync(kBarGather, 32 * kGatherWarps);
      }
      if (gt == 0) {
        bad |= kk > 1 && !wait(&S.plan_free[kk & 1], ((kk - 2) >> 1) & 1, p.status, ab);
        S.plan[kk & 1] = tiles;
        mbar_arrive(&S.plan_full[kk & 1]);
      }
      if (tiles == 0) continue;
      // the lane's entries: lanes 0-15 rows 16 gw .. of the pair's first tile, 16-31 of its second
      auto entry = [&](int pair) {
        const int e = I.e0 + (2 * pair + (lane >> 4)) * kRows + gw * 16 + (lane & 15);
        const int v = e < I.e1 ? (list ? __ldg(list + e) : e) : -1;
        return v < I.len ? v : -1;
      };
      auto page = [&](int v) {
        return v >= 0 && p.page_size
                   ? __ldg(p.page_table + static_cast<int64_t>(I.seq) * p.pages_per_seq + v / p.page_size)
                   : 0;
      };
      auto place = [&](int v, int pg) -> int {      // cache row, -1 = none (the host checks kv_rows < 2^31)
        if (v < 0) return -1;
        const int64_t row = p.page_size ? static_cast<int64_t>(pg) * p.page_size + v % p.page_size : I.base + v;
        if (pg < 0 || row >= p.kv_rows) {
          set_status(p.status, DSA_DEV_BAD_INDEX);
          return -1;
        }
        return static_cast<int>(row);
      };
      auto scale_of = [&](int row) { return row >= 0 ? __ldg(p.scale + (row >> p.block_log2)) : 0.f; };
      int v_cur = entry(0), v_nxt = entry(1);

      // the item's queries, once the products of the last item have read its own; qs has
      // two places, so the softmax must be through with the item before that (it is,
      // unless the last item was a single tile, whose product may run ahead of it)
      bad |= nq > 0 && !wait(&S.q_free, (nq - 1) & 1, p.status, ab);
      if (prev_tiles == 1 && nq > 1) bad |= !wait(&S.s_free[g & 1], ((g - 2) >> 1) & 1, p.status, ab);
      prev_tiles = tiles;
      for (int hl = gw; hl < kHT; hl += kGatherWarps) {
        const int h = I.hg * kHT + hl;
        uint32_t w[9];
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(p.q + (static_cast<int64_t>(I.t) * p.H + h) * DSA_D_QK);
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = h < p.H ? __ldg(src + i * 32 + lane) : 0u;
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 9; ++i) am = max(am, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        am = __reduce_max_sync(0xffffffffu, am);
        // times 2^e: the largest entry in [2^7, 2^8)
        int e = am >= 0x80u ? 7 + 127 - static_cast<int>(am >> 7) : 120;
        e = e > 120 ? 120 : (e < -120 ? -120 : e);
        const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        if (lane == 0) S.qs[nq & 1][hl] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 9; ++i) {
          uint32_t hi, lo;
          split2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up, hi, lo);
          if (am >= 0x7f80u) hi = 0x7f7fu;          // an infinity or NaN: the head's results are NaN
          const int byte = 2 * (lane + 32 * i);
          if (i < 8) {
            const uint32_t at = (((byte & 127) >> 4) ^ (hl & 7)) * 16 + (byte & 15);
            *reinterpret_cast<uint16_t*>(&S.q.lat[i >> 1][hl * 128 + at]) = static_cast<uint16_t>(hi);
            *reinterpret_cast<uint16_t*>(&S.q.lat[i >> 1][(hl + kHT) * 128 + at]) = static_cast<uint16_t>(lo);
          } else {
            const uint32_t at = (((byte & 63) >> 4) ^ ((hl >> 1) & 3)) * 16 + (byte & 15);
            *reinterpret_cast<uint16_t*>(&S.q.rope[hl * 64 + at]) = static_cast<uint16_t>(hi);
            *reinterpret_cast<uint16_t*>(&S.q.rope[(hl + kHT) * 64 + at]) = static_cast<uint16_t>(lo);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_full);
      ++nq;

      // rows, tile by tile; the next pair's page, row and scale are looked up meanwhile
      int row = place(v_cur, page(v_cur));
      float sc = scale_of(row);
      int pg_nxt = page(v_nxt);
      for (int j = 0; j < tiles; ++j, ++g) {
        if (!(sc >= 7.888609e-31f && sc <= 1.2676506e30f)) {   // 2^-100 .. 2^100
          if (row >= 0) set_status(p.status, DSA_DEV_BAD_SCALE);
          row = -1;
          sc = 0.f;
        }
        const int b = g & 1, half = j & 1;
        bad |= g > 1 && !wait(&S.rows_empty[b], ((g - 2) >> 1) & 1, p.status, ab);
        if (__any_sync(0xffffffffu, bad)) break;
        const uint32_t lat = smem_u32(S.rows[b].lat[0]) + (lane >> 3) * (kRows * 128);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int rr = gw * 16 + i;
          const int src = __shfl_sync(0xffffffffu, row, half * 16 + i);
          cp_async16(lat + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4),
                     p.kv8 + static_cast<int64_t>(max(src, 0)) * DSA_D_QK + lane * 16, src < 0 ? 0u : 16u);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rl = i * 8 + (lane >> 2), rr = gw * 16 + rl;
          const int src = __shfl_sync(0xffffffffu, row, half * 16 + rl);
          cp_async16(smem_u32(S.rows[b].rope) + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4),
                     p.kv8 + static_cast<int64_t>(max(src, 0)) * DSA_D_QK + DSA_D_V + (lane & 3) * 16,
                     src < 0 ? 0u : 16u);
        }
        if ((lane >> 4) == half) S.s_row[b][gw * 16 + (lane & 15)] = row < 0 ? 0.f : sc;
        cp_async_arrive_noinc(&S.rows_full[b]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.rows_full[b]);
        if (half) {
          row = place(v_nxt, pg_nxt);
          sc = scale_of(row);
          v_nxt = entry((j >> 1) + 2);
          pg_nxt = page(v_nxt);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    setmaxnreg_dec<kIssueRegs>();
    if (warp == kSoftWarps + kGatherWarps && lane == 0) {
      // ================================================================ S^T = codes . Q^T
      const uint32_t id = instr_desc(0, 0, false, false, 128, 2 * kHT);
      const uint64_t q_lat = smem_desc_sw128(smem_u32(S.q.lat[0]), 16, 1024);
      const uint64_t q_rope = smem_desc_sw64(smem_u32(S.q.rope), 512);
      uint32_t g = 0, nq = 0;
      bool ok = true;
      for (int kk = 0, it = blockIdx.x; it < p.items && ok; ++kk, it += step) {
        if (!wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab)) break;
        const int tiles = S.plan[kk & 1];
        mbar_arrive(&S.plan_free[kk & 1]);
        if (tiles == 0) continue;
        if (!wait(&S.q_full, nq & 1, p.status, ab)) break;
        ++nq;
        for (int j = 0; j < tiles; ++j, ++g) {
          const int b = g & 1;
          const uint32_t ph = (g >> 1) & 1;
          if ((g > 1 && !wait(&S.s_free[b], ph ^ 1, p.status, ab)) ||
              !wait(&S.rows_full[b], ph, p.status, ab)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();                 // cp.async writes -> tensor-core reads
          tc_fence_after();
          const uint64_t a_lat = smem_desc_sw128(smem_u32(S.rows[b].lat[0]), 16, 1024);
          const uint64_t a_rope = smem_desc_sw64(smem_u32(S.rows[b].rope), 512);
          const uint32_t d = tmem + kSCol + b * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8(d, a_lat + c * (kRows * 128 / 16) + k * 2, q_lat + c * (kRows * 128 / 16) + k * 2, id,
                      (c | k) != 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 2; ++k) umma_f8(d, a_rope + k * 2, q_rope + k * 2, id, 1u);
          umma_commit(&S.s_full[b]);
        }
        if (!ok) break;
        umma_commit(&S.q_free);
      }
      umma_commit(&S.done);
      mbar_wait(&S.done, 0, p.status, nullptr);
    } else if (warp == kSoftWarps + kGatherWarps + 1 && lane == 0) {
      // ================================================================ O^T += codes^T . W
      const uint32_t id = instr_desc(0, 0, true, true, 128, kHT);
      const uint64_t w_lo = smem_desc_sw64(smem_u32(S.w_lo), 512);
      uint32_t g = 0, no = 0;
      bool ok = true;
      for (int kk = 0, it = blockIdx.x; it < p.items && ok; ++kk, it += step) {
        if (!wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab)) break;
        const int tiles = S.plan[kk & 1];
        mbar_arrive(&S.plan_free[kk & 1]);
        if (tiles == 0) continue;
        if (no > 0 && !wait(&S.o_free, (no - 1) & 1, p.status, ab)) break;
        ++no;
        for (int j = 0; j < tiles; ++j, ++g) {
          const int b = g & 1;
          if (!wait(&S.w_full, g & 1, p.status, ab)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = smem_desc_sw128(smem_u32(S.rows[b].lat[0]), 16, 1024);
          const uint64_t w_hi = smem_desc_sw64(smem_u32(S.rows[b].rope), 512);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8(tmem + kOCol + mt * 64, a + mt * (kRows * 128 / 16) + k * (32 * 128 / 16),
                      w_lo + k * (32 * 64 / 16), id, (j | k) != 0 ? 1u : 0u);
          umma_commit(&S.wlo_free);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8(tmem + kOCol + mt * 64, a + mt * (kRows * 128 / 16) + k * (32 * 128 / 16),
                      w_hi + k * (32 * 64 / 16), id, 1u);
          umma_commit(&S.rows_empty[b]);
        }
        if (!ok) break;
        umma_commit(&S.o_full);
      }
      umma_commit(&S.done);
      mbar_wait(&S.done, 0, p.status, nullptr);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kGatherWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a split row list: lse = log sum exp(lse_i), out = sum exp(lse_i - lse) o_i.
__global__ void __launch_bounds__(128) combine_kernel(MlaQ8Params p) {
  __shared__ float wgt[kMaxSplits];
  __shared__ float s_lse;
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int64_t at = static_cast<int64_t>(t) * p.splits * p.H + h;
  if (tid < 32) {
    float v[2], mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + 32 * i;
      v[i] = s < p.splits ? p.part_lse[at + static_cast<int64_t>(s) * p.H] : -INFINITY;
      mx = fmaxf(mx, v[i]);
    }
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float e[2], den = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      e[i] = v[i] == -INFINITY ? 0.f : exp2f((v[i] - mx) * 1.4426950408889634f);
      den += e[i];
    }
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (tid + 32 * i < p.splits) wgt[tid + 32 * i] = den == 0.f ? 0.f : e[i] / den;
    if (tid == 0) s_lse = den == 0.f ? -INFINITY : mx + logf(den);
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < p.splits; ++s) {
    const float w = wgt[s];
    if (w == 0.f) continue;                         // also the parts that nothing was written for
    const float4 o =
        *reinterpret_cast<const float4*>(p.part_o + (at + static_cast<int64_t>(s) * p.H) * DSA_D_V + tid * 4);
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * p.H + h) * DSA_D_V + tid * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (tid == 0 && p.lse) p.lse[static_cast<int64_t>(t) * p.H + h] = s_lse;
}

}  // namespace

// Splits of the row lists: with few queries a list is cut so that its parts fill
// the SMs.  The choice minimises (waves of items) x (tiles of an item + 3): an item
// costs about three tiles' time beside its tiles (the queries' split, the first
// row latencies, the output).
int mla_q8_plan(int T, int H, int max_entries, int sms, int* split_tiles) {
  const int64_t base = static_cast<int64_t>(T) * ((H + kHT - 1) / kHT);
  const int tiles = max_entries > 0 ? (max_entries + kRows - 1) / kRows : 1;
  int best = 1, best_tiles = tiles;
  int64_t best_cost = -1;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    const int per = (tiles + s - 1) / s;
    if ((tiles + per - 1) / per != s) continue;
    const int64_t cost = (base * s + sms - 1) / sms * (per + 3);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
      best_tiles = per;
    }
  }
  *split_tiles = best_tiles;
  return best;
}

cudaError_t launch_sparse_mla_q8(const MlaQ8Params& params, int sms, cudaStream_t stream) {
  MlaQ8Params p = params;
  if (p.T == 0) return cudaSuccess;
  const size_t smem = sizeof(Q8Smem);
  cudaError_t e = cudaFuncSetAttribute(mla_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // The register split adds up only at kLaunchRegs per thread: with fewer, an
  // increase would never be granted.
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, mla_q8_kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  p.groups = (p.H + kHT - 1) / kHT;
  const int64_t items = static_cast<int64_t>(p.T) * p.splits * p.groups;
  if (items > 0x7fffffff - sms) return cudaErrorInvalidConfiguration;
  p.items = static_cast<int>(items);
  mla_q8_kernel<<<p.items < sms ? p.items : sms, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (p.splits == 1) return e;
  combine_kernel<<<dim3(p.T, p.H), 128, 0, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dsa
