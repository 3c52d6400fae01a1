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
// The reference m_h puts the sum of the first tile's largest weights at 2^6.25 or more, the
// largest itself at 2^5 (when there are many) to 2^7 (when there is one); E4M3 holds up
// to 2^8.9, so m_h (and with it O and l) changes only when a later weight passes that.
// A weight has 8 significant bits down to 2^-2 and steps of 2^-9 below that, too coarse
// for the thousands of small weights beside a large one.  So they are not rounded to the
// nearest step, which takes them all or none, but up or down in the right proportion: an
// offset that differs from row to row, evenly spread over a step, is added first.  The
// sum of many keeps its value: its deviation is at most 2^-8.6 of the values' size and does
// not grow with the list.  (Rounding to nearest, with the largest at 2^5, lost 3% of the
// output beside a weight of 0.8 over 8191 rows and 12% over 32768.  The offsets cost the
// prefill of 4096 queries 3%.  A largest weight of 2^7 throughout is as exact, but the
// reference then moves in most lists: 3290 us against 2740.)
//
// One CTA per SM works through items (query, 64 heads, split of the row list), the
// first by its index and the others off a counter (lists are ragged).
// TMEM (512 columns): two S^T buffers of 128 columns, O^T as 4 x 64 columns.
// Shared memory (227 KB): Q 72 KB, two row tiles of 72 KB, W_lo 8 KB; W_hi lies over
// the row tile's RoPE part, which only the first product reads.  The second product
// goes by quarters of 32 rows (one K step, all dims, lo and hi), each of which gives
// its rows and weights back, so the next tile's rows and weights follow it closely.
// Bound by the chain through the two row tiles: a tile's rows, S^T, weights and O^T take
// some 8,800 clocks and the tensor work in them 2,850, so a tile takes 4,300 to 4,800;
// beside them an item costs some 10,000 (the queries' split 6,000, first rows, output).
// A third row tile does not fit beside the queries.  Near its limit is the shared-memory
// port: the products read 344 KB of operands per tile (ncu: 48% of its clocks), loads,
// stores and gathers take 32% (tensor pipe 39%, issue slots 51%, DRAM 7%).
// Measured on the device: 4096 queries, 128 heads, 2048 rows each, 2.76 to 2.83 ms (846 to
// 825 TFLOP/s of the bf16 product's work, under the power cap); 64 contexts of 2048 selected
// rows 59 us; 24 ragged contexts of 1 .. 8191 rows, dense, 61 to 67 us; one query 18.5 us.
//
// 32 warps: 0-15 softmax (warp w: rows 32 (w mod 4) .., 16 heads) and, between items,
// the next queries' hi/lo split, 16-23 row gathers (16-byte cp.async), 24-27 the
// output (while the softmax is at the next item), 28 issues S^T, 29 O^T (as whole warps,
// so that the descriptors are worked out in uniform registers; a lone lane's cost
// some 100 clocks a product to issue).  Registers:
// launched at 64 per thread, softmax 80, gathers 56, output 48, issuers 32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kHT = 64;                            // heads per CTA
constexpr int kRows = 128;                         // rows per tile
constexpr int kSoftWarps = 16;
constexpr int kGroups = kSoftWarps / 4;            // softmax groups of four warps (128 rows)
constexpr int kGH = kHT / kGroups;                 // heads per group
constexpr int kGatherWarps = 8;
constexpr int kOutWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kGatherWarps + kOutWarps + 4);
constexpr int kLaunchRegs = 64, kSoftRegs = 80, kGatherRegs = 56, kOutRegs = 48, kIssueRegs = 32;
static_assert(32 * (kSoftWarps * kSoftRegs + kGatherWarps * kGatherRegs + kOutWarps * kOutRegs + 4 * kIssueRegs) ==
                  kThreads * kLaunchRegs,
              "the register split must add up to the launch allocation");
constexpr uint32_t kSCol = 0, kOCol = 256;         // TMEM columns
// Weights are held as w / 2^8 until their codes are formed (see split4).
constexpr float kTop = 7.f - 8.f;                  // log2 of the largest weights' sum when m is set (see top_sum)
constexpr float kLimit = 8.9f - 8.f;               // log2 of the weight that makes m move (codes end below 2^8.9)
constexpr float kStep = 1.f / (1 << 17);           // the smallest step of the weights' codes
constexpr float kNaN = __builtin_nanf("");
constexpr int kMaxSplits = 64;

struct Tile {                                      // 128 rows: latent as 4 x 128 B (SW128), RoPE 64 B (SW64)
  uint8_t lat[4][kRows * 128];
  uint8_t rope[kRows * 64];
};

struct Q8Smem {
  Tile q;                                          // rows 0-63: hi of head h, 64-127: lo
  Tile rows[2];
  uint8_t w_lo[kRows * 64];
  float s_row[2][kRows];                           // row scales, 0 = unused row
  float red[kGroups][4][kGH];
  uint32_t top_s[kGroups][4];                      // largest row scales (bits), beside red
  float qs[kHT];                                   // scale of each head's query
  float m[kHT];                                    // minus the references
  uint64_t rows_full[2], rows_empty[2][4], s_full[2], s_free[2], w_full[4], q_full, q_free, o_full, o_free, l_full,
      l_free, plan_full[2], plan_free[2], vote[kGroups], sync[kGroups], gather_sync, done;
  int over[kGroups][2];                            // a weight of the group passed the limit (by tile parity)
  int plan[2], item[2];                            // tiles of an item and its number, -1 after the last
  int drawn[2];                                    // item numbers on their way to the gather warps
  int last[kGatherWarps];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Q8Smem) <= 232448, "exceeds the 227 KB a CTA can have");

// Every warpgroup calls this first thing in its role: an increase waits until the
// others have given back enough of the launch allocation.
template <int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > kLaunchRegs) setmaxnreg_inc<N>();
  if constexpr (N < kLaunchRegs) setmaxnreg_dec<N>();
}

// Upper words of the operands' descriptors (8-row groups 1024 and 512 bytes apart;
// descriptor version, swizzle); the lower word is the start address over 16.
constexpr uint32_t kDesc128 = (1024u >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDesc64 = (512u >> 4) | 1u << 14 | 4u << 29;
__device__ __forceinline__ uint32_t desc_lo(const void* p) { return ((smem_u32(p) >> 4) & 0x3fffu) | 1u << 16; }

// D[tmem] (+)= A . B, E4M3 operands.
template <uint32_t kDescA, uint32_t kDescB>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a), "n"(kDescA), "r"(b), "n"(kDescB), "r"(id), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 2 x + c on the multiply pipe: the integer pipe (64 lanes a clock and SM, as are the
// fp16 packing and half of it the E4M3 conversions) is what the softmax runs short of.
__device__ __forceinline__ uint32_t twice_plus(uint32_t x, uint32_t c) {
  uint32_t y;
  asm("mad.lo.u32 %0, %1, 2, %2;" : "=r"(y) : "r"(x), "r"(c));
  return y;
}

// Four fp32 values of magnitude below 2 -> E4M3 codes of hi and lo, hi + lo = 2^8 times
// the value to 8 significant bits (byte i = value i).  By way of fp16: with the 2^8
// taken off, E4M3's exponent field equals fp16's low four exponent bits, its
// subnormals start where fp16's do, and a code is bits 7 .. 14 of the fp16 pattern
// (bit 14 is 0 below 2).  So hi is the pattern cut after 3 mantissa bits, lo the
// exact rest rounded to 3.  NaN stays NaN in hi.
// Without kSigned negative values count as 0.
template <bool kSigned>
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  uint32_t x0, x1, r0, r1;
  if (kSigned) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x0) : "f"(b), "f"(a));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x1) : "f"(d), "f"(c));
  } else {
    asm("cvt.rn.relu.f16x2.f32 %0, %1, %2;" : "=r"(x0) : "f"(b), "f"(a));
    asm("cvt.rn.relu.f16x2.f32 %0, %1, %2;" : "=r"(x1) : "f"(d), "f"(c));
  }
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r0) : "r"(x0), "r"(x0 & 0xff80ff80u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(x1), "r"(x1 & 0xff80ff80u));
  hi = __byte_perm(twice_plus(x0, 0), twice_plus(x1, 0), 0x7531);
  lo = __byte_perm(twice_plus(r0, 0x00800080u), twice_plus(r1, 0x00800080u), 0x7531);
  if (kSigned) {                                    // the doubling moved the signs out; lo's is hi's
    const uint32_t sign = __byte_perm(x0, x1, 0x7531);
    hi |= sign & 0x80808080u;
    lo |= sign & 0x80808080u;
  }
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }

// Two bf16 -> fp32 (the lower one shifted up on the multiply pipe).
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  uint32_t lo;
  asm("mad.lo.u32 %0, %1, 65536, 0;" : "=r"(lo) : "r"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Bounded wait that gives up at once when a thread of the CTA has given up.  Warps
// meet on such waits only (no named barriers), so one that leaves strands no other.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* ab) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  return *ab == 0 && mbar_wait(bar, parity, status, ab);
}

// The warps of a group meet (`bar` counts one arrival per warp, `phase` its use).
__device__ __forceinline__ bool meet(uint64_t* bar, uint32_t& phase, int lane, uint32_t* status, volatile int* ab) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  const bool ok = wait(bar, phase & 1, status, ab);
  ++phase;
  __syncwarp();
  return ok;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ float rcp_approx(float x) {   // one ulp; exact for powers of two
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The reduction of v[l mod 16] over the warp's lanes, for lane l.
template <bool kMax>
__device__ __forceinline__ float reduce_transposed(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
}

// An item: query t, heads 64 hg .., entries [e0, e1) of its row list.
struct Item {
  int t, hg, sp;
  int seq, len;
  int64_t base;              // first cache row (contiguous)
  int e0, e1;
  bool ok;
};

// Items go head group by head group (neighbours share their rows in L2), query by query,
// and part by part of the lists, so that the parts that short lists lack come last.
__device__ __forceinline__ void item_place(const MlaQ8Params& p, int it, Item& I) {
  I.hg = it % p.groups;
  const int r = it / p.groups;
  I.t = r % p.T;
  I.sp = r / p.T;
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
    I.ok = I.ok && pos >= 0 && pos < I.len && pos < static_cast<int64_t>(p.splits) * p.split_tiles * kRows;
    n = pos + 1;
  }
  // (a part may reach beyond 2^31 entries: lists of any stated length)
  const int64_t part = static_cast<int64_t>(p.split_tiles) * kRows, e0 = I.sp * part;
  I.e0 = static_cast<int>(min(static_cast<int64_t>(n), e0));
  I.e1 = I.ok ? static_cast<int>(min(static_cast<int64_t>(n), e0 + part)) : I.e0;
}

// Splits the 64 heads' queries of an item into hi and lo (this warp: heads w0 + 16 i) and
// stores them as the first product's operand.  A lane takes 4 neighbouring entries
// of each 128 (and lanes 0-15 4 of the last 64).  The item is the ord-th with rows; the
// first product is through with the queries of the one before.
__device__ __forceinline__ bool split_queries(const MlaQ8Params& p, Q8Smem& S, int t, int hg, uint32_t ord, int w0,
                                              int lane) {
  const uint2* src0 =
      reinterpret_cast<const uint2*>(p.q + (static_cast<int64_t>(t) * p.H + hg * kHT) * DSA_D_QK) + lane;
  const int heads = min(kHT, p.H - hg * kHT);
  auto load = [&](int hl, uint2(&v)[5]) {
    const uint2* src = src0 + hl * (DSA_D_QK / 4);
#pragma unroll
    for (int i = 0; i < 5; ++i)
      v[i] = hl < heads && (i < 4 || lane < 16) ? __ldg(src + i * 32) : make_uint2(0u, 0u);
  };
  auto split = [&](int hl, const uint2(&v)[5]) -> float {
    __nv_bfloat162 top = __habs2(as_bf16x2(v[0].x));
#pragma unroll
    for (int i = 0; i < 5; ++i)
      top = __hmax2_nan(top, __hmax2_nan(__habs2(as_bf16x2(v[i].x)), __habs2(as_bf16x2(v[i].y))));
    const uint32_t two = *reinterpret_cast<const uint32_t*>(&top) & 0x7fff7fffu;
    const uint32_t am = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
    // times 2^e: the largest entry in [2^-1, 1)
    int e = 126 - static_cast<int>(am >> 7);
    if (e > 118) e = 118;
    const float up = __uint_as_float(e >= -126 ? static_cast<uint32_t>(e + 127) << 23 : 0x00800000u >> (-126 - e));
    const bool bad = am >= 0x7f80u;                 // an infinity or NaN: the head's results are NaN
    uint8_t* lat = &S.q.lat[0][hl * 128 + ((lane >> 2) ^ (hl & 7)) * 16 + (lane & 3) * 4];
    uint8_t* rope = &S.q.rope[hl * 64 + (((lane >> 2) & 3) ^ ((hl >> 1) & 3)) * 16 + (lane & 3) * 4];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const float2 a = mul2(unpack2(v[i].x), make_float2(up, up)), b = mul2(unpack2(v[i].y), make_float2(up, up));
      uint32_t hi, lo;
      split4<true>(a.x, a.y, b.x, b.y, hi, lo);
      if (bad) hi = 0x7f7f7f7fu;
      if (i < 4) {
        *reinterpret_cast<uint32_t*>(lat + i * (kRows * 128)) = hi;
        *reinterpret_cast<uint32_t*>(lat + i * (kRows * 128) + kHT * 128) = lo;
      } else if (lane < 16) {
        *reinterpret_cast<uint32_t*>(rope) = hi;
        *reinterpret_cast<uint32_t*>(rope + kHT * 64) = lo;
      }
    }
    return __uint_as_float(static_cast<uint32_t>(119 - e) << 23);   // 2^-(e + 8)
  };
  constexpr int kPer = kHT / kSoftWarps;
  float qs = 0.f;
#pragma unroll 1
  for (int i = 0; i < kPer; i += 2) {
    uint2 w[2][5];                                  // the loads of two heads in flight
#pragma unroll
    for (int u = 0; u < 2; ++u) load(w0 + (i + u) * kSoftWarps, w[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float q = split(w0 + (i + u) * kSoftWarps, w[u]);
      if (lane == i + u) qs = q;
    }
  }
  fence_proxy_async_smem();
  // every warp is through with the last item's logits, which read its scales
  const bool ok = ord == 0 || wait(&S.l_full, (ord - 1) & 1, p.status, &S.abort);
  if (lane < kPer) S.qs[w0 + lane * kSoftWarps] = qs;
  __syncwarp();
  return ok;
}

__global__ void __launch_bounds__(kThreads, 1) mla_q8_kernel(MlaQ8Params p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Q8Smem& S = *reinterpret_cast<Q8Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  volatile int* ab = &S.abort;
  if (tid == 0) {
    S.abort = 0;
    if (smem_u32(raw) & 1023u) {
      S.abort = 1;
      set_status(p.status, DSA_DEV_INTERNAL);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.rows_full[b], 32 * kGatherWarps + kGatherWarps);
      mbar_init(&S.s_full[b], 1);
      mbar_init(&S.s_free[b], kSoftWarps);
      mbar_init(&S.plan_full[b], 1);
      mbar_init(&S.plan_free[b], kSoftWarps + kOutWarps + 2);
      for (int k = 0; k < 4; ++k) mbar_init(&S.rows_empty[b][k], 1);
    }
    for (int k = 0; k < 4; ++k) mbar_init(&S.w_full[k], kGroups);
    for (int k = 0; k < kGroups; ++k) {
      mbar_init(&S.vote[k], 4);
      mbar_init(&S.sync[k], 4);
      S.over[k][0] = S.over[k][1] = 0;
    }
    mbar_init(&S.gather_sync, kGatherWarps);
    mbar_init(&S.q_full, kSoftWarps);
    mbar_init(&S.q_free, 1);
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_free, kOutWarps);
    mbar_init(&S.l_full, kSoftWarps);
    mbar_init(&S.l_free, kOutWarps);
    mbar_init(&S.done, 2);
    fence_mbar_init();
  }
  if (warp == kSoftWarps + kGatherWarps + kOutWarps) tmem_alloc(&S.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, S.tmem, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the status word and the counter are clear
  if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine may queue up

  if (warp < kSoftWarps) {
    // ================================================================ softmax
    set_regs<kSoftRegs>();
    const int grp = warp >> 2, quad = warp & 3;     // heads 16 grp .., rows 32 quad ..
    const int r = quad * 32 + lane;
    const uint32_t s_at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kSCol + grp * kGH;
    const uint32_t o_at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kOCol + grp * kGH;
    const float c0 = p.sm_scale * 1.4426950408889634f;
    uint32_t g = 0, nq = 0, met = 0, votes = 0;     // tiles, non-empty items, meetings, votes so far
    bool bad = false;                               // a wait ran out
    int tiles = 0;                                  // of the item
    // Into the kk-th item, with its queries' operand if it has rows (of the first item
    // before its tiles are known: there is nothing to wait for).  False after the last.
    auto enter = [&](int kk) {
      Item I;
      if (kk == 0) {
        item_place(p, blockIdx.x, I);
        split_queries(p, S, I.t, I.hg, 0, warp, lane);
      }
      bad |= !wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab);
      tiles = S.plan[kk & 1];
      const int it = S.item[kk & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.plan_free[kk & 1]);
      if ((bad = __any_sync(0xffffffffu, bad)) || it < 0) return false;
      if (tiles == 0) return true;
      if (kk > 0) {
        // the products of the last item have read its queries
        bad |= nq > 0 && !wait(&S.q_free, (nq - 1) & 1, p.status, ab);
        __syncwarp();
        item_place(p, it, I);
        bad |= !split_queries(p, S, I.t, I.hg, nq, warp, lane);
      }
      if (lane == 0) mbar_arrive(&S.q_full);
      return true;
    };
    for (int kk = 0; enter(kk); ++kk) {
      float l[kGH];
#pragma unroll
      for (int i = 0; i < kGH; ++i) l[i] = 0.f;
      bool seen = false;                            // a usable row so far
      uint32_t turn = __brev(r);                    // of `dither`, a fraction of 2^32
      float far_s = 0.f;                            // see `far` below
      if (tiles > 0) {
        bad |= !wait(&S.q_full, nq & 1, p.status, ab);
        ++nq;
      }
      if (grp * kGH >= p.H) {
        // Never a head for the group: its columns of W and O are not looked at (16 heads, on
        // the device: 740 queries of a prompt 211 us, 233 without this; 64 sequences 36.9 and
        // 38.4).  With the empty groups of a second part of the heads skipped as well, 740
        // queries of 72 heads took 499 us instead of 466.
        for (int j = 0; j < tiles; ++j, ++g) {
          const int b = g & 1;
          bad |= !wait(&S.s_full[b], (g >> 1) & 1, p.status, ab);
          // (one arrival per tile: the weights of the tile before have been used)
          bad |= g > 0 && !wait(&S.rows_empty[b ^ 1][quad], ((g - 1) >> 1) & 1, p.status, ab);
          if ((bad = __any_sync(0xffffffffu, bad))) break;
          if (lane == 0) {
            mbar_arrive(&S.s_free[b]);
            mbar_arrive(&S.w_full[quad]);
          }
        }
        if (bad) break;
        if (tiles > 0 && lane == 0) mbar_arrive(&S.l_full);
        continue;
      }
      for (int j = 0; j < tiles; ++j, ++g) {
        const int b = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        bad |= !wait(&S.rows_full[b], ph, p.status, ab);
        const float s = S.s_row[b][r];
        const bool usable = s > 0.f;
        const float c = c0 * s;
        const float sg = usable ? lg2_approx(s) : -INFINITY;
        const float inv = usable ? rcp_approx(s) : 0.f;
        bad |= !wait(&S.s_full[b], ph, p.status, ab);
        if ((bad = __any_sync(0xffffffffu, bad))) break;
        tc_fence_after();
        uint32_t wh[4], wl[4];
        float x[kGH];                               // log2 of the weight, then the weight
        auto logits = [&](float add) {
          uint32_t hi[2][8], lo[2][8];
          tmem_ld8(s_at + b * 128, hi[0]);
          tmem_ld8(s_at + b * 128 + kHT, lo[0]);
          tmem_ld_wait();
          tmem_ld8(s_at + b * 128 + 8, hi[1]);
          tmem_ld8(s_at + b * 128 + kHT + 8, lo[1]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (u == 1) tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const int h = u * 8 + i;
              const float2 sc = *reinterpret_cast<const float2*>(&S.qs[grp * kGH + h]);
              const float2 mm = *reinterpret_cast<const float2*>(&S.m[grp * kGH + h]);
              const float2 d = add2(make_float2(__uint_as_float(hi[u][i]), __uint_as_float(hi[u][i + 1])),
                                    make_float2(__uint_as_float(lo[u][i]), __uint_as_float(lo[u][i + 1])));
              // an item's first logits have no reference yet
              const float2 y = ffma2(d, mul2(sc, make_float2(c, c)),
                                     seen ? add2(make_float2(add, add), mm) : make_float2(add, add));
              x[h] = y.x;
              x[h + 1] = y.y;
            }
          }
        };
        logits(sg);
        // The row's offset, in (-kStep / 2, kStep / 2) and 2^-25, half of fp16's smallest step, lower:
        // of what is then rounded to fp16 and to kStep, each to the nearest and ties up, a
        // weight w < kStep becomes 0 or kStep, the latter for w / kStep of all offsets.  Rows
        // go by the bit-reversed sequence, tiles by multiples of the golden ratio.
        const float dither = fmaf(static_cast<float>(turn >> 8), kStep / 16777216.f, -(kStep / 2 + kStep / 256));
        turn += 0x9e3779b9u;                        // 2^32 over the golden ratio
        auto weights = [&]() {
#pragma unroll
          for (int i = 0; i < kGH; ++i) x[i] = ex2_approx(x[i]);
#pragma unroll
          for (int i = 0; i < kGH; i += 4) {
            const float2 a = add2(make_float2(x[i], x[i + 1]), make_float2(dither, dither));
            const float2 b = add2(make_float2(x[i + 2], x[i + 3]), make_float2(dither, dither));
            split4<false>(a.x, a.y, b.x, b.y, wh[i / 4], wl[i / 4]);
          }
        };
        // log2 of the sum of four large weights (the largest of each 32 of the group's rows,
        // 1 to 4 times the largest of all) to within 0.75, of head 16 grp + lane mod 16;
        // not finite where the largest logit is not (or there is none).  red and m may still
        // hold the last item's sums and references.
        bool some = false;                          // (a usable row in the tile)
        auto top_sum = [&]() {
          float v[kGH];
#pragma unroll
          for (int i = 0; i < kGH; ++i) v[i] = usable ? x[i] : -INFINITY;
          const float mine = reduce_transposed<true>(v, lane);
          if (nq > 1) bad |= !wait(&S.l_free, nq & 1, p.status, ab);
          __syncwarp();
          if (lane < kGH) S.red[grp][quad][lane] = mine;
          const uint32_t s_max = __reduce_max_sync(0xffffffffu, __float_as_uint(usable ? s : 0.f));
          if (lane == 0) S.top_s[grp][quad] = s_max;
          bad |= !meet(&S.sync[grp], met, lane, p.status, ab);
          const uint32_t(&ts)[4] = S.top_s[grp];
          const float s_top = __uint_as_float(max(max(ts[0], ts[1]), max(ts[2], ts[3])));
          far_s = fmaxf(far_s, s_top * 8.673617e-19f);   // 2^-60
          some = s_top > 0.f;
          const int hl = lane & (kGH - 1);
          const float a0 = S.red[grp][0][hl], a1 = S.red[grp][1][hl], a2 = S.red[grp][2][hl], a3 = S.red[grp][3][hl];
          const float top = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
          if (!(fabsf(top) < INFINITY)) return top;
          // whole powers of two above the largest, whose weight then needs no rounding
          return top + rintf(0.25f + lg2_approx((ex2_approx(a0 - top) + ex2_approx(a1 - top)) +
                                                (ex2_approx(a2 - top) + ex2_approx(a3 - top))));
        };
        // A row whose scale lies 2^60 below that of a row which set a reference: its weight
        // may be flushed although its share of the denominator (the weight over the scale)
        // counts, so that the warp works the shares out by themselves.
        bool far = false;
        auto shares = [&]() {
#pragma unroll
          for (int i = 0; i < kGH; ++i)
            if (usable) l[i] += ex2_approx(x[i]);
        };
        bool met_now = false;                       // red and m were used: meet again when done
        if (!seen) {
          // set the reference at the first usable rows
          const float mx = top_sum();
          // without a finite logit among its rows the head is NaN
          const float up = fabsf(mx) < INFINITY ? mx - kTop : some ? kNaN : 0.f;
          if ((far = __any_sync(0xffffffffu, usable && s < far_s))) {
            logits(0.f);
#pragma unroll
            for (int i = 0; i < kGH; ++i) x[i] -= __shfl_sync(0xffffffffu, up, i);
            shares();
            logits(sg);
          }
          seen = some;
          if (quad == 0 && lane < kGH) S.m[grp * kGH + lane] = -up;
#pragma unroll
          for (int i = 0; i < kGH; ++i) x[i] -= __shfl_sync(0xffffffffu, up, i);
          weights();
          met_now = true;
          bad |= g > 0 && !wait(&S.rows_empty[b ^ 1][quad], ((g - 1) >> 1) & 1, p.status, ab);   // W_lo is free
        } else {
          float top = x[0];
#pragma unroll
          for (int i = 1; i < kGH - 1; i += 2) top = max3(top, x[i], x[i + 1]);
          top = fmaxf(top, x[kGH - 1]);
          // the group's vote on moving the reference; the weights are worked out meanwhile
          const bool over = __any_sync(0xffffffffu, top > kLimit);
          if (lane == 0) {
            if (over) S.over[grp][votes & 1] = 1;
            mbar_arrive(&S.vote[grp]);
          }
          weights();
          bad |= !wait(&S.vote[grp], votes & 1, p.status, ab);
          bad |= !wait(&S.rows_empty[b ^ 1][quad], ((g - 1) >> 1) & 1, p.status, ab);
          if ((bad = __any_sync(0xffffffffu, bad))) break;
          if (*const_cast<volatile int*>(&S.over[grp][votes & 1])) {
            // move the reference of the heads that need it, or soon may
            logits(sg);
            const float mx = top_sum();
            const float up = mx == INFINITY ? kNaN : mx > kTop ? mx - kTop : 0.f;
            // The factor may lie below fp32's range: O, relative to the new weights, is then
            // nothing, but rows of far smaller scales count in l (w / s), which takes it in halves.
            const float half = ex2_approx(-0.5f * up), f = half * half;
            // O so far: wait for the product of the tile before this one
            bad |= !wait(&S.rows_empty[b ^ 1][3], ((g - 1) >> 1) & 1, p.status, ab);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
              uint32_t o[16];
              tmem_ld16(o_at + mt * kHT, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < kGH; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, f, i));
              tmem_st16(o_at + mt * kHT, o);
            }
            tmem_st_wait();
#pragma unroll
            for (int i = 0; i < kGH; ++i) {
              const float h = __shfl_sync(0xffffffffu, half, i);
              l[i] = l[i] * h * h;
            }
            if (quad == 0) {
              if (lane < kGH) S.m[grp * kGH + lane] -= up;
              if (lane == 0) S.over[grp][votes & 1] = 0;
            }
            bad |= !meet(&S.sync[grp], met, lane, p.status, ab);   // m is set, red may be reused
            logits(sg);
            weights();
          }
          if ((far = __any_sync(0xffffffffu, usable && s < far_s))) {
            logits(0.f);
            shares();
          }
          ++votes;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.s_free[b]);
        const uint32_t at = r * 64 + ((grp ^ ((r >> 1) & 3)) << 4);
        *reinterpret_cast<uint4*>(&S.rows[b].rope[at]) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
        *reinterpret_cast<uint4*>(&S.w_lo[at]) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.w_full[quad]);
        if (!far) {
#pragma unroll
          for (int i = 0; i < kGH; i += 2) {
            const float2 y = ffma2(make_float2(x[i], x[i + 1]), make_float2(inv, inv), make_float2(l[i], l[i + 1]));
            l[i] = y.x;
            l[i + 1] = y.y;
          }
        }
        if (met_now) bad |= !meet(&S.sync[grp], met, lane, p.status, ab);   // m is set, red may be reused
      }
      if ((bad = __any_sync(0xffffffffu, bad))) break;
      if (tiles > 0) {
        // the warp's part of the denominators, for the output warps
        const float mine = reduce_transposed<false>(l, lane);
        if (nq > 1) bad |= !wait(&S.l_free, nq & 1, p.status, ab);
        __syncwarp();
        if (lane < kGH) S.red[grp][quad][lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.l_full);
      }
    }
  } else if (warp < kSoftWarps + kGatherWarps) {
    // ================================================================ rows
    set_regs<kGatherRegs>();
    const int gw = warp - kSoftWarps, gt = tid - 32 * kSoftWarps;
    uint32_t g = 0, met = 0;
    bool bad = false;                               // a wait ran out
    int next = 0;                                   // of the first thread: the next item
    for (int kk = 0, it = blockIdx.x; !bad; ++kk) {
      if (kk > 0) {
        if (gt == 0) S.drawn[kk & 1] = next;
        bad |= !meet(&S.gather_sync, met, lane, p.status, ab);
        it = S.drawn[kk & 1];
      }
      if (it >= p.items) {
        if (gt == 0) {
          bad |= kk > 1 && !wait(&S.plan_free[kk & 1], ((kk - 2) >> 1) & 1, p.status, ab);
          S.item[kk & 1] = -1;
          S.plan[kk & 1] = 0;
          mbar_arrive(&S.plan_full[kk & 1]);
        }
        break;
      }
      Item I;
      item_place(p, it, I);
      item_list(p, I);
      if (!I.ok && gt == 0) set_status(p.status, DSA_DEV_BAD_QUERY);
      int tiles = I.e1 > I.e0 ? (I.e1 - I.e0 + kRows - 1) / kRows : 0;
      const int32_t* list = p.idx ? p.idx + static_cast<int64_t>(I.t) * p.k : nullptr;
      // The warp gathers four rows of each quarter of a tile.  The lane's entries: lanes
      // 4 k + i row 32 k + 4 gw + i of the pair's first tile, lanes 16 + 4 k + i of its second.
      const int my_row = ((lane & 15) >> 2) * 32 + gw * 4 + (lane & 3);
      auto entry = [&](int pair) {
        const int e = I.e0 + (2 * pair + (lane >> 4)) * kRows + my_row;
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
      const int v_cur = entry(0);
      int v_nxt = entry(1);
      // tiles up to the last usable entry
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
        bad |= !meet(&S.gather_sync, met, lane, p.status, ab);
#pragma unroll
        for (int i = 0; i < kGatherWarps; ++i) last = max(last, S.last[i]);
        tiles = last / kRows + (last >= 0 ? 1 : 0);
        bad |= !meet(&S.gather_sync, met, lane, p.status, ab);
      }
      int row = place(v_cur, page(v_cur));
      if (gt == 0) {
        bad |= kk > 1 && !wait(&S.plan_free[kk & 1], ((kk - 2) >> 1) & 1, p.status, ab);
        S.plan[kk & 1] = tiles;
        S.item[kk & 1] = it;
        mbar_arrive(&S.plan_full[kk & 1]);
      }
      float sc = scale_of(row);
      int pg_nxt = page(v_nxt);
      // a tile's rows; the next pair's page, row and scale are looked up meanwhile
      auto gather = [&](int j) {
        if (!(sc >= 7.888609e-31f && sc <= 1.2676506e30f)) {   // 2^-100 .. 2^100
          if (row >= 0) set_status(p.status, DSA_DEV_BAD_SCALE);
          row = -1;
          sc = 0.f;
        }
        const int b = g & 1, half = j & 1;
        const uint32_t lat = smem_u32(S.rows[b].lat[0]) + (lane >> 3) * (kRows * 128);
        const uint32_t rope = smem_u32(S.rows[b].rope);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bad |= g > 1 && !wait(&S.rows_empty[b][k], ((g - 2) >> 1) & 1, p.status, ab);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = k * 32 + gw * 4 + i;
            const int src = __shfl_sync(0xffffffffu, row, half * 16 + k * 4 + i);
            cp_async16(lat + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4),
                       p.kv8 + static_cast<int64_t>(max(src, 0)) * DSA_D_QK + lane * 16, src < 0 ? 0u : 16u);
          }
          const int src = __shfl_sync(0xffffffffu, row, half * 16 + k * 4 + ((lane >> 2) & 3));
          if (lane < 16) {
            const int rr = k * 32 + gw * 4 + (lane >> 2);
            cp_async16(rope + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4),
                       p.kv8 + static_cast<int64_t>(max(src, 0)) * DSA_D_QK + DSA_D_V + (lane & 3) * 16,
                       src < 0 ? 0u : 16u);
          }
        }
        if ((lane >> 4) == half) S.s_row[b][my_row] = row < 0 ? 0.f : sc;
        cp_async_arrive_noinc(&S.rows_full[b]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.rows_full[b]);
        if (half) {
          row = place(v_nxt, pg_nxt);
          sc = scale_of(row);
          v_nxt = entry((j >> 1) + 2);
          pg_nxt = page(v_nxt);
        }
        ++g;
      };
      if (gt == 0 && tiles == 0) next = gridDim.x + atomicAdd(p.counter, 1);
      for (int j = 0; j < tiles; ++j) {
        // The next item is drawn late (a CTA at the start of a long list would take it from an
        // idle one), but early enough that its number is there when the last rows are out.
        if (gt == 0 && (j == tiles - 2 || tiles == 1)) next = gridDim.x + atomicAdd(p.counter, 1);
        gather(j);
        if ((bad = __any_sync(0xffffffffu, bad))) break;
        if (j == tiles - 1 && gw == 0) {            // its queries on their way to L2
          const int n = __shfl_sync(0xffffffffu, next, 0);
          if (n < p.items) {
            Item N;
            item_place(p, n, N);
            const int lines = min(kHT, p.H - N.hg * kHT) * (DSA_D_QK * 2 / 128);
            const char* src =
                reinterpret_cast<const char*>(p.q + (static_cast<int64_t>(N.t) * p.H + N.hg * kHT) * DSA_D_QK);
            for (int i = lane; i < lines; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i * 128));
          }
        }
      }
      bad = __any_sync(0xffffffffu, bad);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kSoftWarps + kGatherWarps + kOutWarps) {
    // ================================================================ output
    set_regs<kOutRegs>();
    const int quad = warp & 3;                      // TMEM lanes 32 quad ..
    const int r = quad * 32 + lane;
    const uint32_t o_at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kOCol;
    uint32_t nq = 0;
    bool bad = false;
    for (int kk = 0;; ++kk) {
      bad |= !wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab);
      const bool any = S.plan[kk & 1] > 0;
      const int it = S.item[kk & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.plan_free[kk & 1]);
      if ((bad = __any_sync(0xffffffffu, bad)) || it < 0) break;
      Item I;
      item_place(p, it, I);
      const int h0 = I.hg * kHT;
      const int64_t row = p.splits == 1 ? static_cast<int64_t>(I.t) * p.H
                                        : (static_cast<int64_t>(I.t) * p.splits + I.sp) * p.H;
      float inv[2];                                 // of heads lane and 32 + lane
      if (any) bad |= !wait(&S.l_full, nq & 1, p.status, ab);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = 32 * u + lane;
        float total = 0.f;
        if (any) {
          const float(&part)[4][kGH] = S.red[h / kGH];
          const int i = h % kGH;
          total = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
        }
        inv[u] = total == 0.f ? 0.f : 0.00390625f / total;       // O holds 2^8 times the weights
        if (quad == 0 && h0 + h < p.H) {
          const float lse = total == 0.f ? -INFINITY : (log2f(total) - S.m[h]) * 0.6931471805599453f;
          if (p.splits > 1)
            p.part_lse[row + h0 + h] = lse;
          else if (p.lse)
            p.lse[row + h0 + h] = lse;
        }
      }
      if (any) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.l_free);
        bad |= !wait(&S.o_full, nq & 1, p.status, ab);
        ++nq;
      }
      if ((bad = __any_sync(0xffffffffu, bad))) break;
      if (!any && p.splits > 1) continue;           // the combine skips parts of weight 0
      tc_fence_after();
      // Lanes hold neighbouring dims of every head.  For bf16 a pair of lanes trades, so that
      // the even one has two dims of an even head and the odd one two dims of the odd head
      // after it.  The next columns are read from TMEM meanwhile.
      const int odd = lane & 1;
      const uint32_t sel = odd ? 0x3276u : 0x5410u;
      float* part = p.part_o + row * DSA_D_V + h0 * DSA_D_V + r;
      uint16_t* out = p.out + (row + h0 + odd) * DSA_D_V + r - odd;
      uint32_t o[2][8];
      if (any) {
        tmem_ld8(o_at, o[0]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[0][i] = o[1][i] = 0;
      }
      const int heads = min(kHT, p.H - h0);         // a multiple of 8
#pragma unroll 1
      for (int hc = 0; hc < heads; hc += 8) {       // 8 heads, then the four groups of 128 dims
        float iv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) iv[i] = __shfl_sync(0xffffffffu, hc < 32 ? inv[0] : inv[1], (hc + i) & 31);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          if (any) {
            tmem_ld_wait();
            if (mt < 3) {
              tmem_ld8(o_at + hc + (mt + 1) * kHT, o[(mt + 1) & 1]);
            } else if (hc + 8 < heads) {
              tmem_ld8(o_at + hc + 8, o[0]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&S.o_free);
            }
          }
          float2 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = mul2(make_float2(__uint_as_float(o[mt & 1][2 * i]), __uint_as_float(o[mt & 1][2 * i + 1])),
                        make_float2(iv[2 * i], iv[2 * i + 1]));
          if (p.splits > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              part[(hc + 2 * i) * DSA_D_V + mt * 128] = y[i].x;
              part[(hc + 2 * i + 1) * DSA_D_V + mt * 128] = y[i].y;
            }
          } else {
            uint32_t z[4], got[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 z2 = __floats2bfloat162_rn(y[i].x, y[i].y);
              z[i] = *reinterpret_cast<const uint32_t*>(&z2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) got[i] = __shfl_xor_sync(0xffffffffu, z[i], 1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint32_t*>(out + (hc + 2 * i) * DSA_D_V + mt * 128) = __byte_perm(z[i], got[i], sel);
          }
        }
      }
    }
  } else {
    set_regs<kIssueRegs>();
    constexpr uint32_t kChunk = kRows * 128 / 16;   // a tile's 128-dim chunk, in descriptor units
    constexpr uint32_t kTile = sizeof(Tile) / 16;
    static_assert(offsetof(Q8Smem, rows) == sizeof(Tile) && offsetof(Q8Smem, w_lo) == 3 * sizeof(Tile), "");
    const uint32_t q0 = __shfl_sync(0xffffffffu, desc_lo(S.q.lat[0]), 0);   // then the row tiles, then W_lo
    uint32_t g = 0, n = 0;                          // tiles, items with rows so far
    bool ok = true;
    if (warp == kSoftWarps + kGatherWarps + kOutWarps) {
      // ================================================================ S^T = codes . Q^T
      constexpr uint32_t id = instr_desc(0, 0, false, false, 128, 2 * kHT);
      for (int kk = 0; ok; ++kk) {
        ok = wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab);
        const int tiles = __shfl_sync(0xffffffffu, S.plan[kk & 1], 0), it = S.item[kk & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.plan_free[kk & 1]);
        if (tiles > 0) ok = ok && wait(&S.q_full, n & 1, p.status, ab);
        if (!(ok = __all_sync(0xffffffffu, ok && it >= 0))) break;
        if (tiles == 0) continue;
        ++n;
        for (int j = 0; j < tiles; ++j, ++g) {
          const uint32_t b = g & 1, ph = (g >> 1) & 1;
          ok = (g <= 1 || wait(&S.s_free[b], ph ^ 1, p.status, ab)) && wait(&S.rows_full[b], ph, p.status, ab);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          const uint32_t a = q0 + kTile + b * kTile, d = tmem + kSCol + b * 128;
          if (elect_one_sync()) {
            fence_proxy_async_smem();               // cp.async writes -> tensor-core reads
            tc_fence_after();
#pragma unroll
            for (uint32_t c = 0; c < 4 * kChunk; c += kChunk)
#pragma unroll
              for (uint32_t s = 0; s < 8; s += 2) mma<kDesc128, kDesc128>(d, a + c + s, q0 + c + s, id, (c | s) != 0);
#pragma unroll
            for (uint32_t s = 0; s < 4; s += 2)
              mma<kDesc64, kDesc64>(d, a + 4 * kChunk + s, q0 + 4 * kChunk + s, id, true);
            umma_commit(&S.s_full[b]);
            if (j == tiles - 1) umma_commit(&S.q_free);
          }
          __syncwarp();
        }
      }
      if (elect_one_sync()) {
        umma_commit(&S.done);
        mbar_wait(&S.done, 0, p.status, nullptr);
      }
    } else if (warp == kSoftWarps + kGatherWarps + kOutWarps + 1) {
      // ================================================================ O^T += codes^T . W
      constexpr uint32_t id = instr_desc(0, 0, true, true, 128, kHT);
      for (int kk = 0; ok; ++kk) {
        ok = wait(&S.plan_full[kk & 1], (kk >> 1) & 1, p.status, ab);
        const int tiles = __shfl_sync(0xffffffffu, S.plan[kk & 1], 0), it = S.item[kk & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.plan_free[kk & 1]);
        if (tiles > 0 && n > 0) ok = ok && wait(&S.o_free, (n - 1) & 1, p.status, ab);
        if (!(ok = __all_sync(0xffffffffu, ok && it >= 0))) break;
        if (tiles == 0) continue;
        ++n;
        for (int j = 0; j < tiles && ok; ++j, ++g) {
          const uint32_t b = g & 1;
          const uint32_t a = q0 + kTile + b * kTile;
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            if (!(ok = __all_sync(0xffffffffu, ok && wait(&S.w_full[k], g & 1, p.status, ab)))) break;
            if (elect_one_sync()) {
              tc_fence_after();
              const uint32_t wk = k * (32 * 64 / 16);
#pragma unroll
              for (uint32_t mt = 0; mt < 4; ++mt) {
                const uint32_t am = a + mt * kChunk + k * (32 * 128 / 16);
                mma<kDesc128, kDesc64>(tmem + kOCol + mt * kHT, am, q0 + 3 * kTile + wk, id, j > 0 || k > 0);
                mma<kDesc128, kDesc64>(tmem + kOCol + mt * kHT, am, a + 4 * kChunk + wk, id, true);
              }
              umma_commit(&S.rows_empty[b][k]);
              if (k == 3 && j == tiles - 1) umma_commit(&S.o_full);
            }
            __syncwarp();
          }
        }
      }
      if (elect_one_sync()) {
        umma_commit(&S.done);
        mbar_wait(&S.done, 0, p.status, nullptr);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kGatherWarps + kOutWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Clears the status word and the item counter, and lets the attention in meanwhile.
__global__ void clear_kernel(uint32_t* status, int32_t* counter) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  *status = 0;
  *counter = 0;
}

// Four floats, or zeros where `take` is false (a predicated load: the loads of a loop go
// out together, which those behind branches do not).
__device__ __forceinline__ float4 load_if(const float* at, bool take) {
  float4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\tmov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
      "@p ld.global.v4.f32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w)
      : "l"(at), "r"(static_cast<uint32_t>(take))
      : "memory");
  return v;
}

// Joins the parts of a split row list: lse = log sum exp(lse_i), out = sum exp(lse_i - lse) o_i.
// A CTA per query and head, four dims per thread.  Every warp works the weights out for
// itself (lane i: parts i and 32 + i).  Parts of weight 0 may never have been written.
// With few CTAs (kEager) latency counts: 16 parts are read while the weights are worked
// out, whatever those turn out to be (one query of 16 parts 18.7 us on the device with the
// attention, against 20.7 the other way).  With many, only parts with a weight are read,
// eight at a time (24 ragged contexts of 128 heads 60.7 us against 66.2).
template <bool kEager>
__global__ void __launch_bounds__(128) combine_kernel(MlaQ8Params p) {
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int64_t at = static_cast<int64_t>(t) * p.splits * p.H + h;
  constexpr int kBatch = kEager ? 16 : 8;
  float4 o[kBatch];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      o[i] = *reinterpret_cast<const float4*>(
          p.part_o + (at + static_cast<int64_t>(min(s0 + i, p.splits - 1)) * p.H) * DSA_D_V + tid * 4);
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts are complete
  if (kEager) load(0);
  float v[2], mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
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
  const float wgt[2] = {den == 0.f ? 0.f : e[0] / den, den == 0.f ? 0.f : e[1] / den};
  const float lse = den == 0.f ? -INFINITY : mx + logf(den);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < p.splits; s0 += kBatch) {
    float w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w[i] = __shfl_sync(0xffffffffu, s0 < 32 ? wgt[0] : wgt[1], (s0 + i) & 31);
    if (!kEager) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        o[i] = load_if(p.part_o + (at + static_cast<int64_t>(s0 + i) * p.H) * DSA_D_V + tid * 4,
                       s0 + i < p.splits && w[i] != 0.f);   // with a NaN among the parts every weight is NaN
    } else if (s0 > 0) {
      load(s0);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (kEager && w[i] == 0.f) continue;
      acc.x = fmaf(w[i], o[i].x, acc.x);
      acc.y = fmaf(w[i], o[i].y, acc.y);
      acc.z = fmaf(w[i], o[i].z, acc.z);
      acc.w = fmaf(w[i], o[i].w, acc.w);
    }
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * p.H + h) * DSA_D_V + tid * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (tid == 0 && p.lse) p.lse[static_cast<int64_t>(t) * p.H + h] = lse;
}

}  // namespace

// Once per device: the kernel's shared memory, and that it was built at the register
// count that its split adds up to (with fewer, an increase would never be granted).
static cudaError_t prepare_device(size_t smem) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(mla_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, mla_q8_kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  ready.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

// Splits of the row lists: with few queries a list is cut so that its parts fill the
// SMs.  `most` and `mean` are the longest list and the mean one.  An item costs about
// three tiles' time beside its tiles (the first row latencies, the first reference,
// the output).  Where the items go round once, the time is that of one item;
// otherwise that of an even share, and one item at the end: 24 contexts of 1 .. 8191
// rows, dense, took 60 us in the parts of 12 tiles chosen here and 68 us in parts of 20
// that go round once.  Lists of 16 tiles that go round more than once are left whole:
// 75 queries of 128 heads 95 us, in halves 98; 149 queries 140 us, in halves 163.
int mla_q8_plan(int T, int H, int64_t most, int64_t mean, int sms, int* split_tiles) {
  const int64_t base = static_cast<int64_t>(T) * ((H + kHT - 1) / kHT);
  const int64_t tiles = most > 0 ? (most + kRows - 1) / kRows : 1;
  const int64_t mean_tiles = mean > 0 ? (mean + kRows - 1) / kRows : 1;
  int64_t best = tiles, best_cost = -1;
  for (int64_t s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    const int64_t per = (tiles + s - 1) / s;
    // parts of lists of one length, or of ragged ones (half a part more per list)
    const int64_t items =
        mean_tiles == tiles ? base * ((tiles + per - 1) / per)
                            : (base * (2 * mean_tiles + per) + 2 * per - 1) / (2 * per);
    const int64_t cost = items <= sms ? per + 3 : (base * mean_tiles + 3 * items + sms - 1) / sms + (s > 1 ? per : 3);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = per;
    }
  }
  *split_tiles = static_cast<int>(best);
  return static_cast<int>((tiles + best - 1) / best);
}

cudaError_t launch_sparse_mla_q8(const MlaQ8Params& params, bool clear, int sms, cudaStream_t stream) {
  MlaQ8Params p = params;
  if (p.T == 0) return clear ? cudaMemsetAsync(p.status, 0, 2 * sizeof(uint32_t), stream) : cudaSuccess;
  const size_t smem = sizeof(Q8Smem);
  cudaError_t e = prepare_device(smem);
  if (e != cudaSuccess) return e;
  p.groups = (p.H + kHT - 1) / kHT;
  const int64_t items = static_cast<int64_t>(p.T) * p.splits * p.groups;
  if (items > 0x7fffffff - sms) return cudaErrorInvalidConfiguration;
  p.items = static_cast<int>(items);
  if (clear) {
    clear_kernel<<<1, 1, 0, stream>>>(p.status, p.counter);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launches(1);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.items < sms ? p.items : sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = clear ? 1 : 0;
  if ((e = cudaLaunchKernelEx(&cfg, mla_q8_kernel, p)) != cudaSuccess) return e;
  count_launches(1);
  if (p.splits == 1) return e;
  cfg.gridDim = dim3(p.T, p.H);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, static_cast<int64_t>(p.T) * p.H <= 8 * sms ? combine_kernel<true> : combine_kernel<false>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dsa
