// Sparse (or dense) MLA over the 8-bit latent cache on sm_100a.
//
// For query t, head h and usable rows i with value c_i = scale_i * code_i:
//   z_i = sm_scale q.c_i, p = softmax(z), out = sum_i p_i c_i[:512], lse = log sum exp z
//
// First form, CUDA cores: one CTA (256 threads) per (query, 8 heads); rows are
// decoded to fp32 in shared memory in tiles of 32, one thread per (head, row)
// logit, a running maximum and sum per head, two output dims x 8 heads per thread.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 8;
constexpr int kRows = 32;
constexpr int kStride = DSA_D_QK + 1;

struct Smem {
  float q[kHeads][kStride];
  float rows[kRows][kStride];
  float p[kHeads][kRows];
  float m[kHeads], l[kHeads], fix[kHeads];
  int64_t row[kRows];
  float scale[kRows];
};

__global__ void __launch_bounds__(kThreads) mla_q8_simple_kernel(MlaQ8Params p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& S = *reinterpret_cast<Smem*>(raw);
  const int t = blockIdx.x, h0 = blockIdx.y * kHeads, tid = threadIdx.x;
  const int seq = p.q_seq[t];
  const bool seq_ok = seq >= 0 && seq < p.num_seqs;
  const int len = seq_ok ? p.kv_len[seq] : 0;
  const int64_t base = seq_ok && p.page_size == 0 ? p.kv_offset[seq] : 0;
  bool ok = seq_ok && len >= 0 &&
            (p.page_size == 0 ? base >= 0 && base + len <= p.kv_rows
                              : len <= static_cast<int64_t>(p.pages_per_seq) * p.page_size);
  const int pos = p.q_pos[t];
  if (!p.idx) ok = ok && pos >= 0 && pos < len;
  if (!ok && tid == 0) set_status(p.status, DSA_DEV_BAD_QUERY);
  for (int i = tid; i < kHeads * DSA_D_QK; i += kThreads) {
    const int h = i / DSA_D_QK, d = i % DSA_D_QK;
    S.q[h][d] = __uint_as_float(static_cast<uint32_t>(p.q[(static_cast<int64_t>(t) * p.H + h0 + h) * DSA_D_QK + d])
                                << 16);
  }
  if (tid < kHeads) {
    S.m[tid] = -INFINITY;
    S.l[tid] = 0.f;
  }
  float o[kHeads][2] = {};
  const int n = !ok ? 0 : (p.idx ? p.k : pos + 1);
  for (int e0 = 0; e0 < n; e0 += kRows) {
    if (tid < kRows) {
      const int e = e0 + tid;
      int v = -1;
      if (e < n) v = p.idx ? p.idx[static_cast<int64_t>(t) * p.k + e] : e;
      int64_t r = -1;
      float s = 0.f;
      if (v >= len) set_status(p.status, DSA_DEV_BAD_INDEX);
      if (v >= 0 && v < len) {
        r = base + v;
        if (p.page_size) {
          const int pg = p.page_table[static_cast<int64_t>(seq) * p.pages_per_seq + v / p.page_size];
          r = static_cast<int64_t>(pg) * p.page_size + v % p.page_size;
          if (pg < 0 || r >= p.kv_rows) {
            set_status(p.status, DSA_DEV_BAD_INDEX);
            r = -1;
          }
        }
        if (r >= 0) {
          s = p.scale[r >> p.block_log2];
          if (!(s >= 7.888609e-31f && s <= 1.2676506e30f)) {
            set_status(p.status, DSA_DEV_BAD_SCALE);
            r = -1;
          }
        }
      }
      S.row[tid] = r;
      S.scale[tid] = s;
    }
    __syncthreads();
    for (int i = tid; i < kRows * DSA_D_QK; i += kThreads) {
      const int r = i / DSA_D_QK, d = i % DSA_D_QK;
      float x = 0.f;
      if (S.row[r] >= 0)
        x = __half2float(__half(__nv_cvt_fp8_to_halfraw(p.kv8[S.row[r] * DSA_D_QK + d], __NV_E4M3))) * S.scale[r];
      S.rows[r][d] = x;
    }
    __syncthreads();
    const int h = tid / kRows, r = tid % kRows;
    float z = -INFINITY;
    if (S.row[r] >= 0) {
      z = 0.f;
      for (int d = 0; d < DSA_D_QK; ++d) z = fmaf(S.q[h][d], S.rows[r][d], z);
      z *= p.sm_scale;
    }
    float mt = z;
    for (int x = 16; x; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
    const float m_old = S.m[h], m = fmaxf(m_old, mt);
    const float pv = S.row[r] >= 0 ? expf(z - (m == -INFINITY ? 0.f : m)) : 0.f;
    float sum = pv;
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    S.p[h][r] = pv;
    __syncwarp();
    if (r == 0) {
      const float fix = m_old == -INFINITY ? 0.f : expf(m_old - m);
      S.fix[h] = fix;
      S.m[h] = m;
      S.l[h] = S.l[h] * fix + sum;
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < kHeads; ++a) {
      o[a][0] *= S.fix[a];
      o[a][1] *= S.fix[a];
      for (int x = 0; x < kRows; ++x) {
        o[a][0] = fmaf(S.p[a][x], S.rows[x][tid], o[a][0]);
        o[a][1] = fmaf(S.p[a][x], S.rows[x][tid + 256], o[a][1]);
      }
    }
    __syncthreads();
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < kHeads; ++a) {
    const float inv = S.l[a] == 0.f ? 0.f : 1.f / S.l[a];
    uint16_t* dst = p.out + (static_cast<int64_t>(t) * p.H + h0 + a) * DSA_D_V;
    dst[tid] = __bfloat16_as_ushort(__float2bfloat16_rn(o[a][0] * inv));
    dst[tid + 256] = __bfloat16_as_ushort(__float2bfloat16_rn(o[a][1] * inv));
  }
  if (p.lse && tid < kHeads)
    p.lse[static_cast<int64_t>(t) * p.H + h0 + tid] = S.l[tid] == 0.f ? -INFINITY : S.m[tid] + logf(S.l[tid]);
}

}  // namespace

cudaError_t launch_sparse_mla_q8(const MlaQ8Params& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(mla_q8_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(Smem)));
  if (e != cudaSuccess) return e;
  mla_q8_simple_kernel<<<dim3(p.T, p.H / kHeads), kThreads, sizeof(Smem), stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dsa
