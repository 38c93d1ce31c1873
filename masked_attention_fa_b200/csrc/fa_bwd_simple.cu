// Backward pass in its simplest form: one warp per query row for dQ and the
// bias's gradient, one warp per key for dK and dV, fp32 on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_bwd.h"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <int D>
struct Row {
  float v[D / 32];
  __device__ __forceinline__ void load(const void* base, int64_t off) {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(base) + off;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) v[x] = __bfloat162float(p[x * 32 + (threadIdx.x & 31)]);
  }
  __device__ __forceinline__ float dot(const Row& o) const {
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) s = fmaf(v[x], o.v[x], s);
    return warp_sum(s);
  }
  __device__ __forceinline__ void add(float w, const Row& o) {
#pragma unroll
    for (int x = 0; x < D / 32; ++x) v[x] = fmaf(w, o.v[x], v[x]);
  }
  __device__ __forceinline__ void store(void* base, int64_t off, float mul) const {
    __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(base) + off;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      p[x * 32 + (threadIdx.x & 31)] = __float2bfloat16_rn(v[x] * mul);
  }
};

__device__ __forceinline__ bool visible(const BwdParams& p, const SeqRec& s, int b, int h,
                                        int64_t i, int64_t j) {
  if (j < row_lo(s, i) || j > row_hi(s, i)) return false;
  return !(s.flags & kSeqDenseMask) || p.mask[b * p.m_sb + h * p.m_sh + i * p.m_si + j] == 0;
}

// Bias of a pair in log2 units.
__device__ __forceinline__ float bias2(const BwdParams& p, int h, int64_t rel) {
  if (p.rel.ext) {
    const int64_t r = imax64(-p.rel.reach, imin64(p.rel.reach, rel));
    return p.rel.ext[(int64_t)h * 4 * p.rel.row + r + p.rel.reach + kRelPad];
  }
  if (!p.slopes) return 0.f;
  const float a = p.slopes[h] * kLog2e;
  const float d = (float)rel;
  return p.alibi == FA_ALIBI_SQRT ? a * copysignf(sqrtf(fabsf(d)), d) : a * d;
}

template <int D>
__global__ void __launch_bounds__(128) bwd_dq_simple(const __grid_constant__ BwdParams p) {
  const BwdItem it = p.q_items[blockIdx.x];
  const SeqRec s = p.seqs[it.b];
  const int64_t bq = it.b * p.q_sb + it.h * p.q_sh, bk = it.b * p.k_sb + it.h * p.k_sh;
  const int W = 2 * p.rel.reach + 1;
  float* part = p.rel_part ? p.rel_part + (int64_t)it.stat * W : nullptr;
  if (part)
    for (int x = threadIdx.x; x < W; x += blockDim.x) part[x] = 0.f;
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < kTileM; r += blockDim.x >> 5) {
    const int64_t i = (int64_t)it.tile * kTileM + r;
    if (i >= s.sq) break;
    Row<D> q, g, acc;
    q.load(p.q, bq + (s.q_off + i) * p.q_st);
    g.load(p.d_o, bq + (s.q_off + i) * p.q_st);
    acc.load(p.q, bq + (s.q_off + i) * p.q_st);
    for (int x = 0; x < D / 32; ++x) acc.v[x] = 0.f;
    const float nl = p.stats[(int64_t)it.stat * 256 + r];
    const float nd = p.stats[(int64_t)it.stat * 256 + 128 + r];
    for (int64_t j = imax64(0, row_lo(s, i)); j <= imin64(s.skv - 1, row_hi(s, i)); ++j) {
      if (!visible(p, s, it.b, it.h, i, j)) continue;
      Row<D> k, v;
      k.load(p.k, bk + (s.kv_off + j) * p.k_st);
      v.load(p.v, bk + (s.kv_off + j) * p.k_st);
      const int64_t rel = j - (i + s.skv - s.sq);
      const float w = exp2f(q.dot(k) * p.scale_log2 + bias2(p, it.h, rel) + nl);
      const float ds = w * (g.dot(v) + nd);
      acc.add(ds, k);
      if (part && (threadIdx.x & 31) == 0)
        part[imax64(-p.rel.reach, imin64(p.rel.reach, rel)) + p.rel.reach] += ds;
    }
    acc.store(p.dq, bq + (s.q_off + i) * p.q_st, p.scale);
  }
}

template <int D>
__global__ void __launch_bounds__(128) bwd_dkv_simple(const __grid_constant__ BwdParams p) {
  const BwdItem it = p.k_items[blockIdx.x];
  const SeqRec s = p.seqs[it.b];
  const int64_t bq = it.b * p.q_sb + it.h * p.q_sh, bk = it.b * p.k_sb + it.h * p.k_sh;
  for (int r = threadIdx.x >> 5; r < kTileN; r += 4) {
    const int64_t j = (int64_t)it.tile * kTileN + r;
    if (j >= s.skv) break;
    Row<D> k, v, dk, dv;
    k.load(p.k, bk + (s.kv_off + j) * p.k_st);
    v.load(p.v, bk + (s.kv_off + j) * p.k_st);
    for (int x = 0; x < D / 32; ++x) dk.v[x] = dv.v[x] = 0.f;
    for (int64_t i = (int64_t)it.lo * kTileM; i < imin64(s.sq, (int64_t)it.hi * kTileM); ++i) {
      if (!visible(p, s, it.b, it.h, i, j)) continue;
      Row<D> q, g;
      q.load(p.q, bq + (s.q_off + i) * p.q_st);
      g.load(p.d_o, bq + (s.q_off + i) * p.q_st);
      const float* st = p.stats + ((int64_t)it.stat + i / kTileM) * 256 + i % kTileM;
      const float w = exp2f(q.dot(k) * p.scale_log2 + bias2(p, it.h, j - (i + s.skv - s.sq)) + st[0]);
      dv.add(w, g);
      dk.add(w * (g.dot(v) + st[128]), q);
    }
    dk.store(p.dk, bk + (s.kv_off + j) * p.k_st, p.scale);
    dv.store(p.dv, bk + (s.kv_off + j) * p.k_st, 1.f);
  }
}

template <int D>
cudaError_t launch_d(const BwdParams& p, cudaStream_t stream) {
  if (p.n_q > 0) bwd_dq_simple<D><<<p.n_q, p.rel_part ? 32 : 128, 0, stream>>>(p);  // bias sums: one warp, one order
  if (p.n_k > 0) bwd_dkv_simple<D><<<p.n_k, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd(int D, const BwdParams& p, int, cudaStream_t stream, const char**) {
  return D == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace fa
