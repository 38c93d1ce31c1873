// The small kernels around the backward pass: row statistics, the tile
// ranges of dense masks, and the relative position bias's expansion by
// distance and reduction to buckets. Each reads its inputs once and is bound
// by memory or, at small sizes, by its launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_bwd.h"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]));
    const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&y[i]));
    s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
  }
  return s;
}

// One CTA per query tile, D / 8 threads per row (16-byte loads, whole rows
// per group of threads): delta_i = sum_d do_id o_id.
template <int D>
__global__ void __launch_bounds__(256) bwd_stats(const __grid_constant__ BwdParams p) {
  constexpr int L = D / 8;            // threads per row
  constexpr int R = 256 / L;          // rows per pass
  const BwdItem it = p.q_items[blockIdx.x];
  const SeqRec s = p.seqs[it.b];
  const int sl = threadIdx.x % L;
  const int64_t base = it.b * p.q_sb + it.h * p.q_sh;
  float* out = p.stats + (int64_t)it.stat * 256;
#pragma unroll
  for (int r0 = 0; r0 < kTileM; r0 += R) {
    const int r = r0 + threadIdx.x / L;
    const int64_t i = (int64_t)it.tile * kTileM + r;
    const bool stored = i < s.sq;
    float d = 0.f;
    if (stored) {
      const int64_t off = base + (s.q_off + i) * p.q_st + sl * 8;
      d = dot8(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.o) + off)),
               __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.d_o) + off)));
    }
#pragma unroll
    for (int x = 1; x < L; x <<= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    if (sl == 0) {
      float nl = -INFINITY, nd = 0.f;
      if (stored) {
        const int64_t at = it.b * p.l_sb + it.h * p.l_sh + s.q_off + i;
        float l = p.lse[at];
        if (l != -INFINITY) {
          // Left-aligned ALiBi: the same weights as the right-aligned bias,
          // which the kernels add, with every score of the row shifted.
          if (p.alibi == FA_ALIBI_LEFT)
            l = fmaf(-p.slopes[it.h], (float)(i + (int64_t)s.skv - s.sq), l);
          nl = -l * kLog2e;
          nd = (p.d_lse ? p.d_lse[at] : 0.f) - d;
        }
      }
      out[r] = nl;
      out[kTileM + r] = nd;
    }
  }
}

// Dense masks: thread n < n_q copies query item n's range, the warps after
// them reduce one key item each: [lo, hi) from the first to the last query
// tile with a visible pair, and the longest run of fully visible ones (the
// first on ties). A FULL class covers 128 stored keys.
__global__ void __launch_bounds__(256) bwd_ranges(BwdOccParams a, int q_blocks) {
  if ((int)blockIdx.x < q_blocks) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.n_q) return;
    BwdItem it = a.q_items[n];
    const TileRange r = a.ranges[(it.b * a.occ_sb + it.h * a.occ_sh) * a.n_qt + it.tile];
    it.lo = r.lo, it.hi = r.hi, it.full_lo = r.full_lo, it.full_hi = r.full_hi;
    a.q_items[n] = it;
    return;
  }
  const int lane = threadIdx.x & 31;
  const int n = (blockIdx.x - q_blocks) * 8 + (threadIdx.x >> 5);
  if (n >= a.n_k) return;
  BwdItem it = a.k_items[n];
  const uint8_t* cls = a.cls + (it.b * a.occ_sb + it.h * a.occ_sh) * a.n_qt * (int64_t)a.n_kt + it.tile;
  int lo = 0x7fffffff, hi = 0;
  int best = 0, best_at = 0, run = 0;  // the same in every lane
  for (int t0 = 0; t0 < a.n_qt; t0 += 32) {
    const int t = t0 + lane;
    const int c = t < a.n_qt ? cls[(int64_t)t * a.n_kt] : 0;
    const uint32_t any = __ballot_sync(0xffffffffu, c != FA_TILE_EMPTY);
    const uint32_t full = __ballot_sync(0xffffffffu, c == FA_TILE_FULL);
    if (any) {
      lo = min(lo, t0 + __ffs(any) - 1);
      hi = t0 + 32 - __clz(any);
    }
    for (int x = 0; x < 32; ++x) {
      run = (full >> x) & 1u ? run + 1 : 0;
      if (run > best) {
        best = run;
        best_at = t0 + x + 1 - run;
      }
    }
  }
  if (lane != 0) return;
  it.lo = hi > 0 ? lo : 0;
  it.hi = hi;
  it.full_lo = best > 0 ? best_at : it.lo;
  it.full_hi = best > 0 ? best_at + best : it.lo;
  a.k_items[n] = it;
}

__global__ void __launch_bounds__(256) rel_expand(const float* __restrict__ table,
                                                  const int32_t* __restrict__ bucket_of,
                                                  float* __restrict__ ext, int N, int num_buckets,
                                                  int reach, int row) {
  const int h = blockIdx.y;
  const int x = blockIdx.x * 256 + threadIdx.x;
  if (x >= row) return;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int rel = min(max(x + s - reach - kRelPad, -reach), reach);
    ext[((int64_t)h * 4 + s) * row + x] = table[(int64_t)bucket_of[rel + reach] * N + h] * kLog2e;
  }
}

// First step: dist[h][e] = sum over head h's query tiles, in 64 bits. One CTA
// per head and 32 distances; warp w adds tiles w, w + 8, ... and the eight
// sums are added in warp order.
__global__ void __launch_bounds__(256) rel_sum_tiles(const float* __restrict__ part,
                                                     double* __restrict__ dist, int tiles, int W) {
  __shared__ double sm[8][32];
  const int h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (d < W)
    for (int t = w; t < tiles; t += 8) s += part[((int64_t)h * tiles + t) * W + d];
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && d < W) {
    double a = sm[0][lane];
    for (int x = 1; x < 8; ++x) a += sm[x][lane];
    dist[(int64_t)h * W + d] = a;
  }
}

// Second step: one warp per (bucket, head) adds the distances of its bucket,
// those past the reach with the end they clip to.
__global__ void __launch_bounds__(256) rel_sum_buckets(const double* __restrict__ dist,
                                                       const int32_t* __restrict__ bucket_of,
                                                       float* __restrict__ dtable, int N, int W,
                                                       int reach, int num_buckets) {
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (n >= (int64_t)num_buckets * N) return;
  const int c = (int)(n / N), h = (int)(n % N);
  double s = 0.0;
  for (int e = lane; e < W; e += 32)
    if (bucket_of[min(max(e - kRelPad, 0), 2 * reach)] == c) s += dist[(int64_t)h * W + e];
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  if (lane == 0) dtable[n] = (float)s;
}

}  // namespace

cudaError_t launch_bwd_stats(int D, const BwdParams& p, cudaStream_t stream) {
  if (p.n_q <= 0) return cudaSuccess;
  if (D == 128) bwd_stats<128><<<p.n_q, 256, 0, stream>>>(p);
  else bwd_stats<64><<<p.n_q, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_bwd_ranges(const BwdOccParams& a, cudaStream_t stream) {
  const int qb = (a.n_q + 255) / 256, kb = (a.n_k + 7) / 8;
  if (qb + kb > 0) bwd_ranges<<<qb + kb, 256, 0, stream>>>(a, qb);
  return cudaGetLastError();
}

cudaError_t launch_rel_expand(const float* table, const int32_t* bucket_of, float* ext, int32_t N,
                              int32_t num_buckets, int32_t reach, cudaStream_t stream) {
  const int row = rel_row(reach);
  rel_expand<<<dim3((row + 255) / 256, N), 256, 0, stream>>>(table, bucket_of, ext, N, num_buckets,
                                                             reach, row);
  return cudaGetLastError();
}

cudaError_t launch_rel_reduce(const float* rel_part, double* dist, const int32_t* bucket_of,
                              float* dtable, int32_t N, int32_t tiles, int32_t num_buckets,
                              int32_t reach, cudaStream_t stream) {
  const int W = rel_width(reach);
  rel_sum_tiles<<<dim3((W + 31) / 32, N), 256, 0, stream>>>(rel_part, dist, tiles, W);
  rel_sum_buckets<<<(int)(((int64_t)num_buckets * N + 7) / 8), 256, 0, stream>>>(
      dist, bucket_of, dtable, N, W, reach, num_buckets);
  return cudaGetLastError();
}

}  // namespace fa
