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

// Entries [256 chunk, 256 chunk + 256) of the four copies of head h.
__device__ __forceinline__ void expand_chunk(const RelTable& t, int h, int chunk) {
  const int row = rel_row(t.reach);
  const int x = chunk * 256 + threadIdx.x;
  if (x >= row) return;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int rel = min(max(x + s - t.reach - kRelPad, -t.reach), t.reach);
    t.ext[((int64_t)h * 4 + s) * row + x] =
        t.table[(int64_t)t.bucket_of[rel + t.reach] * t.N + h] * kLog2e;
  }
}

__global__ void __launch_bounds__(256) rel_expand(RelTable t, unsigned int* zero, int64_t n_zero) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t first = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  for (int64_t x = first; x < n_zero; x += (int64_t)gridDim.x * gridDim.y * 256) zero[x] = 0u;
  expand_chunk(t, blockIdx.y, blockIdx.x);
}

// One CTA per query tile, D / 8 threads per row (16-byte loads, whole rows
// per group of threads): delta_i = sum_d do_id o_id.
template <int D>
__global__ void __launch_bounds__(256) bwd_stats(const __grid_constant__ BwdParams p) {
  // The query walk may set itself up meanwhile.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x >= p.n_q) {  // the CTAs past the query tiles lay the bias out
    const int x = blockIdx.x - p.n_q, chunks = (rel_row(p.rel_table.reach) + 255) / 256;
    if (x == 0)
      for (int h = threadIdx.x; h < p.rel_table.N; h += 256) p.rel_done[h] = 0u;
    expand_chunk(p.rel_table, x / chunks, x % chunks);
    return;
  }
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

// Dense masks: thread n < n_q copies query item n's range, the n_g threads
// after them join those of a dQ item, the warps after them reduce one key item each: [lo, hi) from the first to the last query
// tile with a visible pair, and the longest run of fully visible ones (the
// first on ties). A FULL class covers 128 stored keys.
__global__ void __launch_bounds__(256) bwd_ranges(BwdOccParams a, int q_blocks) {
  if ((int)blockIdx.x < q_blocks) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.n_q) {
      const int m = n - a.n_q;
      if (m >= a.n_g) return;
      BwdItem it = a.g_items[m];
      const TileRange* r = a.ranges + (it.b * a.occ_sb + it.h * a.occ_sh) * a.n_qt + it.tile * 2;
      it.lo = it.hi = 0;
      for (int x = 0; x < 2 && it.tile * 2 + x < a.n_qt; ++x) {
        if (r[x].hi <= r[x].lo) continue;
        it.lo = it.hi > 0 ? min(it.lo, r[x].lo) : r[x].lo;
        it.hi = max(it.hi, r[x].hi);
      }
      a.g_items[m] = it;
      return;
    }
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
  a.spans[it.span].lo = it.lo;
  a.spans[it.span].hi = it.hi;
}

// dist[h][e] = sum over head h's key tiles, in 64 bits: one CTA per head and
// 32 distances, warp w adds tiles w, w + 8, ... and the eight sums are added
// in warp order. The last CTA of a head to finish then sums the distances of
// each bucket, those past the reach with the end they clip to: one warp per
// bucket. Every order is fixed.
__global__ void __launch_bounds__(256) rel_reduce(const float* __restrict__ part, double* dist,
                                                  unsigned int* done,
                                                  const int32_t* __restrict__ bucket_of,
                                                  float* __restrict__ dtable, int N, int tiles,
                                                  int reach, int num_buckets) {
  __shared__ double sm[8][32];
  __shared__ double by_dist[2 * kRelMaxReach + 1 + 2 * kRelPad];
  __shared__ int32_t bucket[2 * kRelMaxReach + 1 + 2 * kRelPad];
  __shared__ bool last;
  const int W = rel_width(reach);
  const int h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (d < W)
    for (int t = w; t < tiles; t += 8) s += part[((int64_t)h * tiles + t) * W + d];
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0) {
    if (d < W) {
      double a = sm[0][lane];
      for (int x = 1; x < 8; ++x) a += sm[x][lane];
      dist[(int64_t)h * W + d] = a;
    }
    __threadfence();
    __syncwarp();
    if (lane == 0) last = atomicAdd(done + h, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int e = threadIdx.x; e < W; e += 256) {
    by_dist[e] = __ldcg(dist + (int64_t)h * W + e);
    bucket[e] = bucket_of[min(max(e - kRelPad, 0), 2 * reach)];
  }
  __syncthreads();
  for (int c = w; c < num_buckets; c += 8) {
    double a = 0.0;
    for (int e = lane; e < W; e += 32)
      if (bucket[e] == c) a += by_dist[e];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
    if (lane == 0) dtable[(int64_t)c * N + h] = (float)a;
  }
}

}  // namespace

cudaError_t launch_bwd_stats(int D, const BwdParams& p, cudaStream_t stream) {
  if (p.n_q <= 0) return cudaSuccess;
  const int grid =
      p.n_q + (p.rel.ext ? (rel_row(p.rel_table.reach) + 255) / 256 * p.rel_table.N : 0);
  if (D == 128) bwd_stats<128><<<grid, 256, 0, stream>>>(p);
  else bwd_stats<64><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_bwd_ranges(const BwdOccParams& a, cudaStream_t stream) {
  const int qb = (a.n_q + a.n_g + 255) / 256, kb = (a.n_k + 7) / 8;
  if (qb + kb > 0) bwd_ranges<<<qb + kb, 256, 0, stream>>>(a, qb);
  return cudaGetLastError();
}

cudaError_t launch_rel_expand(const RelTable& t, unsigned int* zero, int64_t n_zero,
                              cudaStream_t stream) {
  rel_expand<<<dim3((rel_row(t.reach) + 255) / 256, t.N), 256, 0, stream>>>(t, zero, n_zero);
  return cudaGetLastError();
}

cudaError_t launch_rel_reduce(const float* rel_part, double* dist, unsigned int* done,
                              const int32_t* bucket_of, float* dtable, int32_t N, int32_t tiles,
                              int32_t num_buckets, int32_t reach, cudaStream_t stream) {
  rel_reduce<<<dim3((rel_width(reach) + 31) / 32, N), 256, 0, stream>>>(
      rel_part, dist, done, bucket_of, dtable, N, tiles, reach, num_buckets);
  return cudaGetLastError();
}

}  // namespace fa
