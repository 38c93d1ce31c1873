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

// One CTA per tile; warp w takes the 32 x 32 blocks (w / 2, 2 (w % 2) + 0, 1):
// lane l reads key l of every row, so that a vote gives a row's word and the
// lane gathers its key's.
__device__ __forceinline__ void mask_tile(const BwdMaskParams& a, int64_t tile) {
  const int kt = (int)(tile % a.n_kt), qt = (int)(tile / a.n_kt % a.n_qt);
  const int64_t plane = tile / a.n_kt / a.n_qt;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqRec& s = a.geo;
  const uint8_t* m = a.mask + plane * s.sq * (int64_t)s.skv;
  const int64_t rows = (int64_t)a.n_qt * kTileM, keys = (int64_t)a.n_kt * kTileN;
  const int row0 = qt * kTileM + (w >> 1) * 32;
  bool any = false, full = true;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int key0 = kt * kTileN + ((w & 1) * 2 + y) * 32;
    const int j = key0 + lane;
    uint32_t hidden_row = 0u, hidden_key = 0u;
    uint8_t v[32];
    // Addresses are kept inside the mask, so that all loads are in flight.
    const uint8_t* col = m + min(j, s.skv - 1);
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = __ldg(col + (int64_t)min(row0 + r, s.sq - 1) * s.skv);
    if (row0 + 32 > s.sq || key0 + 32 > s.skv) {
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (row0 + r >= s.sq || j >= s.skv) v[r] = 1;
    }
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const uint32_t word = __ballot_sync(0xffffffffu, v[r] != 0);
      if (lane == r) hidden_row = word;
      hidden_key |= (v[r] != 0 ? 1u : 0u) << r;
    }
    a.bits_q[(plane * (keys / 32) + key0 / 32) * rows + row0 + lane] = hidden_row;
    a.bits_k[(plane * (rows / 32) + row0 / 32) * keys + j] = hidden_key;
    // Row row0 + lane against the window of the geometry.
    const int i = row0 + lane;
    if (i < s.sq) {
      const int64_t lo = imax64(row_lo(s, i) - key0, 0), hi = imin64(row_hi(s, i) - key0, 31);
      uint32_t window = 0u;
      if (lo <= hi) window = (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
      const uint32_t see = window & ~hidden_row;
      any |= see != 0u;
      full &= see == 0xffffffffu;
    }
  }
  const int some = __syncthreads_or(any), all = __syncthreads_and(full);
  if (threadIdx.x == 0)
    a.cls[tile] = some ? (all ? FA_TILE_FULL : FA_TILE_PARTIAL) : FA_TILE_EMPTY;
}

// One CTA per query tile, D / 8 threads per row (16-byte loads, whole rows
// per group of threads): delta_i = sum_d do_id o_id. Bound by memory.
template <int D>
__global__ void __launch_bounds__(256) bwd_stats(const __grid_constant__ BwdParams p,
                                                 const __grid_constant__ BwdMaskParams a,
                                                 int mask_tiles) {
  // The query walk may set itself up meanwhile.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x < mask_tiles) {
    mask_tile(a, blockIdx.x);
    return;
  }
  const int block = blockIdx.x - mask_tiles;
  if (block == 0)
    for (int x = threadIdx.x; x < p.n_claims; x += 256) p.claims[x] = 0u;
  if (block >= p.n_q) {  // the CTAs past the query tiles lay the bias out
    const int x = block - p.n_q, chunks = (rel_row(p.rel_table.reach) + 255) / 256;
    if (x == 0)
      for (int h = threadIdx.x; h < p.rel_table.N; h += 256) p.rel_done[h] = 0u;
    expand_chunk(p.rel_table, x / chunks, x % chunks);
    return;
  }
  constexpr int L = D / 8;            // threads per row
  constexpr int R = 256 / L;          // rows per pass
  const BwdItem it = p.q_items[block];
  const SeqRec s = p.seqs[it.b];
  const int sl = threadIdx.x % L;
  const int64_t base = it.b * p.q_sb + it.h * p.q_sh;
  const int row = threadIdx.x;  // of the first 128 threads
  const int64_t i0 = (int64_t)it.tile * kTileM;
  const bool stored = row < kTileM && i0 + row < s.sq;
  const int64_t at = it.b * p.l_sb + it.h * p.l_sh + s.q_off + i0 + row;
  float l = stored ? p.lse[at] : -INFINITY;
  const float dl = stored && p.d_lse ? p.d_lse[at] : 0.f;
  // Addresses are kept inside the sequence, so that all loads are in flight.
  uint4 vo[kTileM / R], vd[kTileM / R];
#pragma unroll
  for (int x = 0; x < kTileM / R; ++x) {
    const int64_t i = imin64(i0 + x * R + threadIdx.x / L, s.sq - 1);
    const int64_t off = base + (s.q_off + i) * p.q_st + sl * 8;
    vo[x] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.o) + off));
    vd[x] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.d_o) + off));
  }
  __shared__ float delta[kTileM];
#pragma unroll
  for (int x = 0; x < kTileM / R; ++x) {
    float d = dot8(vo[x], vd[x]);
#pragma unroll
    for (int y = 1; y < L; y <<= 1) d += __shfl_xor_sync(0xffffffffu, d, y);
    if (sl == 0) delta[x * R + threadIdx.x / L] = d;
  }
  __syncthreads();
  if (row >= kTileM) return;
  float nl = -INFINITY, nd = 0.f;
  if (l != -INFINITY) {
    // Left-aligned ALiBi: the same weights as the right-aligned bias, which
    // the kernels add, with every score of the row shifted.
    if (p.alibi == FA_ALIBI_LEFT)
      l = fmaf(-p.slopes[it.h], (float)(i0 + row + (int64_t)s.skv - s.sq), l);
    nl = -l * kLog2e;
    nd = dl - delta[row];
  }
  float* out = p.stats + (int64_t)it.stat * 256;
  out[row] = nl;
  out[kTileM + row] = nd;
}

// [lo, hi) and the longest run of FULL (the first on ties) of n classes
// `stride` apart; the same in every lane of the warp.
__device__ TileRange class_range(const uint8_t* cls, int n, int64_t stride) {
  const int lane = threadIdx.x & 31;
  int lo = 0x7fffffff, hi = 0;
  int best = 0, best_at = 0, run = 0;
  for (int t0 = 0; t0 < n; t0 += 32) {
    const int t = t0 + lane;
    const int c = t < n ? cls[t * stride] : FA_TILE_EMPTY;
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
  TileRange r;
  r.lo = hi > 0 ? lo : 0;
  r.hi = hi;
  r.full_lo = best > 0 ? best_at : r.lo;
  r.full_hi = best > 0 ? best_at + best : r.lo;
  return r;
}

// One warp per item: query items, key items (and their spans), dQ items.
__global__ void __launch_bounds__(256) bwd_ranges(BwdMaskParams a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  auto plane = [&](const BwdItem& it) {
    return a.cls + (int64_t)(it.b * a.m_sb + it.h * a.m_sh) * a.n_qt * a.n_kt;
  };
  auto put = [&](BwdItem* at, const TileRange& r) {
    at->lo = r.lo, at->hi = r.hi, at->full_lo = r.full_lo, at->full_hi = r.full_hi;
  };
  if (n < a.n_q) {
    const BwdItem it = a.q_items[n];
    const TileRange r = class_range(plane(it) + (int64_t)it.tile * a.n_kt, a.n_kt, 1);
    if (lane == 0) put(a.q_items + n, r);
    return;
  }
  n -= a.n_q;
  if (n < a.n_k) {
    const BwdItem it = a.k_items[n];
    const TileRange r = class_range(plane(it) + it.tile, a.n_qt, a.n_kt);
    if (lane == 0) {
      put(a.k_items + n, r);
      a.spans[it.span].lo = r.lo;
      a.spans[it.span].hi = r.hi;
    }
    return;
  }
  n -= a.n_k;
  if (n < a.n_g) {
    const BwdItem it = a.g_items[n];
    TileRange u{0, 0, 0, 0};
    for (int x = 0; x < 2 && it.tile * 2 + x < a.n_qt; ++x) {
      const TileRange r = class_range(plane(it) + (int64_t)(it.tile * 2 + x) * a.n_kt, a.n_kt, 1);
      if (r.hi <= r.lo) continue;
      u.lo = u.hi > 0 ? min(u.lo, r.lo) : r.lo;
      u.hi = max(u.hi, r.hi);
    }
    if (lane == 0) put(a.g_items + n, u);
  }
}

// dist[h][e] = sum over head h's key tiles, in 64 bits: one CTA per head and
// 32 distances, warp w adds tiles w, w + 8, ... and the eight sums are added
// in warp order. The last CTA of a head to finish then sums the distances of
// each bucket, those past the reach with the end they clip to, in 64 bits too:
// one warp per bucket. Every order is fixed.
__global__ void __launch_bounds__(256) rel_reduce(const float* __restrict__ part, double* dist,
                                                  unsigned int* done,
                                                  const int32_t* __restrict__ bucket_of,
                                                  float* __restrict__ dtable, int N, int tiles,
                                                  int reach, int num_buckets) {
  __shared__ double sm[8][32];
  constexpr int kRoom = (2 * kRelMaxReach + 1 + 2 * kRelPad + 127) / 128 * 128;
  __shared__ double by_dist[kRoom];  // 64 bits: distances of a bucket may cancel
  __shared__ int32_t bucket[kRoom];
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
  const int padded = (W + 127) / 128 * 128;
  for (int e = threadIdx.x; e < padded; e += 256) {
    by_dist[e] = e < W ? __ldcg(dist + (int64_t)h * W + e) : 0.0;
    bucket[e] = e < W ? bucket_of[min(max(e - kRelPad, 0), 2 * reach)] : -1;
  }
  __syncthreads();
  for (int c = w; c < num_buckets; c += 8) {
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    for (int e = lane; e < padded; e += 128)
#pragma unroll
      for (int y = 0; y < 4; ++y) a[y] += bucket[e + 32 * y] == c ? by_dist[e + 32 * y] : 0.0;
    double sum = (a[0] + a[1]) + (a[2] + a[3]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) dtable[(int64_t)c * N + h] = (float)sum;
  }
}

}  // namespace

cudaError_t launch_bwd_stats(int D, const BwdParams& p, const BwdMaskParams& mask,
                             cudaStream_t stream) {
  if (p.n_q <= 0) return cudaSuccess;
  const int64_t tiles = mask.planes * mask.n_qt * mask.n_kt;
  const int64_t grid =
      tiles + p.n_q + (p.rel.ext ? (rel_row(p.rel_table.reach) + 255) / 256 * p.rel_table.N : 0);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (D == 128) bwd_stats<128><<<(int)grid, 256, 0, stream>>>(p, mask, (int)tiles);
  else bwd_stats<64><<<(int)grid, 256, 0, stream>>>(p, mask, (int)tiles);
  if (tiles > 0) {
    const int64_t items = (int64_t)mask.n_q + mask.n_k + mask.n_g;
    bwd_ranges<<<(int)((items + 7) / 8), 256, 0, stream>>>(mask);
  }
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
