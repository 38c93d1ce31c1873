// Forward with the learned relative position bias for sequences of a few query
// rows (a decoding step): softmax(scale q.k + bias) v, and the log-sum-exp.
//
// With one to four rows there is no matrix product to feed the tensor cores:
// every key and value is read once for a handful of multiply-adds, so memory
// bounds it. The keys of each (sequence, head) are split over CTAs (few rows
// alone would leave most SMs idle), inside a CTA over its warps and over the
// groups of D / 8 threads that share a key, 8 dimensions each; every such
// group runs the online softmax (running maximum m, running sum l, both fp32)
// over its keys, several keys' loads in flight. The groups' states are joined
// by shuffles and through shared memory, and the last CTA of a (sequence,
// head) to finish joins the splits in their order, so the result does not
// depend on which one that is.
//
// Measured on 8 x 16 heads, one row against 8,191 keys of dimension 128 (537
// MB, 82 us at the card's copy rate): 96 us, 5.6 TB/s, against 120 us by the
// tensor-core kernel. Three keys a thread group, three CTAs an SM: 2 keys 102,
// 4 keys (two CTAs) 104 us; loads a step ahead and one softmax step for all
// keys in flight 100 against 109; heads-first order of the grid 96 against 100.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_rows.h"

namespace fa {
namespace {

constexpr int kSlice = 8;      // dimensions per thread (16: 106 us against 96)
constexpr int kWarps = 8;
constexpr int kPad = 4;        // a partial row: o[D], m, l, two pad floats
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Factor that brings a state of maximum m to the larger maximum m_new.
__device__ __forceinline__ float to_max(float m, float m_new) {
  return m == -INFINITY ? 0.f : ex2(m - m_new);
}

// R: rows a sequence may have. KEYS: keys of a thread group in flight. CTAS:
// CTAs that share an SM.
template <int D, int R, int KEYS, int CTAS>
__global__ void __launch_bounds__(32 * kWarps, CTAS) rows_forward(const RowsParams p) {
  constexpr int L = D / kSlice;        // threads per key
  constexpr int kVec = kSlice / 8;     // 16-byte loads of a thread's slice
  constexpr int G = 32 / L;            // keys a warp reads at once
  constexpr int kPass = kWarps * G;    // keys the CTA reads at once
  __shared__ float sm[kWarps][R][D + kPad];
  __shared__ bool last;
  // The bias is laid out and the counters are 0 once the launch ahead is done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Heads first: the CTAs in flight read the same tokens, whose heads are
  // adjacent in two of the layouts.
  const int h = blockIdx.x % p.N, s = (blockIdx.x / p.N) % p.splits;
  const int b = blockIdx.x / p.N / p.splits, bh = b * p.N + h;
  const SeqRec sr = p.seqs[b];
  if (sr.sq == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / L, sl = lane % L;
  const int delta = sr.skv - sr.sq;
  // Visible keys of all rows, and this CTA's share of them.
  const int64_t lo = imax64(0, row_lo(sr, 0));
  const int64_t hi = imin64((int64_t)sr.skv - 1, row_hi(sr, sr.sq - 1));
  const int64_t n = imax64(0, hi - lo + 1);
  const int64_t share = (n + p.splits - 1) / p.splits;
  const int key0 = (int)imin64(lo + s * share, hi + 1), key1 = (int)imin64(key0 + share, hi + 1);

  const int64_t q_off = b * p.q_sb + h * p.q_sh + (int64_t)sr.q_off * p.q_st;
  const int64_t k_off = b * p.k_sb + h * p.k_sh + (int64_t)sr.kv_off * p.k_st + sl * kSlice;
  const __nv_bfloat16* kb = reinterpret_cast<const __nv_bfloat16*>(p.k) + k_off;
  const __nv_bfloat16* vb = reinterpret_cast<const __nv_bfloat16*>(p.v) + k_off;
  const float* ext = p.rel.ext + (int64_t)h * 4 * p.rel.row + p.rel.reach + kRelPad;
  float q[R][kSlice], o[R][kSlice], m[R], l[R];
  int jlo[R], jhi[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    jlo[r] = 1, jhi[r] = 0;
    m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int x = 0; x < kSlice; ++x) q[r][x] = o[r][x] = 0.f;
    if (r < sr.sq) {
      jlo[r] = (int)imin64(imax64(0, row_lo(sr, r)), sr.skv);
      jhi[r] = (int)imax64(imin64((int64_t)sr.skv - 1, row_hi(sr, r)), -1);
      const uint4* src = reinterpret_cast<const uint4*>(
          reinterpret_cast<const __nv_bfloat16*>(p.q) + q_off + r * p.q_st + sl * kSlice);
#pragma unroll
      for (int y = 0; y < kSlice / 8; ++y) unpack8(__ldg(src + y), q[r] + 8 * y);
#pragma unroll
      for (int x = 0; x < kSlice; ++x) q[r][x] *= p.scale_log2;
    }
  }
  uint4 kv[KEYS][kVec], vv[KEYS][kVec], kn[KEYS][kVec], vn[KEYS][kVec];
  auto load = [&](int j0, uint4 (&kd)[KEYS][kVec], uint4 (&vd)[KEYS][kVec]) {
#pragma unroll
    for (int e = 0; e < KEYS; ++e) {
      const int j = j0 + e * kPass;
      const uint4* ks = reinterpret_cast<const uint4*>(kb + (int64_t)j * p.k_st);
      const uint4* vs = reinterpret_cast<const uint4*>(vb + (int64_t)j * p.k_st);
#pragma unroll
      for (int y = 0; y < kVec; ++y) {
        kd[e][y] = j < key1 ? __ldg(ks + y) : make_uint4(0u, 0u, 0u, 0u);
        vd[e][y] = j < key1 ? __ldg(vs + y) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  const int j_first = key0 + warp * G + grp;
  load(j_first, kv, vv);
  for (int j0 = j_first; j0 - grp < key1; j0 += KEYS * kPass) {
    load(j0 + KEYS * kPass, kn, vn);  // the next keys are under way while these are used
    float t[R][KEYS];
#pragma unroll
    for (int e = 0; e < KEYS; ++e) {
      float kf[kSlice];
#pragma unroll
      for (int y = 0; y < kVec; ++y) unpack8(kv[e][y], kf + 8 * y);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int x = 0; x < kSlice; x += 2) {
          d0 = fmaf(q[r][x], kf[x], d0);
          d1 = fmaf(q[r][x + 1], kf[x + 1], d1);
        }
        t[r][e] = d0 + d1;
      }
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < KEYS; ++e) t[r][e] += __shfl_xor_sync(0xffffffffu, t[r][e], d);
    // One step of the online softmax for all of these keys.
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mm = m[r];
#pragma unroll
      for (int e = 0; e < KEYS; ++e) {
        const int j = j0 + e * kPass;
        const int rel = min(max(j - (r + delta), -p.rel.reach), p.rel.reach);
        const float bias = __ldg(ext + rel);
        t[r][e] = j < key1 && j >= jlo[r] && j <= jhi[r] ? t[r][e] + bias : -INFINITY;
        mm = fmaxf(mm, t[r][e]);
      }
      const float ref = mm == -INFINITY ? 0.f : mm;  // no visible key yet: every weight is 0
      const float a = ex2(m[r] - ref);
      m[r] = mm;
      l[r] *= a;
#pragma unroll
      for (int x = 0; x < kSlice; ++x) o[r][x] *= a;
#pragma unroll
      for (int e = 0; e < KEYS; ++e) {
        t[r][e] = ex2(t[r][e] - ref);
        l[r] += t[r][e];
      }
    }
#pragma unroll
    for (int e = 0; e < KEYS; ++e) {
      float vf[kSlice];
#pragma unroll
      for (int y = 0; y < kVec; ++y) unpack8(vv[e][y], vf + 8 * y);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int x = 0; x < kSlice; ++x) o[r][x] = fmaf(t[r][e], vf[x], o[r][x]);
    }
#pragma unroll
    for (int e = 0; e < KEYS; ++e)
#pragma unroll
      for (int y = 0; y < kVec; ++y) kv[e][y] = kn[e][y], vv[e][y] = vn[e][y];
  }
  // Join the warp's groups, then the warps in their order.
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int d = L; d < 32; d <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[r], d);
      const float mm = fmaxf(m[r], m2);
      const float a = to_max(m[r], mm), a2 = to_max(m2, mm);
      l[r] = l[r] * a + __shfl_xor_sync(0xffffffffu, l[r], d) * a2;
#pragma unroll
      for (int x = 0; x < kSlice; ++x)
        o[r][x] = o[r][x] * a + __shfl_xor_sync(0xffffffffu, o[r][x], d) * a2;
      m[r] = mm;
    }
    if (grp == 0) {
#pragma unroll
      for (int x = 0; x < kSlice; ++x) sm[warp][r][sl * kSlice + x] = o[r][x];
      if (sl == 0) {
        sm[warp][r][D] = m[r];
        sm[warp][r][D + 1] = l[r];
      }
    }
  }
  __syncthreads();
  float* part = p.part + ((int64_t)bh * p.splits + s) * kFewRows * (D + kPad);
  const int rows = R == 1 ? 1 : sr.sq;
  // One thread per (row, dimension): state of `count` rows of D + kPad floats,
  // `stride` floats apart.
  auto join = [&](const float* src, int count, int64_t stride, float& acc, float& mm, float& ll,
                  int d, bool global) {
    mm = -INFINITY;
    for (int c = 0; c < count; ++c) {
      const float* x = src + c * stride + D;
      mm = fmaxf(mm, global ? __ldcg(x) : *x);
    }
    acc = ll = 0.f;
    for (int c = 0; c < count; ++c) {
      const float* x = src + c * stride;
      const float a = to_max(global ? __ldcg(x + D) : x[D], mm);
      ll += (global ? __ldcg(x + D + 1) : x[D + 1]) * a;
      acc += (global ? __ldcg(x + d) : x[d]) * a;
    }
  };
  auto put = [&](int r, int d, float acc, float mm, float ll) {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + q_off + r * p.q_st;
    // A row that sees nothing has the sum 0; a NaN score makes it NaN, which
    // o and lse keep.
    const bool none = ll == 0.f;
    dst[d] = __float2bfloat16_rn(none ? 0.f : acc / ll);
    if (d == 0)
      p.lse[b * p.l_sb + h * p.l_sh + sr.q_off + r] =
          none ? -INFINITY : (mm + log2f(ll)) * kLn2;
  };
  for (int x = threadIdx.x; x < rows * D; x += 32 * kWarps) {
    const int r = x / D, d = x % D;
    float acc, mm, ll;
    join(&sm[0][r][0], kWarps, R * (D + kPad), acc, mm, ll, d, false);
    if (p.splits == 1) {
      put(r, d, acc, mm, ll);
    } else {
      float* dst = part + r * (D + kPad);
      dst[d] = acc;
      if (d == 0) {
        dst[D] = mm;
        dst[D + 1] = ll;
      }
    }
  }
  if (p.splits == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.done + bh, 1u) == (unsigned)p.splits - 1u;
  __syncthreads();
  if (!last) return;
  __threadfence();
  const float* first = p.part + (int64_t)bh * p.splits * kFewRows * (D + kPad);
  for (int x = threadIdx.x; x < rows * D; x += 32 * kWarps) {
    const int r = x / D, d = x % D;
    float acc, mm, ll;
    join(first + r * (D + kPad), p.splits, kFewRows * (D + kPad), acc, mm, ll, d, true);
    put(r, d, acc, mm, ll);
  }
}

template <int D, int R, int KEYS, int CTAS>
cudaError_t launch_d(const RowsParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.N * p.splits));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at = {};  // the CTAs may take their places before the layout is done
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_forward<D, R, KEYS, CTAS>, p);
}

}  // namespace

int32_t rows_splits(int64_t groups, int64_t max_keys, int num_sms) {
  // About 8 CTAs per SM, of at least 256 keys each.
  const int64_t want = (8 * (int64_t)num_sms + groups - 1) / (groups > 0 ? groups : 1);
  const int64_t most = (max_keys + 255) / 256;
  const int64_t s = want < most ? want : most;
  return (int32_t)(s < 1 ? 1 : (s > 128 ? 128 : s));
}

size_t rows_part_bytes(int D, int64_t groups, int32_t splits) {
  return (size_t)groups * splits * kFewRows * (D + kPad) * sizeof(float);
}

cudaError_t launch_rows(int D, int max_rows, const RowsParams& p, const RelTable& table,
                        cudaStream_t stream) {
  const cudaError_t e = launch_rel_expand(table, p.done, p.B * p.N, stream);
  if (e != cudaSuccess) return e;
  if (D == 128)
    return max_rows <= 1 ? launch_d<128, 1, 3, 3>(p, stream) : launch_d<128, kFewRows, 2, 2>(p, stream);
  return max_rows <= 1 ? launch_d<64, 1, 3, 3>(p, stream) : launch_d<64, kFewRows, 2, 2>(p, stream);
}

}  // namespace fa
