// C ABI front end of the backward pass and of the relative position bias's
// device tables: checks, work lists, scratch and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <iterator>
#include <vector>

#include "../../include/fa.h"
#include "fa_bwd.h"
#include "fa_handle.h"
#include "fa_kernel.h"
#include "fa_plan.h"

using namespace fa;

namespace fa {

fa_status_t ensure_buffer(fa_handle_t h, DeviceBuffer* buf, size_t bytes) {
  if (buf->ptr != nullptr && buf->bytes >= bytes) return FA_OK;
  if (env_flag("FA_TEST_FAIL_ALLOC")) return fail(FA_ERR_ALLOC, "device workspace (test hook)");
  if (buf->ptr != nullptr) {
    if (h->any_call) cudaEventSynchronize(h->last_call);
    cudaFree(buf->ptr);
    *buf = DeviceBuffer{};
  }
  const size_t want = align_up(bytes < 4096 ? 4096 : bytes, 4096);
  const cudaError_t e = cudaMalloc(&buf->ptr, want);
  if (e != cudaSuccess) {
    buf->ptr = nullptr;
    cudaGetLastError();
    return fail(FA_ERR_ALLOC, "cudaMalloc(%zu): %s", want, cudaGetErrorString(e));
  }
  buf->bytes = want;
  return FA_OK;
}

fa_status_t refuse_capture(cudaStream_t stream) {
  bool capturing = false;
  const fa_status_t st = stream_capturing(stream, &capturing);
  if (st == FA_OK && capturing)
    return fail(FA_ERR_UNSUPPORTED, "this call cannot be captured into a graph");
  return st;
}

void release_training(fa_handle_t h) {
  for (DeviceBuffer* b : {&h->bwd.lists, &h->bwd.scratch, &h->bwd.spill, &h->rel.map, &h->rel.ext,
                          &h->rel.rows})
    if (b->ptr) cudaFree(b->ptr);
  if (h->bwd.stage_done) {
    cudaEventSynchronize(h->bwd.stage_done);
    cudaEventDestroy(h->bwd.stage_done);
  }
  if (h->bwd.stage) cudaFreeHost(h->bwd.stage);
}

fa_status_t validate_rel(const fa_desc_t* d, const fa_relbias_t* bias) {
  if (!bias || !bias->table || !bias->bucket_of)
    return fail(FA_ERR_NULLPTR, "the bias, its table and its bucket map are required");
  if (d->alibi != FA_ALIBI_NONE)
    return fail(FA_ERR_PARAM_INVALID, "the handle names an ALiBi variant, not a learned bias");
  if (d->mask_kind != FA_MASK_NONE)
    return fail(FA_ERR_UNSUPPORTED, "a relative position bias with an attenMask is not supported");
  if (bias->reach < 1 || bias->num_buckets < 1)
    return fail(FA_ERR_PARAM_INVALID, "reach and num_buckets must be >= 1 (got %d, %d)",
                bias->reach, bias->num_buckets);
  if (bias->reach > kRelMaxReach || bias->num_buckets > kRelMaxBuckets)
    return fail(FA_ERR_UNSUPPORTED, "reach <= %d and num_buckets <= %d (got %d, %d)", kRelMaxReach,
                kRelMaxBuckets, bias->reach, bias->num_buckets);
  if ((uintptr_t)bias->table & 3u)
    return fail(FA_ERR_PARAM_INVALID, "the bias table must be 4-byte aligned");
  for (int32_t x = 0; x <= 2 * bias->reach; ++x)
    if (bias->bucket_of[x] < 0 || bias->bucket_of[x] >= bias->num_buckets)
      return fail(FA_ERR_PARAM_INVALID, "bucket_of[%d] = %d is outside [0, %d)", x,
                  bias->bucket_of[x], bias->num_buckets);
  return FA_OK;
}

fa_status_t prepare_rel(fa_handle_t h, const fa_relbias_t* bias, cudaStream_t stream, RelBias* out,
                        RelTable* table) {
  const int32_t N = (int32_t)h->desc.N, R = bias->reach, row = rel_row(R);
  // An earlier call on another stream may still read the tables.
  fa_status_t st = order_after_last(h, false, stream);
  if (st != FA_OK) return st;
  const size_t entries = (size_t)(2 * R + 1);
  st = ensure_buffer(h, &h->rel.ext, (size_t)N * 4 * row * sizeof(float));
  if (st != FA_OK) return st;
  std::vector<int32_t>& held = h->rel.bucket_of;
  if (held.size() != entries || !std::equal(held.begin(), held.end(), bias->bucket_of)) {
    held.clear();
    st = ensure_buffer(h, &h->rel.map, entries * sizeof(int32_t));
    if (st != FA_OK) return st;
    // From the handle's own copy, which is pageable: the call returns once it
    // has been read. (The caller's map may be pinned memory, which the copy
    // would read later, when the caller has rewritten it.)
    held.assign(bias->bucket_of, bias->bucket_of + entries);
    const cudaError_t e = cudaMemcpyAsync(h->rel.map.ptr, held.data(), entries * sizeof(int32_t),
                                          cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) {
      held.clear();
      return cuda_fail(e, "cudaMemcpyAsync(bucket map)");
    }
  }
  float* ext = static_cast<float*>(h->rel.ext.ptr);
  *out = RelBias{ext, R, row};
  *table = RelTable{bias->table, static_cast<const int32_t*>(h->rel.map.ptr), ext, N, R};
  return FA_OK;
}

}  // namespace fa

namespace {

// At most 4 GiB of dS are held at once (the test hook makes it less).
int64_t spill_tiles() {
  if (const char* t = std::getenv("FA_TEST_SPILL_TILES")) return std::atoll(t);
  return (int64_t(4) << 30) / (128 * 128 * 2);
}

// Longest first, in buckets of similar length inside which the items of one
// (sequence, head) stand together: the tiles in flight then share their
// operands through L2 (see order_work_list). The kernels claim them in this
// order; the last, without a tile, are zeros to write, which fill the end of
// the SMs that are done (164 us on a band 2 x 8k of 32 heads, 167 with them in
// front, 170 with them spread).
void order_items(std::vector<BwdItem>::iterator first, std::vector<BwdItem>::iterator last,
                 int num_sms) {
  const int32_t bucket = claims_items(last - first, num_sms) ? kLocalityTiles : 1;
  std::sort(first, last, [bucket](const BwdItem& a, const BwdItem& c) {
    const int32_t la = std::max(a.hi - a.lo, 0), lc = std::max(c.hi - c.lo, 0);
    const int32_t ba = (la + bucket - 1) / bucket, bc = (lc + bucket - 1) / bucket;
    if (ba != bc) return ba > bc;
    if (a.b != c.b) return a.b < c.b;
    if (a.h != c.h) return a.h < c.h;
    if (la != lc) return la > lc;
    return a.tile < c.tile;
  });
}

// Room for `tiles` tiles of dS.
bool room_for_ds(fa_handle_t h, int64_t tiles) {
  if (const char* t = std::getenv("FA_TEST_SPILL_ROOM"))
    if (tiles > std::atoll(t)) return false;
  if (ensure_buffer(h, &h->bwd.spill, (size_t)tiles * 128 * 128 * 2) == FA_OK) return true;
  clear_error();
  return false;
}

// The most tiles of dS held at once when heads are taken in order into shares
// of at most `cap` tiles; need[b] is a head's of sequence b.
int64_t largest_share(const std::vector<int64_t>& need, int64_t N, int64_t cap) {
  int64_t most = 0, used = 0;
  for (int64_t n : need) {
    for (int64_t hd = 0; hd < N; ++hd) {
      if (used + n > cap) used = 0;
      used += n;
      most = std::max(most, used);
    }
  }
  return most;
}

// Builds and uploads the lists of this call's lengths unless the handle
// holds them already. Where dS is written, its room is found here, so that a
// call keeps its way of working, and its bits, until the lengths change.
fa_status_t refresh_lists(fa_handle_t h, const int64_t* prefix, const int64_t* cu_q,
                          const int64_t* cu_kv, int has_mask, cudaStream_t stream) {
  BwdState& bw = h->bwd;
  std::vector<int64_t> key = make_key(&h->desc, prefix, cu_q, cu_kv, has_mask);
  if (bw.valid && key == bw.key) return FA_OK;
  const std::vector<SeqRec> recs = decode_geometry(&h->desc, prefix, cu_q, cu_kv, has_mask);
  const int32_t N = (int32_t)h->desc.N;
  int64_t tiles = 0, k_tiles = 0;
  for (const SeqRec& s : recs) {
    tiles += (s.sq + kTileM - 1) / kTileM;
    k_tiles += (s.skv + kTileN - 1) / kTileN;
  }
  if (std::max(tiles, k_tiles) * N > 0x3fffffff)
    return fail(FA_ERR_UNSUPPORTED, "too many work items");
  std::vector<TileRange> kr;       // of every key tile, sequence by sequence
  std::vector<int64_t> need;       // tiles of dS of one head; a mask's are not known here
  kr.reserve((size_t)k_tiles);
  need.reserve(recs.size());
  for (const SeqRec& s : recs) {
    const int32_t nq = (s.sq + kTileM - 1) / kTileM, nk = (s.skv + kTileN - 1) / kTileN;
    int64_t n = 0;
    for (int32_t t = 0; t < nk; ++t) {
      kr.push_back(key_tile_rows(s, (int64_t)t * kTileN));
      n += has_mask ? nq : kr.back().hi - kr.back().lo;
    }
    need.push_back(n);
  }
  // Two products less against 32 KB written and read a pair of tiles, and one
  // after the other instead of side by side. Causal, D = 128: 16 heads x 2048
  // (512 items) 71 us with dS written, 68 by two walks, 8 heads x 2048 60 and
  // 45, but 32 heads x 2048 (1,024 items) 136 and 149, 32 x 4096 430 and 459.
  // At D = 64 the products weigh half: 651 and 610 us on the bias backward of
  // 32 heads x 4096.
  bool spill = bwd_may_write_ds(h->desc.D) && (tiles + k_tiles) * N > 4 * h->num_sms;
  bw.valid = false;
  // Shares as large as there is memory for: their size changes no bit. When
  // there is none for one head's, two walks.
  int64_t cap = spill_tiles();
  const int64_t head = need.empty() ? 0 : *std::max_element(need.begin(), need.end());
  if (head > cap) spill = false;
  while (spill && head > 0) {
    const int64_t most = largest_share(need, N, cap);
    if (room_for_ds(h, most)) break;
    if (most <= head) spill = false;
    else cap = std::max(head, most / 2);
  }
  std::vector<BwdItem> qi, ki, gi;
  std::vector<KeySpan> spans((size_t)(k_tiles * N));
  qi.reserve((size_t)(tiles * N));
  ki.reserve((size_t)(k_tiles * N));
  std::vector<BwdState::Chunk> chunks;
  int64_t q_base = 0, k_base = 0, used = 0;  // used: tiles of dS in the current chunk
  for (size_t b = 0; b < recs.size(); ++b) {
    const SeqRec& s = recs[b];
    const int32_t nq = (s.sq + kTileM - 1) / kTileM, nk = (s.skv + kTileN - 1) / kTileN;
    std::vector<TileRange> qr((size_t)nq);
    for (int32_t t = 0; t < nq; ++t) qr[t] = tile_range(s, (int64_t)t * kTileM);
    const TileRange* kt = kr.data() + k_base;
    for (int32_t hd = 0; hd < N; ++hd) {
      for (int32_t t = 0; t < nq; ++t)
        qi.push_back(BwdItem{(int32_t)b, hd, t, (int32_t)(hd * tiles + q_base + t), qr[t].lo,
                             qr[t].hi, qr[t].full_lo, qr[t].full_hi, 0, {0, 0, 0}});
      if (spill && (chunks.empty() || used + need[b] > cap)) {
        chunks.push_back(
            {(int32_t)ki.size(), (int32_t)ki.size(), (int32_t)gi.size(), (int32_t)gi.size(), 0});
        used = 0;
      }
      const int32_t span = (int32_t)(hd * k_tiles + k_base);
      for (int32_t t = 0; t < nk; ++t) {
        ki.push_back(BwdItem{(int32_t)b, hd, t, (int32_t)(hd * tiles + q_base), kt[t].lo, kt[t].hi,
                             kt[t].full_lo, kt[t].full_hi, span + t, {0, 0, 0}});
        spans[span + t] = KeySpan{(int32_t)(has_mask ? used : used - kt[t].lo), kt[t].lo, kt[t].hi, 0};
        if (spill) used += has_mask ? nq : kt[t].hi - kt[t].lo;
      }
      for (int32_t t = 0; spill && t < nq; t += 2) {
        TileRange r = qr[t];
        if (t + 1 < nq && qr[t + 1].hi > qr[t + 1].lo) {
          r.lo = r.hi > r.lo ? std::min(r.lo, qr[t + 1].lo) : qr[t + 1].lo;
          r.hi = std::max(r.hi, qr[t + 1].hi);
        }
        gi.push_back(BwdItem{(int32_t)b, hd, t / 2, 0, r.lo, r.hi, 0, 0, span, {0, 0, 0}});
      }
      if (spill) {
        chunks.back().k1 = (int32_t)ki.size();
        chunks.back().g1 = (int32_t)gi.size();
        chunks.back().tiles = used;
      }
    }
    q_base += nq;
    k_base += nk;
  }
  order_items(qi.begin(), qi.end(), h->num_sms);
  if (!spill) order_items(ki.begin(), ki.end(), h->num_sms);
  for (const BwdState::Chunk& c : chunks) {
    order_items(ki.begin() + c.k0, ki.begin() + c.k1, h->num_sms);
    order_items(gi.begin() + c.g0, gi.begin() + c.g1, h->num_sms);
  }
  const size_t seq_bytes = align_up(recs.size() * sizeof(SeqRec), 256);
  const size_t q_bytes = align_up(qi.size() * sizeof(BwdItem), 256);
  const size_t k_bytes = align_up(ki.size() * sizeof(BwdItem), 256);
  const size_t g_bytes = align_up(gi.size() * sizeof(BwdItem), 256);
  const size_t total = seq_bytes + q_bytes + k_bytes + g_bytes + spans.size() * sizeof(KeySpan);
  fa_status_t st = ensure_buffer(h, &bw.lists, total);
  if (st != FA_OK) return st;
  st = ensure_pinned(&bw.stage, &bw.stage_bytes, bw.stage_done, total);
  if (st != FA_OK) return st;
  uint8_t* at = static_cast<uint8_t*>(bw.stage);
  auto put = [&](const void* src, size_t bytes, size_t room) {
    if (bytes) std::memcpy(at, src, bytes);
    at += room;
  };
  put(recs.data(), recs.size() * sizeof(SeqRec), seq_bytes);
  put(qi.data(), qi.size() * sizeof(BwdItem), q_bytes);
  put(ki.data(), ki.size() * sizeof(BwdItem), k_bytes);
  put(gi.data(), gi.size() * sizeof(BwdItem), g_bytes);
  put(spans.data(), spans.size() * sizeof(KeySpan), 0);
  cudaError_t e = cudaMemcpyAsync(bw.lists.ptr, bw.stage, total, cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(backward lists)");
  e = cudaEventRecord(bw.stage_done, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
  bw.key.swap(key);
  bw.valid = true;
  bw.n_q = (int32_t)qi.size();
  bw.n_k = (int32_t)ki.size();
  bw.n_g = (int32_t)gi.size();
  bw.tiles = (int32_t)tiles;
  bw.k_tiles = (int32_t)k_tiles;
  bw.chunks.swap(chunks);
  bw.geo0 = recs.empty() ? SeqRec{} : recs[0];
  return FA_OK;
}

struct BwdArgs {
  const void *q, *k, *v;
  const uint8_t* atten_mask;
  const float* slopes;
  const fa_relbias_t* bias;
  const void* o;
  const float* lse;
  const void* d_o;
  const float* d_lse;
  const int64_t *prefix, *cu_q, *cu_kv;
  void *dq, *dk, *dv;
  float* dtable;
};

// A gradient written over an operand, or over another gradient, would be read
// by the kernels beside its writer.
bool outputs_apart(const fa_desc_t* d, const BwdArgs& a) {
  const size_t seqs = d->layout == FA_TND ? 1 : (size_t)d->B, N = (size_t)d->N;
  const size_t row_side = seqs * N * (size_t)d->Sq, key_side = seqs * N * (size_t)d->Skv,
               D2 = (size_t)d->D * 2;
  struct Range {
    const void* at;
    size_t bytes;
  };
  const size_t table = a.bias ? (size_t)a.bias->num_buckets * N * 4 : 0;
  const size_t mask = (size_t)mask_planes(d, a.atten_mask != nullptr && d->sparse_mode <= 1) *
                      (size_t)d->Sq * (size_t)d->Skv;
  const Range ranges[] = {{a.dq, row_side * D2}, {a.dk, key_side * D2}, {a.dv, key_side * D2},
                          {a.dtable, table},     {a.q, row_side * D2},  {a.k, key_side * D2},
                          {a.v, key_side * D2},  {a.o, row_side * D2},  {a.d_o, row_side * D2},
                          {a.lse, row_side * 4}, {a.d_lse, row_side * 4},
                          {a.slopes, N * 4},     {a.bias ? a.bias->table : nullptr, table},
                          {a.atten_mask, mask}};
  constexpr int kOutputs = 4;
  for (int i = 0; i < kOutputs; ++i)
    for (const Range* r = ranges + i + 1; r != std::end(ranges); ++r) {
      const uintptr_t x = (uintptr_t)ranges[i].at, y = (uintptr_t)r->at;
      if (x && y && r->bytes && ranges[i].bytes && x < y + r->bytes && y < x + ranges[i].bytes)
        return false;
    }
  return true;
}

fa_status_t enqueue_backward(fa_handle_t h, const BwdArgs& a, void* cuda_stream) {
  const fa_desc_t* d = &h->desc;
  const bool rows = d->Sq > 0, keys = d->Skv > 0;
  if (rows && (!a.q || !a.o || !a.lse || !a.d_o || !a.dq))
    return fail(FA_ERR_NULLPTR, "q, o, lse, d_o and dq are required");
  if (keys && (!a.k || !a.v || !a.dk || !a.dv))
    return fail(FA_ERR_NULLPTR, "k, v, dk and dv are required");
  const int has_mask = d->sparse_mode <= 1 && a.atten_mask != nullptr;
  fa_status_t st = validate_call(d, a.prefix, a.cu_q, a.cu_kv, has_mask);
  if (st != FA_OK) return st;
  const uintptr_t align = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.o |
                          (uintptr_t)a.d_o | (uintptr_t)a.dq | (uintptr_t)a.dk | (uintptr_t)a.dv;
  if (align & 15u)
    return fail(FA_ERR_PARAM_INVALID, "q, k, v, o, d_o, dq, dk and dv must be 16-byte aligned");
  if (((uintptr_t)a.lse | (uintptr_t)a.d_lse | (uintptr_t)a.slopes | (uintptr_t)a.dtable) & 3u)
    return fail(FA_ERR_PARAM_INVALID, "lse, d_lse, slopes and dtable must be 4-byte aligned");
  if (!outputs_apart(d, a))
    return fail(FA_ERR_PARAM_INVALID, "a gradient overlaps an operand or another gradient");
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  st = refuse_capture(stream);
  if (st != FA_OK) return st;
  st = bind_device(h);
  if (st != FA_OK) return st;
  st = ensure_workspace(h, kHeaderBytes, stream);  // the error word
  if (st != FA_OK) return st;
  st = order_after_last(h, false, stream);  // lists and scratch are rewritten
  if (st != FA_OK) return st;
  FailedCall failed{h, stream, true};
  st = refresh_lists(h, a.prefix, a.cu_q, a.cu_kv, has_mask, stream);
  if (st != FA_OK) return st;
  int64_t ds_tiles = 0;
  for (const BwdState::Chunk& c : h->bwd.chunks) ds_tiles = std::max(ds_tiles, c.tiles);
  const BwdState& bw = h->bwd;

  // Scratch: row statistics | bias sums by tile and by distance, counters |
  // claim counters | the dense mask's bits both ways and classes.
  const size_t stat_bytes = align_up((size_t)bw.tiles * d->N * 256 * sizeof(float), 256);
  const size_t W = a.bias ? (size_t)rel_width(a.bias->reach) : 0;
  const size_t part_bytes = align_up((size_t)bw.k_tiles * d->N * W * sizeof(float), 256);
  const size_t dist_bytes = align_up((size_t)d->N * W * sizeof(double), 256);
  const int64_t planes = mask_planes(d, has_mask);
  const int64_t m_rows = (int64_t)align_up((size_t)d->Sq, kTileM),
                m_keys = (int64_t)align_up((size_t)d->Skv, kTileN);
  const size_t bits_bytes = planes ? align_up((size_t)(planes * m_rows * m_keys / 8), 256) : 0;
  const size_t occ_bytes =
      planes ? 2 * bits_bytes + (size_t)(planes * (m_rows / kTileM) * (m_keys / kTileN)) : 0;
  const size_t done_bytes = a.bias ? align_up((size_t)d->N * sizeof(unsigned int), 256) : 0;
  const size_t n_claims = 3 * std::max<size_t>(1, bw.chunks.size());
  const size_t claim_bytes = align_up(n_claims * sizeof(unsigned int), 256);
  st = ensure_buffer(h, &h->bwd.scratch,
                     stat_bytes + part_bytes + dist_bytes + done_bytes + claim_bytes + occ_bytes);
  if (st != FA_OK) return st;
  uint8_t* scratch = static_cast<uint8_t*>(bw.scratch.ptr);
  uint8_t* lists = static_cast<uint8_t*>(bw.lists.ptr);
  const size_t seq_bytes = align_up((size_t)d->B * sizeof(SeqRec), 256);

  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.seqs = reinterpret_cast<const SeqRec*>(lists);
  uint8_t* at = lists + seq_bytes;
  auto take = [&](int32_t n) {
    BwdItem* items = reinterpret_cast<BwdItem*>(at);
    at += align_up((size_t)n * sizeof(BwdItem), 256);
    return items;
  };
  BwdItem* q_items = take(bw.n_q);
  BwdItem* k_items = take(bw.n_k);
  BwdItem* g_items = take(bw.n_g);
  KeySpan* spans = reinterpret_cast<KeySpan*>(at);
  p.q_items = q_items;
  p.k_items = k_items;
  p.spans = spans;
  p.n_q = bw.n_q;
  p.n_k = bw.n_k;
  p.stats = reinterpret_cast<float*>(scratch);
  p.err_word = reinterpret_cast<unsigned int*>(h->d_ws);
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.d_o = a.d_o;
  p.lse = a.lse;
  p.d_lse = a.d_lse;
  p.dq = a.dq;
  p.dk = a.dk;
  p.dv = a.dv;
  operand_strides(d, d->Sq, &p.q_sb, &p.q_sh, &p.q_st);
  operand_strides(d, d->Skv, &p.k_sb, &p.k_sh, &p.k_st);
  p.tnd = d->layout == FA_TND ? 1 : 0;
  p.l_sb = p.tnd ? 0 : d->N * d->Sq;
  p.l_sh = d->Sq;
  p.scale = (float)d->scale;
  p.scale_log2 = (float)(d->scale * 1.4426950408889634073599);
  p.timeout_ns = h->timeout_ns;
  if (d->alibi != FA_ALIBI_NONE) {
    p.slopes = a.slopes;
    p.alibi = d->alibi;
  }
  // An operand without elements is never loaded from: any valid address does.
  const void* ops[4] = {a.q, a.k, a.v, a.d_o};
  CUtensorMap* maps[4] = {&p.tm_q, &p.tm_k, &p.tm_v, &p.tm_do};
  for (int i = 0; i < 4; ++i) {
    const bool row_side = i == 0 || i == 3;
    const int64_t S = row_side ? d->Sq : d->Skv;
    const int64_t sb = row_side ? p.q_sb : p.k_sb, sh = row_side ? p.q_sh : p.k_sh,
                  tok = row_side ? p.q_st : p.k_st;
    const int64_t S1 = S > 0 ? S : 1;
    if (!encode_operand_map(maps[i], S > 0 ? ops[i] : scratch, d->D, S, d->N, p.tnd ? 1 : d->B, tok,
                            sh > 0 ? sh : d->D, p.tnd ? S1 * d->N * d->D : (sb > 0 ? sb : d->N * d->D)))
      return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed for operand %d", i);
  }
  if (a.bias) {
    st = prepare_rel(h, a.bias, stream, &p.rel, &p.rel_table);
    if (st != FA_OK) return st;
    p.rel_done = reinterpret_cast<unsigned int*>(scratch + stat_bytes + part_bytes + dist_bytes);
    p.rel_part = reinterpret_cast<float*>(scratch + stat_bytes);
  }
  BwdMaskParams m;
  std::memset(&m, 0, sizeof(m));
  if (has_mask) {
    uint8_t* occ = scratch + stat_bytes + part_bytes + dist_bytes + done_bytes + claim_bytes;
    m.mask = a.atten_mask;
    m.bits_q = reinterpret_cast<uint32_t*>(occ);
    m.bits_k = reinterpret_cast<uint32_t*>(occ + bits_bytes);
    m.cls = occ + 2 * bits_bytes;
    m.geo = bw.geo0;
    m.q_items = q_items;
    m.k_items = k_items;
    m.g_items = g_items;
    m.spans = spans;
    m.planes = planes;
    m.m_sb = d->mask_kind == FA_MASK_SS ? 0 : (d->mask_kind == FA_MASK_B1SS ? 1 : (int32_t)d->N);
    m.m_sh = d->mask_kind == FA_MASK_BNSS ? 1 : 0;
    m.n_q = bw.n_q;
    m.n_k = bw.n_k;
    m.n_g = bw.n_g;
    m.n_qt = (int32_t)(m_rows / kTileM);
    m.n_kt = (int32_t)(m_keys / kTileN);
    if (planes * m.n_qt * m.n_kt > 0x7fffffff)
      return fail(FA_ERR_UNSUPPORTED, "too many mask tiles");
    p.bits_q = m.bits_q;
    p.bits_k = m.bits_k;
    p.m_sb = m.m_sb;
    p.m_sh = m.m_sh;
    p.m_rows = (int32_t)m_rows;
    p.m_keys = (int32_t)m_keys;
  }
  p.claims = reinterpret_cast<unsigned int*>(scratch + stat_bytes + part_bytes + dist_bytes + done_bytes);
  p.n_claims = (int32_t)n_claims;
  cudaError_t e = p.n_q > 0 ? launch_bwd_stats((int)d->D, p, m, stream)
                : cudaMemsetAsync(p.claims, 0, n_claims * sizeof(unsigned int), stream);
  if (e != cudaSuccess) return cuda_fail(e, "row statistics launch");
  const char* why = nullptr;
  if (ds_tiles > 0) {
    p.ds = static_cast<__nv_bfloat16*>(bw.spill.ptr);
    for (size_t c = 0; c < bw.chunks.size() && e == cudaSuccess; ++c) {
      const BwdState::Chunk& ch = bw.chunks[c];
      p.k_items = k_items + ch.k0;
      p.n_k = ch.k1 - ch.k0;
      p.g_items = g_items + ch.g0;
      p.n_g = ch.g1 - ch.g0;
      if (c > 0) p.claims += 3;
      e = launch_bwd((int)d->D, p, h->num_sms, stream, &why);
    }
  } else {
    e = launch_bwd((int)d->D, p, h->num_sms, stream, &why);
  }
  if (e != cudaSuccess) {
    if (why) return fail(FA_ERR_UNSUPPORTED, "launch refused: %s", why);
    return cuda_fail(e, "backward launch");
  }
  if (a.bias) {
    if (bw.n_q > 0)
      e = launch_rel_reduce(p.rel_part, reinterpret_cast<double*>(scratch + stat_bytes + part_bytes),
                            p.rel_done, p.rel_table.bucket_of, a.dtable, (int32_t)d->N, bw.k_tiles,
                            a.bias->num_buckets, a.bias->reach, stream);
    else
      e = cudaMemsetAsync(a.dtable, 0, (size_t)a.bias->num_buckets * d->N * sizeof(float), stream);
    if (e != cudaSuccess) return cuda_fail(e, "bias gradient launch");
  }
  failed.armed = false;
  return record_call(h, false, stream);
}

fa_status_t backward(fa_handle_t h, const BwdArgs& a, void* cuda_stream) try {
  return enqueue_backward(h, a, cuda_stream);
} catch (const std::exception& e) {
  return host_exception(e);
}

}  // namespace

extern "C" {

fa_status_t fa_bwd(fa_handle_t h, const void* q, const void* k, const void* v,
                   const uint8_t* atten_mask, const void* o, const float* lse, const void* d_o,
                   const float* d_lse, const int64_t* prefix, const int64_t* actual_seq_qlen,
                   const int64_t* actual_seq_kvlen, void* dq, void* dk, void* dv,
                   void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (h->desc.alibi != FA_ALIBI_NONE)
    return fail(FA_ERR_PARAM_INVALID,
                "the handle names an ALiBi variant: call fa_bwd_alibi with the slopes");
  return backward(h, BwdArgs{q, k, v, atten_mask, nullptr, nullptr, o, lse, d_o, d_lse, prefix,
                             actual_seq_qlen, actual_seq_kvlen, dq, dk, dv, nullptr},
                  cuda_stream);
}

fa_status_t fa_bwd_alibi(fa_handle_t h, const void* q, const void* k, const void* v,
                         const float* slopes, const void* o, const float* lse, const void* d_o,
                         const float* d_lse, const int64_t* prefix, const int64_t* actual_seq_qlen,
                         const int64_t* actual_seq_kvlen, void* dq, void* dk, void* dv,
                         void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (!slopes) return fail(FA_ERR_NULLPTR, "slopes is NULL");
  if (h->desc.alibi == FA_ALIBI_NONE)
    return fail(FA_ERR_PARAM_INVALID, "fa_bwd_alibi needs a handle with an ALiBi variant");
  return backward(h, BwdArgs{q, k, v, nullptr, slopes, nullptr, o, lse, d_o, d_lse, prefix,
                             actual_seq_qlen, actual_seq_kvlen, dq, dk, dv, nullptr},
                  cuda_stream);
}

fa_status_t fa_bwd_relbias(fa_handle_t h, const void* q, const void* k, const void* v,
                           const fa_relbias_t* bias, const void* o, const float* lse,
                           const void* d_o, const float* d_lse, const int64_t* prefix,
                           const int64_t* actual_seq_qlen, const int64_t* actual_seq_kvlen,
                           void* dq, void* dk, void* dv, float* dtable, void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  fa_status_t st = validate_rel(&h->desc, bias);
  if (st != FA_OK) return st;
  if (!dtable) return fail(FA_ERR_NULLPTR, "dtable is NULL");
  return backward(h, BwdArgs{q, k, v, nullptr, nullptr, bias, o, lse, d_o, d_lse, prefix,
                             actual_seq_qlen, actual_seq_kvlen, dq, dk, dv, dtable},
                  cuda_stream);
}

}  // extern "C"
