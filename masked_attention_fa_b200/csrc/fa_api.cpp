// C ABI front end: handles, per-call plan caching and the kernel launch.
//
// Two-stage use as the aclnnScatterPaKvCache page's host flow describes it:
// the descriptor is checked once (fa_create), then each fa_fwd validates its
// per-call arrays, reuses or rebuilds the cached work list, copies it to the
// handle's device workspace through pinned staging memory and enqueues the
// persistent kernel on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <new>
#include <vector>

#include "../../include/fa.h"
#include "fa_handle.h"
#include "fa_rows.h"
#include "fa_kernel.h"
#include "fa_plan.h"

using namespace fa;

namespace {

constexpr size_t kClaimOffset = 128;  // two work-claim counters, 64 bytes apart

}  // namespace

namespace fa {

bool env_flag(const char* name) {
  const char* v = std::getenv(name);
  return v != nullptr && v[0] != '\0' && v[0] != '0';
}

fa_status_t cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();  // reported here: the next call's launches do not find it
  return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Planes of the attenMask the occupancy pre-pass reduces: SS one plane for
// every batch and head, B1SS one per batch, BNSS one per batch and head; 0
// when the call reads no mask.
int64_t mask_planes(const fa_desc_t* d, int has_mask) {
  if (!has_mask) return 0;
  if (d->mask_kind == FA_MASK_SS) return 1;
  if (d->mask_kind == FA_MASK_B1SS) return d->B;
  return d->B * d->N;
}

}  // namespace fa

namespace {

// Dense-mask calls keep, after the work list, each item's two ranges
// (item_tr, 32 bytes per item) and then the pre-pass's scratch.
size_t item_tr_offset(int32_t n_seqs, int32_t n_items) {
  return align_up(kHeaderBytes + align_up((size_t)n_seqs * sizeof(SeqRec), 256) +
                      (size_t)n_items * sizeof(WorkItem),
                  256);
}
size_t occupancy_offset(int32_t n_seqs, int32_t n_items) {
  return item_tr_offset(n_seqs, n_items) +
         align_up((size_t)n_items * 2 * sizeof(TileRange), 256);
}

// Point the pre-pass at `scratch`: the ranges, then (256-byte aligned) the
// classes; `a` already has its shape.
void occupancy_bind(OccParams* a, uint8_t* scratch) {
  a->ranges = reinterpret_cast<TileRange*>(scratch);
  a->cls = scratch + align_up((size_t)(a->n_planes * a->n_qt) * sizeof(TileRange), 256);
}

}  // namespace

namespace fa {

fa_status_t bind_device(fa_handle_t h) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (h->device >= 0) {
    if (dev != h->device)
      return fail(FA_ERR_PARAM_INVALID, "handle is bound to device %d, current device is %d",
                  h->device, dev);
    return FA_OK;
  }
  int major = 0, minor = 0, sms = 0;
  e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (major != 10 || minor != 0)
    return fail(FA_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library runs on sm_100 (B200)", dev,
                major, minor);
  e = cudaEventCreateWithFlags(&h->stage_done, cudaEventDisableTiming);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventCreate");
  e = cudaEventCreateWithFlags(&h->bwd.stage_done, cudaEventDisableTiming);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventCreate");
  e = cudaEventCreateWithFlags(&h->last_call, cudaEventDisableTiming);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventCreate");
  h->device = dev;
  h->num_sms = sms;
  return FA_OK;
}


fa_status_t stream_capturing(cudaStream_t stream, bool* capturing) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(stream, &cap);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  *capturing = cap != cudaStreamCaptureStatusNone;
  return FA_OK;
}

fa_status_t order_after_last(fa_handle_t h, bool capturing, cudaStream_t stream) {
  if (!h->any_call || capturing) return FA_OK;
  const cudaError_t e = cudaStreamWaitEvent(stream, h->last_call, 0);
  return e == cudaSuccess ? FA_OK : cuda_fail(e, "cudaStreamWaitEvent");
}

fa_status_t record_call(fa_handle_t h, bool capturing, cudaStream_t stream) {
  if (capturing) {
    h->captured = true;
    return FA_OK;
  }
  const cudaError_t e = cudaEventRecord(h->last_call, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
  h->any_call = true;
  return FA_OK;
}

// The graph of a captured call reads the workspace's list at every replay: a
// new list goes into a new workspace, and the old one is kept.
void retire_captured(fa_handle_t h) {
  if (!h->captured) return;
  h->retired.push_back(h->d_ws);
  h->d_ws = nullptr;
  h->ws_bytes = 0;
  h->captured = false;
}

// Make sure the device workspace holds `bytes`; the error word is zeroed
// whenever the workspace is (re)allocated. The plan in the old one goes with
// it, also when there is no memory for a new one: a later call that finds its
// lengths in the plan's key would run on a workspace without its list.
// The header is cleared on the call's stream: on the default stream it could
// wait behind other work there while the call's kernels, on a stream that does
// not wait for that one, already read the claim counters.
fa_status_t ensure_workspace(fa_handle_t h, size_t bytes, cudaStream_t stream) {
  if (h->d_ws != nullptr && h->ws_bytes >= bytes) return FA_OK;
  if (h->d_ws != nullptr) {
    if (h->any_call) cudaEventSynchronize(h->last_call);
    cudaFree(h->d_ws);
    h->d_ws = nullptr;
    h->ws_bytes = 0;
  }
  h->plan_valid = false;
  size_t want = align_up(bytes < 4096 ? 4096 : bytes, 4096);
  if (env_flag("FA_TEST_FAIL_ALLOC")) want = (size_t)1 << 60;  // more than there is
  cudaError_t e = cudaMalloc(&h->d_ws, want);
  if (e != cudaSuccess) {
    h->d_ws = nullptr;
    cudaGetLastError();
    return fail(FA_ERR_ALLOC, "cudaMalloc(%zu): %s", want, cudaGetErrorString(e));
  }
  e = cudaMemsetAsync(h->d_ws, 0, kHeaderBytes, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  h->ws_bytes = want;
  return FA_OK;
}

}  // namespace fa

namespace fa {

fa_status_t ensure_pinned(void** stage, size_t* have, cudaEvent_t done, size_t bytes) {
  const cudaError_t s = cudaEventSynchronize(done);
  if (s != cudaSuccess) return cuda_fail(s, "cudaEventSynchronize");
  if (*stage != nullptr && *have >= bytes) return FA_OK;
  if (*stage != nullptr) cudaFreeHost(*stage);
  *stage = nullptr;
  *have = 0;
  const size_t want = align_up(bytes < 4096 ? 4096 : bytes, 4096);
  const cudaError_t e = cudaMallocHost(stage, want);
  if (e != cudaSuccess) {
    *stage = nullptr;
    cudaGetLastError();
    return fail(FA_ERR_ALLOC, "cudaMallocHost(%zu): %s", want, cudaGetErrorString(e));
  }
  *have = want;
  return FA_OK;
}

}  // namespace fa

namespace fa {

std::vector<int64_t> make_key(const fa_desc_t* d, const int64_t* prefix, const int64_t* cu_q,
                              const int64_t* cu_kv, int has_mask) {
  std::vector<int64_t> key;
  key.push_back(has_mask);
  if (d->sparse_mode == 5 || d->sparse_mode == 6) key.insert(key.end(), prefix, prefix + d->B);
  if (d->layout == FA_TND) {
    key.insert(key.end(), cu_q, cu_q + d->B);
    key.insert(key.end(), cu_kv, cu_kv + d->B);
  }
  return key;
}

}  // namespace fa

namespace {

// A captured upload would read the staging memory of a later call at replay.
fa_status_t no_plan_in_capture() {
  return fail(FA_ERR_UNSUPPORTED,
              "these lengths need a new work list, which cannot be captured: make the call once "
              "outside the capture first");
}

fa_status_t refresh_plan(fa_handle_t h, const int64_t* prefix, const int64_t* cu_q,
                         const int64_t* cu_kv, int has_mask, bool capturing, cudaStream_t stream) {
  std::vector<int64_t> key = make_key(&h->desc, prefix, cu_q, cu_kv, has_mask);
  if (h->plan_valid && key == h->plan_key) return FA_OK;
  if (capturing) return no_plan_in_capture();
  std::vector<SeqRec> recs = decode_geometry(&h->desc, prefix, cu_q, cu_kv, has_mask);
  std::vector<WorkItem> items = build_items(&h->desc, recs);
  if (items.size() > (size_t)0x7fffffff) return fail(FA_ERR_UNSUPPORTED, "too many work items");
  // Claimed lists (closed form only) take the L2-locality order.
  if (!has_mask && claims_items((int64_t)items.size(), h->num_sms))
    order_work_list(items.data(), items.data() + items.size(), true);
  const size_t seq_bytes = recs.size() * sizeof(SeqRec);
  const size_t item_bytes = items.size() * sizeof(WorkItem);
  const int64_t planes = mask_planes(&h->desc, has_mask);
  // Each item's two sub-tile ranges follow the list (item_tr): computed
  // here from the closed form and uploaded with it, or for a dense mask
  // written on the device by the rebuild kernel, followed by the pre-pass's
  // scratch. The kernel then reads a range with one load that does not wait
  // for the item record (computing it took ~1-2k cycles at each boundary).
  const size_t tr_off = item_tr_offset((int32_t)recs.size(), (int32_t)items.size());
  const size_t tr_bytes = items.size() * 2 * sizeof(TileRange);
  const size_t payload = planes ? align_up(seq_bytes, 256) + item_bytes
                                : tr_off - kHeaderBytes + tr_bytes;
  const size_t occ = planes ? occupancy_bytes(planes, h->desc.Sq, h->desc.Skv) : 0;
  retire_captured(h);
  fa_status_t st = ensure_workspace(
      h, planes ? occupancy_offset((int32_t)recs.size(), (int32_t)items.size()) + occ
                : kHeaderBytes + payload,
      stream);
  if (st != FA_OK) return st;
  st = ensure_pinned(&h->h_stage, &h->stage_bytes, h->stage_done, payload);
  if (st != FA_OK) return st;
  // A kernel of this handle on another stream may still read the old list.
  st = order_after_last(h, false, stream);
  if (st != FA_OK) return st;
  uint8_t* hs = static_cast<uint8_t*>(h->h_stage);
  std::memcpy(hs, recs.data(), seq_bytes);
  if (item_bytes) std::memcpy(hs + align_up(seq_bytes, 256), items.data(), item_bytes);
  if (!planes) {  // each item's two sub-tile ranges, from the closed form
    TileRange* tr = reinterpret_cast<TileRange*>(hs + (tr_off - kHeaderBytes));
    for (size_t n = 0; n < items.size(); ++n) {
      const SeqRec& sr = recs[(size_t)items[n].b];
      for (int st = 0; st < kSubTiles; ++st) {
        const int64_t r0 = (int64_t)items[n].qblk * kBlockM + st * kTileM;
        tr[2 * n + st] = r0 < sr.sq ? tile_range(sr, r0) : TileRange{0, 0, 0, 0};
      }
    }
  }
  h->plan_valid = false;  // until the new one is whole
  cudaError_t e = cudaMemcpyAsync(static_cast<uint8_t*>(h->d_ws) + kHeaderBytes, hs, payload,
                      cudaMemcpyHostToDevice, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(work list)");
  e = cudaEventRecord(h->stage_done, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
  h->plan_key.swap(key);
  h->plan_valid = true;
  h->n_items = (int32_t)items.size();
  h->n_seqs = (int32_t)recs.size();
  if (!recs.empty()) h->geo0 = recs[0];
  h->max_rows = h->max_keys = 0;
  for (const SeqRec& r : recs) {
    h->max_rows = std::max(h->max_rows, r.sq);
    h->max_keys = std::max(h->max_keys, r.skv);
  }
  return FA_OK;
}

// The forward with the learned bias for sequences of a few rows.
fa_status_t forward_rows(fa_handle_t h, const void* q, const void* k, const void* v,
                         const fa_relbias_t* bias, void* o, float* lse, cudaStream_t stream) {
  const fa_desc_t* d = &h->desc;
  RowsParams p;
  std::memset(&p, 0, sizeof(p));
  RelTable table;
  fa_status_t st = prepare_rel(h, bias, stream, &p.rel, &table);
  if (st != FA_OK) return st;
  const int64_t groups = d->B * d->N;
  p.splits = rows_splits(groups, h->max_keys, h->num_sms);
  const size_t count = align_up((size_t)groups * sizeof(unsigned int), 256);
  st = ensure_buffer(h, &h->rel.rows,
                     count + (p.splits > 1 ? rows_part_bytes((int)d->D, groups, p.splits) : 0));
  if (st != FA_OK) return st;
  p.done = static_cast<unsigned int*>(h->rel.rows.ptr);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(h->rel.rows.ptr) + count);
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.seqs = reinterpret_cast<const SeqRec*>(static_cast<uint8_t*>(h->d_ws) + kHeaderBytes);
  operand_strides(d, d->Sq, &p.q_sb, &p.q_sh, &p.q_st);
  operand_strides(d, d->Skv, &p.k_sb, &p.k_sh, &p.k_st);
  p.l_sb = d->layout == FA_TND ? 0 : d->N * d->Sq;
  p.l_sh = d->Sq;
  p.B = (int32_t)d->B;
  p.N = (int32_t)d->N;
  p.scale_log2 = (float)(d->scale * 1.4426950408889634073599);
  const cudaError_t e = launch_rows((int)d->D, h->max_rows, p, table, stream);
  if (e != cudaSuccess) return cuda_fail(e, "few-row launch");
  return FA_OK;
}

}  // namespace

namespace fa {

// Element strides (batch, head, token) of Q/O or K/V in the handle's layout.
void operand_strides(const fa_desc_t* d, int64_t S, int64_t* sb, int64_t* sh, int64_t* st) {
  const int64_t N = d->N, D = d->D;
  switch (d->layout) {
    case FA_BNSD:
      *sb = N * S * D;
      *sh = S * D;
      *st = D;
      break;
    case FA_BSND:
      *sb = S * N * D;
      *sh = D;
      *st = N * D;
      break;
    default:  // TND: batch stride unused (tokens are global)
      *sb = 0;
      *sh = D;
      *st = N * D;
      break;
  }
}

}  // namespace fa

namespace {

fa_status_t encode_maps(fa_handle_t h, const void* q, const void* k, const void* v) {
  const void* ptrs[3] = {q, k, v};
  const fa_desc_t* d = &h->desc;
  for (int i = 0; i < 3; ++i) {
    if (h->tm_key[i] == ptrs[i]) continue;
    const int64_t S = (i == 0) ? d->Sq : d->Skv;
    int64_t sb, sh, st;
    operand_strides(d, S, &sb, &sh, &st);
    const bool tnd = d->layout == FA_TND;
    // dims (D, S, N, B); TND: (D, T, N, 1) with a dummy (valid) batch stride
    const int64_t b_extent = tnd ? 1 : d->B;
    const int64_t b_stride = tnd ? (S > 0 ? S : 1) * d->N * d->D : sb;
    if (!encode_operand_map(&h->tm[i], ptrs[i], d->D, S, d->N, b_extent, st, sh, b_stride)) {
      h->tm_key[i] = nullptr;
      return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed for operand %d", i);
    }
    h->tm_key[i] = ptrs[i];
  }
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status_t fa_create(const fa_desc_t* desc, fa_handle_t* out) {
  clear_error();
  if (!out) return fail(FA_ERR_NULLPTR, "out is NULL");
  *out = nullptr;
  fa_status_t st = validate_desc(desc);
  if (st != FA_OK) return st;
  if (env_flag("FA_TEST_FAIL_ALLOC")) return fail(FA_ERR_ALLOC, "handle (test hook)");
  fa_handle_t h = new (std::nothrow) fa_handle_s();
  if (!h) return fail(FA_ERR_ALLOC, "handle");
  h->desc = *desc;
  if (const char* t = std::getenv("FA_WAIT_TIMEOUT_MS")) {
    long long ms = std::atoll(t);
    if (ms > 0) h->timeout_ns = (uint64_t)ms * 1000000ull;
  }
  if (env_flag("FA_TEST_DROP_FIRST_Q")) h->debug_flags |= kDebugDropFirstQ;
  *out = h;
  return FA_OK;
}

}  // extern "C"

namespace {

// fa_fwd and fa_fwd_with_ranges. `ranges` (or null): the dense-mask
// occupancy of this mask, already computed by fa_mask_occupancy.
fa_status_t forward(fa_handle_t h, const void* q, const void* k, const void* v,
                    const uint8_t* atten_mask, const int32_t* ranges, const float* slopes,
                    const fa_relbias_t* bias, const int64_t* prefix, const int64_t* actual_seq_qlen,
                    const int64_t* actual_seq_kvlen, void* o, float* lse, void* cuda_stream) try {
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (!q || !k || !v || !o || !lse) return fail(FA_ERR_NULLPTR, "q, k, v, o and lse are required");
  const fa_desc_t* d = &h->desc;
  if (d->alibi != FA_ALIBI_NONE && !slopes)
    return fail(FA_ERR_PARAM_INVALID,
                "the handle names an ALiBi variant: call fa_fwd_alibi with the slopes");
  if (slopes && ((uintptr_t)slopes & 3u))
    return fail(FA_ERR_PARAM_INVALID, "slopes must be 4-byte aligned");
  const int m = d->sparse_mode;
  const int has_mask = (m <= 1) && atten_mask != nullptr;
  fa_status_t st = validate_call(d, prefix, actual_seq_qlen, actual_seq_kvlen, has_mask);
  if (st != FA_OK) return st;
  const uintptr_t align = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o;
  if (align & 15u) return fail(FA_ERR_PARAM_INVALID, "q, k, v and o must be 16-byte aligned");
  if ((uintptr_t)lse & 3u) return fail(FA_ERR_PARAM_INVALID, "lse must be 4-byte aligned");
  st = bind_device(h);
  if (st != FA_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  bool capturing = false;
  st = bias ? refuse_capture(stream) : stream_capturing(stream, &capturing);
  if (st != FA_OK) return st;
  FailedCall failed{h, stream, !capturing};
  st = refresh_plan(h, prefix, actual_seq_qlen, actual_seq_kvlen, has_mask, capturing, stream);
  if (st != FA_OK) return st;
  if (h->n_items == 0) return FA_OK;  // no query rows: nothing to write
  if (bias && few_rows(h->max_rows, d->B * d->N, h->num_sms)) {
    st = forward_rows(h, q, k, v, bias, o, lse, stream);
    if (st != FA_OK) return st;
    failed.armed = false;
    return record_call(h, capturing, stream);
  }
  st = encode_maps(h, q, k, v);
  if (st != FA_OK) return st;

  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.tm_q = h->tm[0];
  p.tm_k = h->tm[1];
  p.tm_v = h->tm[2];
  uint8_t* ws = static_cast<uint8_t*>(h->d_ws);
  p.err_word = reinterpret_cast<unsigned int*>(ws);
  p.seqs = reinterpret_cast<const SeqRec*>(ws + kHeaderBytes);
  p.items = reinterpret_cast<const WorkItem*>(
      ws + kHeaderBytes + align_up((size_t)h->n_seqs * sizeof(SeqRec), 256));
  p.o = o;
  p.lse = lse;
  p.mask = atten_mask;
  operand_strides(d, d->Sq, &p.o_sb, &p.o_sh, &p.o_st);
  if (d->layout == FA_TND) {
    p.l_sb = 0;
    p.l_sh = d->Sq;
  } else {
    p.l_sb = d->N * d->Sq;
    p.l_sh = d->Sq;
  }
  if (has_mask) {
    const int64_t plane = d->Sq * d->Skv;
    p.m_si = d->Skv;
    p.m_sb = (d->mask_kind == FA_MASK_SS) ? 0 : (d->mask_kind == FA_MASK_B1SS ? plane : d->N * plane);
    p.m_sh = (d->mask_kind == FA_MASK_BNSS) ? plane : 0;
  }
  if (has_mask) {
    // Reduce the mask to per-sub-tile key-tile ranges (unless the caller
    // already did), then rebuild the work list from them on the device, all
    // on the same stream ahead of the attention kernel.
    OccParams a;
    std::memset(&a, 0, sizeof(a));
    occupancy_shape(&a, h->geo0, mask_planes(d, has_mask));
    a.mask = atten_mask;
    SchedParams sp;
    std::memset(&sp, 0, sizeof(sp));
    sp.B = (int32_t)d->B;
    sp.N = (int32_t)d->N;
    sp.nblk = (int32_t)((d->Sq + kBlockM - 1) / kBlockM);
    if ((int64_t)sp.B * sp.N * sp.nblk != h->n_items)
      return fail(FA_ERR_DEVICE, "internal: dense-mask work list has %d items, expected %lld",
                  h->n_items, (long long)sp.B * sp.N * sp.nblk);
    // The list, item_tr and the pre-pass's table are rewritten every call:
    // a kernel of this handle on another stream may still be reading them.
    st = order_after_last(h, capturing, stream);
    if (st != FA_OK) return st;
    if (ranges != nullptr) {
      a.ranges = reinterpret_cast<TileRange*>(const_cast<int32_t*>(ranges));
    } else {
      occupancy_bind(&a, ws + occupancy_offset(h->n_seqs, h->n_items));
      cudaError_t e = launch_occupancy(a, h->num_sms, stream);
      if (e != cudaSuccess) return cuda_fail(e, "occupancy pre-pass launch");
    }
    sp.ranges = a.ranges;
    sp.items = const_cast<WorkItem*>(p.items);
    sp.item_tr = reinterpret_cast<TileRange*>(ws + item_tr_offset(h->n_seqs, h->n_items));
    sp.occ_sb = (d->mask_kind == FA_MASK_SS) ? 0 : (d->mask_kind == FA_MASK_B1SS ? 1 : d->N);
    sp.occ_sh = (d->mask_kind == FA_MASK_BNSS) ? 1 : 0;
    sp.n_qt = a.n_qt;
    sp.sq = (int32_t)d->Sq;
    sp.n_kt = a.n_kt;
    cudaError_t e = launch_schedule(sp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "work list schedule launch");
    p.item_tr = sp.item_tr;
  }
  if (!has_mask)
    p.item_tr = reinterpret_cast<const TileRange*>(ws + item_tr_offset(h->n_seqs, h->n_items));
  p.n_items = h->n_items;
  // Closed-form lists (descending lpt_key: items without a key tile last)
  // with many items per CTA are claimed at run time.
  if (!has_mask && claims_items(h->n_items, h->num_sms)) {
    p.claim = reinterpret_cast<unsigned int*>(ws + kClaimOffset);
    p.claim_done = reinterpret_cast<unsigned int*>(ws + kClaimOffset + 64);
  }
  if (d->alibi != FA_ALIBI_NONE) {
    p.slopes = slopes;
    p.alibi = d->alibi;
  }
  if (bias) {
    RelTable table;
    st = prepare_rel(h, bias, stream, &p.rel, &table);
    if (st != FA_OK) return st;
    const cudaError_t er = launch_rel_expand(table, nullptr, 0, stream);
    if (er != cudaSuccess) return cuda_fail(er, "bias expansion launch");
  }
  p.tnd = d->layout == FA_TND ? 1 : 0;
  p.scale_log2 = (float)(d->scale * 1.4426950408889634073599);
  p.debug_flags = h->debug_flags;
  p.timeout_ns = h->timeout_ns;
  const int grid = h->n_items < h->num_sms ? h->n_items : h->num_sms;
  const char* why = nullptr;
  cudaError_t e = launch_fwd((int)d->D, p, grid, stream, &why);
  if (e != cudaSuccess) {
    if (why) return fail(FA_ERR_UNSUPPORTED, "launch refused: %s", why);
    return cuda_fail(e, "kernel launch");
  }
  failed.armed = false;
  return record_call(h, capturing, stream);
} catch (const std::exception& e) {
  return host_exception(e);
}

}  // namespace

extern "C" {

fa_status_t fa_fwd(fa_handle_t h, const void* q, const void* k, const void* v,
                   const uint8_t* atten_mask, const int64_t* prefix,
                   const int64_t* actual_seq_qlen, const int64_t* actual_seq_kvlen, void* o,
                   float* lse, void* cuda_stream) {
  clear_error();
  return forward(h, q, k, v, atten_mask, nullptr, nullptr, nullptr, prefix, actual_seq_qlen,
                 actual_seq_kvlen, o, lse, cuda_stream);
}

fa_status_t fa_fwd_alibi(fa_handle_t h, const void* q, const void* k, const void* v,
                         const float* slopes, const int64_t* prefix,
                         const int64_t* actual_seq_qlen, const int64_t* actual_seq_kvlen,
                         void* o, float* lse, void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (!slopes) return fail(FA_ERR_NULLPTR, "slopes is NULL");
  if (h->desc.alibi == FA_ALIBI_NONE)
    return fail(FA_ERR_PARAM_INVALID, "fa_fwd_alibi needs a handle with an ALiBi variant");
  return forward(h, q, k, v, nullptr, nullptr, slopes, nullptr, prefix, actual_seq_qlen,
                 actual_seq_kvlen, o, lse, cuda_stream);
}

fa_status_t fa_fwd_relbias(fa_handle_t h, const void* q, const void* k, const void* v,
                           const fa_relbias_t* bias, const int64_t* prefix,
                           const int64_t* actual_seq_qlen, const int64_t* actual_seq_kvlen,
                           void* o, float* lse, void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  fa_status_t st = validate_rel(&h->desc, bias);
  if (st != FA_OK) return st;
  return forward(h, q, k, v, nullptr, nullptr, nullptr, bias, prefix, actual_seq_qlen,
                 actual_seq_kvlen, o, lse, cuda_stream);
}

fa_status_t fa_fwd_with_ranges(fa_handle_t h, const void* q, const void* k, const void* v,
                               const uint8_t* atten_mask, const int32_t* ranges, void* o,
                               float* lse, void* cuda_stream) {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (h->desc.sparse_mode > 1 || h->desc.mask_kind == FA_MASK_NONE || !atten_mask)
    return fail(FA_ERR_PARAM_INVALID,
                "fa_fwd_with_ranges needs sparse_mode 0 or 1 with a mask kind and atten_mask");
  if (!ranges) return fail(FA_ERR_NULLPTR, "ranges is NULL");
  if ((uintptr_t)ranges & 15u) return fail(FA_ERR_PARAM_INVALID, "ranges must be 16-byte aligned");
  return forward(h, q, k, v, atten_mask, ranges, nullptr, nullptr, nullptr, nullptr, nullptr, o, lse,
                 cuda_stream);
}

fa_status_t fa_fwd_paged(fa_handle_t h, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, int64_t num_blocks, int32_t block_size,
                         int32_t max_blocks, const int64_t* prefix, const int64_t* actual_seq_qlen,
                         const int64_t* actual_seq_kvlen, void* o, float* lse,
                         void* cuda_stream) try {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  if (!q || !k_cache || !v_cache || !block_table || !o || !lse)
    return fail(FA_ERR_NULLPTR, "q, k_cache, v_cache, block_table, o and lse are required");
  const fa_desc_t* d = &h->desc;
  fa_status_t st = validate_paged(d, prefix, actual_seq_qlen, actual_seq_kvlen, num_blocks,
                                  block_size, max_blocks);
  if (st != FA_OK) return st;
  const uintptr_t align = (uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)o;
  if (align & 15u)
    return fail(FA_ERR_PARAM_INVALID, "q, k_cache, v_cache and o must be 16-byte aligned");
  if (((uintptr_t)lse | (uintptr_t)block_table) & 3u)
    return fail(FA_ERR_PARAM_INVALID, "lse and block_table must be 4-byte aligned");
  st = bind_device(h);
  if (st != FA_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  bool capturing = false;
  st = stream_capturing(stream, &capturing);
  if (st != FA_OK) return st;
  FailedCall failed{h, stream, !capturing};
  const int64_t D = d->D;
  std::vector<int64_t> key = {-2, block_size, max_blocks};
  key.insert(key.end(), actual_seq_qlen, actual_seq_qlen + d->B);
  key.insert(key.end(), actual_seq_kvlen, actual_seq_kvlen + d->B);
  if (d->sparse_mode == 5 || d->sparse_mode == 6) key.insert(key.end(), prefix, prefix + d->B);
  const int32_t hpu = paged_heads_per_unit(d->N, (int)D);
  const size_t part_unit = (size_t)hpu * kPagedRows * (size_t)(D + 4) * sizeof(float);
  if (!h->plan_valid || key != h->plan_key) {
    if (capturing) return no_plan_in_capture();
    std::vector<SeqRec> recs = decode_geometry(d, prefix, actual_seq_qlen, actual_seq_kvlen, 0);
    std::vector<PagedGroup> groups;
    std::vector<PagedUnit> units;
    int32_t max_rows = 0;
    for (const SeqRec& r : recs) max_rows = std::max(max_rows, std::min(r.sq, (int32_t)kPagedRows));
    build_paged(d, recs, paged_slots((int)D, max_rows, hpu, h->num_sms), hpu, &groups, &units);
    if (units.size() > (size_t)0x7fffffff || groups.size() > (size_t)0x7fffffff)
      return fail(FA_ERR_UNSUPPORTED, "too many paged work units");
    const size_t seq_bytes = align_up(recs.size() * sizeof(SeqRec), 256);
    const size_t group_bytes = align_up(groups.size() * sizeof(PagedGroup), 256);
    const size_t payload = seq_bytes + group_bytes + units.size() * sizeof(PagedUnit);
    retire_captured(h);
    st = ensure_workspace(h, align_up(kHeaderBytes + payload, 256) + units.size() * part_unit,
                          stream);
    if (st != FA_OK) return st;
    st = ensure_pinned(&h->h_stage, &h->stage_bytes, h->stage_done, payload);
    if (st != FA_OK) return st;
    st = order_after_last(h, false, stream);
    if (st != FA_OK) return st;
    uint8_t* hs = static_cast<uint8_t*>(h->h_stage);
    std::memcpy(hs, recs.data(), recs.size() * sizeof(SeqRec));
    if (!groups.empty()) std::memcpy(hs + seq_bytes, groups.data(), groups.size() * sizeof(PagedGroup));
    if (!units.empty())
      std::memcpy(hs + seq_bytes + group_bytes, units.data(), units.size() * sizeof(PagedUnit));
    h->plan_valid = false;
    cudaError_t e = cudaMemcpyAsync(static_cast<uint8_t*>(h->d_ws) + kHeaderBytes, hs, payload,
                        cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(paged work list)");
    e = cudaEventRecord(h->stage_done, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaEventRecord");
    h->plan_key.swap(key);
    h->plan_valid = true;
    h->n_seqs = (int32_t)recs.size();
    h->n_groups = (int32_t)groups.size();
    h->n_units = (int64_t)units.size();
    h->n_items = 0;
    h->paged_rows = 0;
    for (const PagedGroup& g : groups) h->paged_rows = std::max(h->paged_rows, g.nrows);
  } else {
    // The partial buffer is rewritten.
    st = order_after_last(h, capturing, stream);
    if (st != FA_OK) return st;
  }
  if (h->n_groups == 0) return FA_OK;  // no query rows
  uint8_t* ws = static_cast<uint8_t*>(h->d_ws);
  const size_t seq_bytes = align_up((size_t)h->n_seqs * sizeof(SeqRec), 256);
  const size_t group_bytes = align_up((size_t)h->n_groups * sizeof(PagedGroup), 256);
  const size_t payload = seq_bytes + group_bytes + (size_t)h->n_units * sizeof(PagedUnit);
  PagedParams pp;
  std::memset(&pp, 0, sizeof(pp));
  pp.q = q;
  pp.k_cache = k_cache;
  pp.v_cache = v_cache;
  pp.block_table = block_table;
  pp.seqs = reinterpret_cast<const SeqRec*>(ws + kHeaderBytes);
  pp.groups = reinterpret_cast<const PagedGroup*>(ws + kHeaderBytes + seq_bytes);
  pp.units = reinterpret_cast<const PagedUnit*>(ws + kHeaderBytes + seq_bytes + group_bytes);
  pp.part = reinterpret_cast<float*>(ws + align_up(kHeaderBytes + payload, 256));
  pp.o = o;
  pp.lse = lse;
  pp.err_word = reinterpret_cast<unsigned int*>(ws);
  pp.num_blocks = num_blocks;
  pp.t_q = d->Sq;
  pp.n_units = h->n_units;
  pp.n_heads = (int32_t)d->N;
  pp.block_size = block_size;
  pp.max_blocks = max_blocks;
  pp.n_groups = h->n_groups;
  pp.heads_per_unit = hpu;
  pp.bs_shift = -1;
  if ((block_size & (block_size - 1)) == 0)
    for (int sh = 0; sh < 31; ++sh)
      if ((1 << sh) == block_size) pp.bs_shift = sh;
  pp.scale_log2 = (float)(d->scale * 1.4426950408889634073599);
  cudaError_t e = launch_paged((int)D, h->paged_rows, pp, stream);
  if (e != cudaSuccess) return cuda_fail(e, "paged kernel launch");
  failed.armed = false;
  return record_call(h, capturing, stream);
} catch (const std::exception& e) {
  return host_exception(e);
}

fa_status_t fa_mask_occupancy(const fa_desc_t* desc, const uint8_t* atten_mask,
                              uint8_t* tile_class, int32_t* ranges, void* cuda_stream) try {
  clear_error();
  if (!desc) return fail(FA_ERR_NULLPTR, "desc is NULL");
  if (!atten_mask || !tile_class || !ranges)
    return fail(FA_ERR_NULLPTR, "atten_mask, tile_class and ranges are required");
  fa_status_t st = validate_desc(desc);
  if (st != FA_OK) return st;
  if (desc->sparse_mode > 1 || desc->mask_kind == FA_MASK_NONE)
    return fail(FA_ERR_PARAM_INVALID, "the occupancy pre-pass needs sparse_mode 0 or 1 with a mask");
  st = validate_call(desc, nullptr, nullptr, nullptr, 1);
  if (st != FA_OK) return st;
  if ((uintptr_t)ranges & 15u) return fail(FA_ERR_PARAM_INVALID, "ranges must be 16-byte aligned");
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  if (major != 10 || minor != 0)
    return fail(FA_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library runs on sm_100 (B200)", dev,
                major, minor);
  std::vector<SeqRec> recs = decode_geometry(desc, nullptr, nullptr, nullptr, 1);
  if (recs.empty()) return FA_OK;
  OccParams a;
  std::memset(&a, 0, sizeof(a));
  occupancy_shape(&a, recs[0], mask_planes(desc, 1));
  a.mask = atten_mask;
  a.cls = tile_class;
  a.ranges = reinterpret_cast<TileRange*>(ranges);
  e = launch_occupancy(a, sms, static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return cuda_fail(e, "occupancy pre-pass launch");
  return FA_OK;
} catch (const std::exception& e) {
  return host_exception(e);
}

fa_status_t fa_sync_status(fa_handle_t h) try {
  clear_error();
  if (!h) return fail(FA_ERR_NULLPTR, "handle is NULL");
  cudaError_t e = h->any_call ? cudaEventSynchronize(h->last_call) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "cudaEventSynchronize");
  unsigned int word = 0;
  // The workspace (none before the first call, or when one since then found
  // no memory) and those that captured calls use.
  std::vector<void*> all = h->retired;
  if (h->d_ws != nullptr) all.push_back(h->d_ws);
  for (void* ws : all) {
    unsigned int w = 0;
    e = cudaMemcpy(&w, ws, sizeof(w), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(error word)");
    if (w == 0) continue;
    word |= w;
    // Clear the whole header: the error word and, should an aborted launch
    // have left them set, the claim counters.
    e = cudaMemset(ws, 0, kHeaderBytes);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the next call may not wait for it
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset(header)");
  }
  if (word == 0) return FA_OK;
  if (word & kErrTimeout)
    return fail(FA_ERR_TIMEOUT, "a device-side wait gave up (site %u); outputs are undefined",
                (word >> kErrWhereShift) & 0xffu);
  if (word & kErrBadBlock)
    return fail(FA_ERR_DEVICE,
                "a block_table entry was outside [0, num_blocks); its keys were left out");
  return fail(FA_ERR_DEVICE, "device error word 0x%08x", word);
} catch (const std::exception& e) {
  return host_exception(e);
}

fa_status_t fa_destroy(fa_handle_t h) {
  clear_error();
  if (!h) return FA_OK;
  if (h->any_call) cudaEventSynchronize(h->last_call);
  if (h->stage_done) cudaEventSynchronize(h->stage_done);
  if (h->d_ws) cudaFree(h->d_ws);
  for (void* ws : h->retired) cudaFree(ws);
  if (h->h_stage) cudaFreeHost(h->h_stage);
  if (h->stage_done) cudaEventDestroy(h->stage_done);
  if (h->last_call) cudaEventDestroy(h->last_call);
  release_training(h);
  delete h;
  return FA_OK;
}

}  // extern "C"
