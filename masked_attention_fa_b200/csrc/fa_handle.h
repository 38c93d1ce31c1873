// The handle and the host helpers that the forward and the backward share.
#pragma once

#include <cuda_runtime.h>

#include <vector>

#include "../../include/fa.h"
#include "fa_bwd.h"
#include "fa_kernel.h"
#include "fa_plan.h"

namespace fa {

// A device buffer that only grows.
struct DeviceBuffer {
  void* ptr = nullptr;
  size_t bytes = 0;
};

// What the backward calls of a handle keep: the two work lists (built again
// when the lengths or prefixes change) and the scratch of one call.
struct BwdState {
  std::vector<int64_t> key;
  bool valid = false;
  int32_t n_q = 0, n_k = 0;  // query and key items
  int32_t n_g = 0;           // items of the dQ kernel
  int32_t tiles = 0, k_tiles = 0;  // query and key tiles per head, over all sequences
  // dS is written out (see launch_bwd) in these shares of the key and dQ
  // lists, each of a bounded number of tiles; empty: it is not.
  struct Chunk {
    int32_t k0, k1, g0, g1;
    int64_t tiles;
  };
  std::vector<Chunk> chunks;
  SeqRec geo0{};             // geometry of sequence 0
  // Pinned staging of the lists (beside the forward's, so that neither waits
  // for the other's upload) and the event of their last upload.
  void* stage = nullptr;
  size_t stage_bytes = 0;
  cudaEvent_t stage_done = nullptr;
  DeviceBuffer lists;        // [SeqRec x B][BwdItem x n_q][x n_k][x n_g][KeySpan x k_tiles N]
  DeviceBuffer scratch;      // row statistics, dense-mask ranges, bias sums
  DeviceBuffer spill;        // dS
};

// The bucket map of the relative position bias and the bias by distance.
struct RelState {
  std::vector<int32_t> bucket_of;
  DeviceBuffer map;
  DeviceBuffer ext;
  DeviceBuffer rows;  // few-row forward: counters and partial results
};

}  // namespace fa

struct fa_handle_s {
  fa_desc_t desc{};
  int device = -1;
  int num_sms = 0;
  // plan cache: the per-call arrays the current work list was built from
  std::vector<int64_t> plan_key;
  bool plan_valid = false;
  int32_t n_items = 0;
  int32_t n_seqs = 0;
  fa::SeqRec geo0{};  // geometry of sequence 0 (every sequence's, outside TND)
  int32_t max_rows = 0, max_keys = 0;  // longest sequence of the plan
  // paged K/V calls: [header][SeqRec x B][PagedGroup x n_groups][PagedUnit x
  // n_units] then the units' partial results (the plan key starts with -2)
  int32_t n_groups = 0;
  int64_t n_units = 0;
  int32_t paged_rows = 0;  // most query rows in one group
  // device workspace: [error word | claim counter at 128 | claim_done at 192 |
  // pad to 256 B][SeqRec x B][WorkItem x n]
  // [item_tr: 2 x TileRange per item] then, for a dense attenMask, the
  // occupancy pre-pass's ranges and classes
  void* d_ws = nullptr;
  size_t ws_bytes = 0;
  // pinned staging of the work list and the event of its last upload
  void* h_stage = nullptr;
  size_t stage_bytes = 0;
  cudaEvent_t stage_done = nullptr;
  cudaEvent_t last_call = nullptr;
  bool any_call = false;
  // A graph reads the workspace's list (see retire_captured); workspaces of
  // earlier lists that graphs read.
  bool captured = false;
  std::vector<void*> retired;
  // tensor maps of the last call's operands
  const void* tm_key[3] = {nullptr, nullptr, nullptr};
  CUtensorMap tm[3];
  uint64_t timeout_ns = 2000000000ull;
  uint32_t debug_flags = 0;
  fa::BwdState bwd;
  fa::RelState rel;
};

namespace fa {

constexpr size_t kHeaderBytes = 256;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool env_flag(const char* name);
fa_status_t cuda_fail(cudaError_t e, const char* what);
// Orders the handle's later calls after a call that fails half-way: what it
// has uploaded until then may still be on its way, and counts as uploaded.
struct FailedCall {
  fa_handle_t h;
  cudaStream_t stream;
  bool armed;
  ~FailedCall() {
    if (armed && cudaEventRecord(h->last_call, stream) == cudaSuccess) h->any_call = true;
  }
};
// Binds the handle to the current device at its first call and refuses
// calls with another device current.
fa_status_t bind_device(fa_handle_t h);
fa_status_t ensure_workspace(fa_handle_t h, size_t bytes, cudaStream_t stream);
// Grows a buffer to `bytes` (waiting for the handle's last call before the
// old one is freed); its contents are lost.
fa_status_t ensure_buffer(fa_handle_t h, DeviceBuffer* buf, size_t bytes);
fa_status_t stream_capturing(cudaStream_t stream, bool* capturing);
// Makes the stream wait for the handle's last call. Not in a capture: what
// orders a replay is the stream it is launched on, and an event recorded
// outside cannot be waited for inside.
fa_status_t order_after_last(fa_handle_t h, bool capturing, cudaStream_t stream);
// Notes the call that has just been enqueued as the handle's last. An event
// recorded in a capture could not be waited for outside: a captured call is
// none that later calls wait for.
fa_status_t record_call(fa_handle_t h, bool capturing, cudaStream_t stream);
void retire_captured(fa_handle_t h);
// Calls whose tables are uploaded or rebuilt per call are not captured into
// graphs: a replay would read another call's.
fa_status_t refuse_capture(cudaStream_t stream);
// Waits for the last upload from a pinned buffer and gives it at least `bytes`.
fa_status_t ensure_pinned(void** stage, size_t* have, cudaEvent_t done, size_t bytes);
// Frees what the backward and the relative position bias hold.
void release_training(fa_handle_t h);
// The handle's copy of the bias by distance (see RelBias) and what lays it out
// for this call: launch_rel_expand(*table), or the row statistics' launch.
fa_status_t prepare_rel(fa_handle_t h, const fa_relbias_t* bias, cudaStream_t stream, RelBias* out,
                        RelTable* table);
fa_status_t validate_rel(const fa_desc_t* d, const fa_relbias_t* bias);
int64_t mask_planes(const fa_desc_t* d, int has_mask);
std::vector<int64_t> make_key(const fa_desc_t* d, const int64_t* prefix, const int64_t* cu_q,
                              const int64_t* cu_kv, int has_mask);
void operand_strides(const fa_desc_t* d, int64_t S, int64_t* sb, int64_t* sh, int64_t* st);

}  // namespace fa
