// Launch interface of the few-row forward with the learned relative position
// bias.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_bwd.h"
#include "fa_internal.h"
#include "fa_kernel.h"

namespace fa {

constexpr int kFewRows = 4;  // query rows of a sequence it can take
// Whether a call of `groups` = B * N pairs whose sequences have at most
// max_rows query rows takes it. One row: always (8 x 16 heads against 8,191
// keys of dimension 128: 96 us against 120 by the tensor-core kernel, calls back
// to back; 1 x 16 heads 29 against 113). More rows: the sums over a key's threads
// add up (4 rows on the first: 190 against 120 us), and only what the split brings
// where the pairs leave SMs idle is worth it (2 x 8 heads, 4 rows, 2,000 keys of
// dimension 64: 20 against 40 us, caches flushed). The grid, groups times
// at most 128 splits, stays below 2^31.
inline bool few_rows(int32_t max_rows, int64_t groups, int num_sms) {
  return groups < (1 << 24) && (max_rows <= 1 || (max_rows <= kFewRows && 2 * groups <= num_sms));
}

struct RowsParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  const SeqRec* seqs;
  float* part;               // [B][N][splits][kFewRows][D + 4], unused with one split
  unsigned int* done;        // [B][N] counters, 0
  RelBias rel;
  int64_t q_sb, q_sh, q_st;  // element strides of Q and O: batch, head, token
  int64_t k_sb, k_sh, k_st;  // of K and V
  int64_t l_sb, l_sh;        // of lse
  int32_t B, N, splits;
  float scale_log2;
};

// Splits of the longest sequence's keys, for a grid that fills num_sms SMs.
int32_t rows_splits(int64_t groups, int64_t max_keys, int num_sms);
size_t rows_part_bytes(int D, int64_t groups, int32_t splits);
// Lays the bias out, sets the counters to 0 and runs the forward; max_rows is
// the most query rows of a sequence.
cudaError_t launch_rows(int D, int max_rows, const RowsParams& p, const RelTable& table,
                        cudaStream_t stream);

}  // namespace fa
