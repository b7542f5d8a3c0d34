// Host-side helpers shared by the Uno entry points.
#pragma once

#include <cstdint>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "uno.h"

namespace uno_host {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// UNO_OK when the current device is an sm_100 part (compute capability 10.0),
// UNO_ERR_DEVICE otherwise, UNO_ERR_CUDA when the runtime cannot say. The
// answer is cached per device ordinal.
int check_device();

// cuTensorMapEncodeTiled (dualpath.cu), or null when the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Fault bits of the block attention's waits (block_attention.cu); the caller
// has synchronised the device.
int attention_fault_flags(bool clear, unsigned* flags);

// One inverse-CDF draw per softmax row (draft_sample.cu): row n of sequence b
// (logits + ((b * rows_per_seq + n) * V)) draws with the uniform of Philox
// word `word` of the block (b, row_key[b][n] or n, step); rows with
// n >= n_rows[b] are skipped and get -1 (n_rows null: all rows are used); a
// row with no finite logit gets -1. Arguments are checked by the caller.
struct RowDraws {
  const void* logits;
  int B, rows_per_seq, V, dtype;
  int seq_rows = 0;  // rows from one sequence's block to the next (0: rows_per_seq)
  const int32_t* row_key;
  const int32_t* n_rows;
  int word;
  uint64_t seed, step;
  int32_t* out;
};
int sample_rows(const RowDraws& r, cudaStream_t st);

// Sizes of a paged 8-bit cache and of the B x T new rows that meet it, as
// uno_kv_append and uno_block_attention accept them. Positions stay below 2^30,
// so that sums of a position and a page stay in 32 bits.
inline bool cache_sizes_ok(int B, int T, int Hkv, int D, int page, int width, int num_pages) {
  return B >= 0 && B <= 65535 && T >= 0 && T <= (1 << 20) && Hkv >= 1 && Hkv <= 1024 &&
         (D == 64 || D == 128) && (page == 16 || page == 32 || page == 64 || page == 128) &&
         width >= 0 && width <= (1 << 30) / page && num_pages >= 0;
}

}  // namespace uno_host
