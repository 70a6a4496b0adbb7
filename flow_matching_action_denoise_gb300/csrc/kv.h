// Declarations shared by the paged prefix-cache operators (not part of the ABI).
#pragma once

#include "internal.h"

namespace fm {

// Error-word bit: a batch outside its bounds, or a token without a page.
constexpr int kErrBadBatch = 2;

// Host checks of the descriptors; FM_OK, or a status with the reason recorded.
int kv_check(const fm_kv_cache* c);
int kv_batch_check(const fm_kv_cache* c, const fm_kv_batch* b);
// The batch with max_tokens no larger than its packed rows: a loose bound costs no empty CTAs.
inline fm_kv_batch bounded_batch(fm_kv_batch b) {
  if (b.max_tokens > b.tokens) b.max_tokens = b.tokens;
  return b;
}

// Device address of the policy-free building blocks' error word on the current device, or nullptr.
int* standalone_error_word();

// Rows [tok_begin, tok_begin + rows) of every layer's prefix (keys [L][P][Hkv][Dh], values transposed
// [L][Hkv][Dh][p_pad]) from tokens [seq_tok, seq_tok + rows) of sequence `seq` of a cache with as many layers.
cudaError_t prefix_from_pages_launch(const fm_kv_cache& c, int seq, int seq_tok, int rows, __nv_bfloat16* kcache,
                                     __nv_bfloat16* vtcache, int P, int p_pad, int tok_begin, int* err, cudaStream_t st);

}  // namespace fm
