// shared_latent.h -- argument blocks and launch entry points of the page planning and
// shared-latent operators.  Not a public header.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "stief.h"
#include "stief_internal.h"

namespace stief {

struct PlanArgs {
  const int32_t* new_tokens;
  const int32_t* seq_lens;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* slots;         // may be null
  int32_t* q_start;       // may be null
  int32_t* kv_start;      // may be null
  int32_t* seq_lens_out;  // may be null, may be seq_lens
  int32_t* free_count_out;  // may be free_count
  uint32_t* ticket;       // zero between calls
  uint32_t* dev_status;
  int B, num_pages, page_size, max_pages, max_tokens, device;
};
cudaError_t launch_page_plan(const PlanArgs& a, int sms, cudaStream_t stream);

struct SharedAppendArgs {
  const uint16_t* c;
  const uint16_t* pe;  // null when dr == 0
  const int32_t* slots;
  uint16_t* pages;
  uint32_t* dev_status;
  long long ld_c, ld_pe;  // row strides in elements
  int N, r, dr, device;
  long long num_slots;
};
cudaError_t launch_shared_append(const SharedAppendArgs& a, int sms, cudaStream_t stream);

struct SharedDecodeArgs {
  const uint16_t* q;
  const uint16_t* pages;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint16_t* out;
  float* workspace;
  uint32_t* dev_status;
  int B, Hq, r, dr, num_pages, page_size, max_pages, max_seq_len;
  float scale;
  int device, sms;
};
cudaError_t launch_shared_decode(const SharedDecodeArgs& a, cudaStream_t stream);
size_t shared_decode_workspace_bytes(int B, int Hq, int r);

struct SharedExpandArgs {
  const uint16_t* pages;
  const int32_t* block_table;
  const int32_t* kv_start;
  const uint16_t* W_K;
  const uint16_t* W_V;
  uint16_t* k;
  uint16_t* v;
  uint16_t* pe;  // null when dr == 0
  uint32_t* dev_status;
  int B, N, H, r, dr, num_pages, page_size, max_pages;
  int device, sms;
};
cudaError_t launch_shared_expand(const SharedExpandArgs& a, cudaStream_t stream);

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* pe;  // null when dr == 0
  const int32_t* q_start;
  const int32_t* kv_start;
  uint16_t* out;
  uint32_t* dev_status;
  int B, Hq, Hkv, dr, Nq, Nkv, max_q;
  float scale;
  int device, sms;
};
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_one_tile(const PrefillArgs& a, int pack, int split, cudaStream_t stream);

}  // namespace stief
