// shared_api.cu -- the C ABI of page planning and the shared-latent operators: argument
// checking and launches.  Host code only.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "shared_latent.h"
#include "stief.h"

namespace {

constexpr int kMaxPlanSequences = 8192;  // the plan keeps 28 bytes a sequence in shared memory
constexpr int kPageQuantum = 64;
constexpr size_t kPlanWorkspace = 256;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

stief_status device_check(int* dev, int* sms) {
  bool sm100 = false;
  if (!stief::query_device(dev, sms, &sm100)) return STIEF_ERR_CUDA;
  return sm100 ? STIEF_OK : STIEF_ERR_UNSUPPORTED_DEVICE;
}

bool row_ok(int r, int dr) {
  return r >= 16 && r <= 512 && r % 16 == 0 && dr >= 0 && dr <= 64 && dr % 16 == 0;
}

// A pool of rows and its block table: pages of a multiple of 64 rows, fewer than 2^31 in all.
stief_status check_pool(int num_pages, int page_size, int max_pages) {
  if (num_pages < 1 || max_pages < 1 || page_size < kPageQuantum || page_size % kPageQuantum != 0)
    return STIEF_ERR_INVALID_ARG;
  if ((long long)num_pages * page_size >= (1LL << 31) || (long long)max_pages * page_size >= (1LL << 31))
    return STIEF_ERR_INVALID_ARG;
  return STIEF_OK;
}

stief_status launched(cudaError_t e) { return e == cudaSuccess ? STIEF_OK : STIEF_ERR_CUDA; }

}  // namespace

extern "C" {

size_t stief_plan_workspace_bytes(void) { return kPlanWorkspace; }

stief_status stief_plan_pages(const int32_t* new_tokens, const int32_t* seq_lens, int32_t* block_table,
                              const int32_t* free_pages, const int32_t* free_count, int32_t* slots,
                              int32_t* q_start, int32_t* kv_start, int32_t* seq_lens_out,
                              int32_t* free_count_out, void* workspace, size_t workspace_bytes, int B,
                              int num_pages, int page_size, int max_pages, int max_tokens,
                              uint32_t* dev_status, stief_stream_t stream) {
  if (!new_tokens || !seq_lens || !block_table || !free_pages || !free_count || !free_count_out)
    return STIEF_ERR_INVALID_ARG;
  if (B < 1 || B > kMaxPlanSequences || max_tokens < 0) return STIEF_ERR_INVALID_ARG;
  stief_status st = check_pool(num_pages, page_size, max_pages);
  if (st != STIEF_OK) return st;
  for (const void* p : {(const void*)new_tokens, (const void*)seq_lens, (const void*)block_table,
                        (const void*)free_pages, (const void*)free_count, (const void*)slots,
                        (const void*)q_start, (const void*)kv_start, (const void*)seq_lens_out,
                        (const void*)free_count_out})
    if (!aligned(p, 4)) return STIEF_ERR_ALIGNMENT;
  if (!aligned16(workspace)) return STIEF_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kPlanWorkspace) return STIEF_ERR_WORKSPACE;
  stief::PlanArgs a{};
  int sms = 0;
  st = device_check(&a.device, &sms);
  if (st != STIEF_OK) return st;
  a.new_tokens = new_tokens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.slots = slots;
  a.q_start = q_start;
  a.kv_start = kv_start;
  a.seq_lens_out = seq_lens_out;
  a.free_count_out = free_count_out;
  a.ticket = static_cast<uint32_t*>(workspace);
  a.dev_status = dev_status;
  a.B = B;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.max_tokens = max_tokens;
  return launched(stief::launch_page_plan(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

stief_status stief_append_shared_paged(const uint16_t* c_new, const uint16_t* pe_new, const int32_t* slots,
                                       uint16_t* pages, int N, int r, int dr, int64_t c_stride,
                                       int64_t pe_stride, int num_pages, int page_size,
                                       uint32_t* dev_status, stief_stream_t stream) {
  if (N < 0 || !row_ok(r, dr)) return STIEF_ERR_INVALID_ARG;
  stief_status st = check_pool(num_pages, page_size, 1);
  if (st != STIEF_OK) return st;
  if (N == 0) return STIEF_OK;
  if (!c_new || !slots || !pages || (dr > 0 && !pe_new)) return STIEF_ERR_INVALID_ARG;
  if (c_stride < r || (dr > 0 && pe_stride < dr)) return STIEF_ERR_INVALID_ARG;
  if (!aligned16(c_new) || !aligned16(pages) || !aligned(slots, 4) || c_stride % 8 != 0 ||
      (dr > 0 && (!aligned16(pe_new) || pe_stride % 8 != 0)))
    return STIEF_ERR_ALIGNMENT;
  stief::SharedAppendArgs a{};
  int sms = 0;
  st = device_check(&a.device, &sms);
  if (st != STIEF_OK) return st;
  a.c = c_new;
  a.pe = pe_new;
  a.slots = slots;
  a.pages = pages;
  a.dev_status = dev_status;
  a.ld_c = c_stride;
  a.ld_pe = dr > 0 ? pe_stride : 0;
  a.N = N;
  a.r = r;
  a.dr = dr;
  a.num_slots = (long long)num_pages * page_size;
  return launched(stief::launch_shared_append(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t stief_decode_shared_workspace_bytes(int B, int Hq, int r) {
  if (B < 1 || Hq < 1 || Hq > 256 || !row_ok(r, 0)) return 0;
  return stief::shared_decode_workspace_bytes(B, Hq, r);
}

stief_status stief_decode_shared_paged(const uint16_t* q, const uint16_t* pages, const int32_t* block_table,
                                       const int32_t* seq_lens, uint16_t* out, void* workspace,
                                       size_t workspace_bytes, int B, int Hq, int r, int dr, int num_pages,
                                       int page_size, int max_pages, int max_seq_len, float scale,
                                       uint32_t* dev_status, stief_stream_t stream) {
  if (!q || !pages || !block_table || !seq_lens || !out) return STIEF_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || Hq < 1 || Hq > 256 || !row_ok(r, dr) || max_seq_len < 0 || !std::isfinite(scale))
    return STIEF_ERR_INVALID_ARG;
  stief_status st = check_pool(num_pages, page_size, max_pages);
  if (st != STIEF_OK) return st;
  if (max_seq_len > (long long)max_pages * page_size) return STIEF_ERR_CAPACITY;
  // the work list counts 64-token tiles in 32 bits
  if ((long long)B * ((max_seq_len + 63LL) / 64) >= (1LL << 30)) return STIEF_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(pages) || !aligned16(out) || !aligned16(workspace) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return STIEF_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < stief::shared_decode_workspace_bytes(B, Hq, r)) return STIEF_ERR_WORKSPACE;
  stief::SharedDecodeArgs a{};
  st = device_check(&a.device, &a.sms);
  if (st != STIEF_OK) return st;
  a.q = q;
  a.pages = pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.workspace = static_cast<float*>(workspace);
  a.dev_status = dev_status;
  a.B = B;
  a.Hq = Hq;
  a.r = r;
  a.dr = dr;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.max_seq_len = max_seq_len;
  a.scale = scale;
  return launched(stief::launch_shared_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

stief_status stief_expand_shared_paged(const uint16_t* pages, const int32_t* block_table,
                                       const int32_t* kv_start, const uint16_t* W_K, const uint16_t* W_V,
                                       uint16_t* k, uint16_t* v, uint16_t* k_pe, int B, int N, int H, int d,
                                       int r, int dr, int num_pages, int page_size, int max_pages,
                                       uint32_t* dev_status, stief_stream_t stream) {
  if (B < 1 || B > 65535 || N < 0 || H < 1 || H > 256 || d != 128 || !row_ok(r, dr)) return STIEF_ERR_INVALID_ARG;
  stief_status st = check_pool(num_pages, page_size, max_pages);
  if (st != STIEF_OK) return st;
  if (N == 0) return STIEF_OK;
  if (!pages || !block_table || !kv_start || !W_K || !W_V || !k || !v || (dr > 0 && !k_pe))
    return STIEF_ERR_INVALID_ARG;
  if (!aligned16(pages) || !aligned16(W_K) || !aligned16(W_V) || !aligned16(k) || !aligned16(v) ||
      (dr > 0 && !aligned16(k_pe)) || !aligned(block_table, 4) || !aligned(kv_start, 4))
    return STIEF_ERR_ALIGNMENT;
  stief::SharedExpandArgs a{};
  st = device_check(&a.device, &a.sms);
  if (st != STIEF_OK) return st;
  a.pages = pages;
  a.block_table = block_table;
  a.kv_start = kv_start;
  a.W_K = W_K;
  a.W_V = W_V;
  a.k = k;
  a.v = v;
  a.pe = dr > 0 ? k_pe : nullptr;
  a.dev_status = dev_status;
  a.B = B;
  a.N = N;
  a.H = H;
  a.r = r;
  a.dr = dr;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  return launched(stief::launch_shared_expand(a, reinterpret_cast<cudaStream_t>(stream)));
}

stief_status stief_prefill_attention(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                     const uint16_t* k_pe, const int32_t* q_start, const int32_t* kv_start,
                                     uint16_t* out, int B, int Hq, int Hkv, int d, int dr, int Nq, int Nkv,
                                     int max_q_len, float scale, uint32_t* dev_status,
                                     stief_stream_t stream) {
  if (B < 1 || B > 65535 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 256 || d != 128 || dr < 0 || dr > 64 ||
      dr % 16 != 0 || Nq < 0 || Nkv < 0 || max_q_len < 0 || !std::isfinite(scale))
    return STIEF_ERR_INVALID_ARG;
  if (Nq == 0 || max_q_len == 0) return STIEF_OK;
  const long long tiles = ((max_q_len < Nq ? max_q_len : Nq) + 127LL) / 128;
  if (tiles * Hq * B >= (1LL << 31)) return STIEF_ERR_INVALID_ARG;  // one block each
  if (!q || !q_start || !kv_start || !out || (Nkv > 0 && (!k || !v || (dr > 0 && !k_pe))))
    return STIEF_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_pe) || !aligned16(out) ||
      !aligned(q_start, 4) || !aligned(kv_start, 4))
    return STIEF_ERR_ALIGNMENT;
  stief::PrefillArgs a{};
  const stief_status st = device_check(&a.device, &a.sms);
  if (st != STIEF_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.pe = dr > 0 ? k_pe : nullptr;
  a.q_start = q_start;
  a.kv_start = kv_start;
  a.out = out;
  a.dev_status = dev_status;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.dr = dr;
  a.Nq = Nq;
  a.Nkv = Nkv;
  a.max_q = max_q_len < Nq ? max_q_len : Nq;
  a.scale = scale;
  return launched(stief::launch_prefill(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
