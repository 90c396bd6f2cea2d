// shared_decode.cu -- absorbed attention of one query token a sequence over a cache of shared
// latent rows, for sm_100a.
//
// Every head's keys and values come from one row a token, c_t (r values) and k^R_t (dr values):
// with the key and value maps folded into the query and the output projection (the absorbed
// form), head h computes
//     s_t = scale * q~_h . [c_t | k^R_t],   p = softmax(s),   o~_h = sum_t p_t c_t.
// This kernel: one CTA a (head, sequence), tiles of 64 tokens, an online softmax in fp32.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"

namespace stief {

namespace {
constexpr int kTok = 64;
}

__global__ void __launch_bounds__(256) stief_shared_decode_kernel(const SharedDecodeArgs a) {
  __shared__ float qf[576], s[kTok];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w = a.r + a.dr;
  int L = a.seq_lens[b];
  if (L < 0 || L > a.max_seq_len) {
    if (tid == 0 && h == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    L = 0;
  }
  for (int i = tid; i < w; i += 256) qf[i] = bf16_to_f32(a.q[((size_t)b * a.Hq + h) * w + i]) * a.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int t0 = 0; t0 < L; t0 += kTok) {
    const int page = a.block_table[(size_t)b * a.max_pages + t0 / a.page_size];
    const bool mapped = page >= 0 && page < a.num_pages;
    const uint16_t* rows = a.pages + ((size_t)(mapped ? page : 0) * a.page_size + t0 % a.page_size) * w;
    const int n = min(kTok, L - t0);
    for (int t = warp; t < n; t += 8) {
      float d = 0.f;
      for (int i = lane; i < w; i += 32) d += qf[i] * (mapped ? bf16_to_f32(rows[(size_t)t * w + i]) : 0.f);
      for (int k = 16; k; k >>= 1) d += __shfl_xor_sync(~0u, d, k);
      if (lane == 0) s[t] = d;
    }
    __syncthreads();
    float mt = m;
    for (int t = 0; t < n; ++t) mt = fmaxf(mt, s[t]);
    const float f = m == mt ? 1.f : __expf(m - mt);
    l *= f, o[0] *= f, o[1] *= f;
    m = mt;
    for (int t = 0; t < n; ++t) {
      const float p = __expf(s[t] - m);
      l += p;
      for (int j = 0; j < 2; ++j)
        if (tid + 256 * j < a.r && mapped) o[j] += p * bf16_to_f32(rows[(size_t)t * w + tid + 256 * j]);
    }
    __syncthreads();
  }
  for (int j = 0; j < 2; ++j)
    if (tid + 256 * j < a.r)
      a.out[((size_t)b * a.Hq + h) * a.r + tid + 256 * j] = f32_to_bf16_rn(L > 0 ? o[j] / l : 0.f);
}

size_t shared_decode_workspace_bytes(int B, int Hq, int r) { return (size_t)256 + 0 * ((size_t)B * Hq * r); }

cudaError_t launch_shared_decode(const SharedDecodeArgs& a, cudaStream_t stream) {
  stief_shared_decode_kernel<<<dim3(a.Hq, a.B), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace stief
