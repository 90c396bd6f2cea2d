// shared_expand.cu -- the expanded form of shared latents: keys and values of every head from
// the cache rows, for sm_100a:  k[t][h] = c_t . W_K[h]^T,  v[t][h] = c_t . W_V[h]^T.
// This kernel: a CTA takes 16 tokens and 256 outputs, fp32 sums in order.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"

namespace stief {

__global__ void __launch_bounds__(256) stief_shared_expand_kernel(const SharedExpandArgs a) {
  __shared__ float rows[16][512];
  const int tid = threadIdx.x, t0 = blockIdx.x * 16, w = a.r + a.dr;
  const int end = min(a.N, a.kv_start[a.B]);
  if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && a.kv_start[a.B] > a.N) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
  for (int t = 0; t < 16; ++t) {
    const int i = t0 + t;
    if (i >= end) break;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.kv_start[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int pos = i - a.kv_start[lo], pi = pos / a.page_size;
    const int page = pi < a.max_pages ? a.block_table[(size_t)lo * a.max_pages + pi] : -1;
    const bool mapped = page >= 0 && page < a.num_pages;
    const uint16_t* src = a.pages + ((size_t)(mapped ? page : 0) * a.page_size + pos % a.page_size) * w;
    for (int c = tid; c < a.r; c += 256) rows[t][c] = mapped ? bf16_to_f32(src[c]) : 0.f;
    if (blockIdx.y == 0)
      for (int c = tid; c < a.dr; c += 256) a.pe[(size_t)i * a.dr + c] = mapped ? src[a.r + c] : (uint16_t)0;
  }
  __syncthreads();
  const int h = blockIdx.y;
  const uint16_t* W = (tid < 128 ? a.W_K : a.W_V) + ((size_t)h * 128 + (tid & 127)) * a.r;
  float acc[16] = {};
  for (int c = 0; c < a.r; ++c) {
    const float x = bf16_to_f32(W[c]);
    for (int t = 0; t < 16; ++t) acc[t] += x * rows[t][c];
  }
  uint16_t* dst = tid < 128 ? a.k : a.v;
  for (int t = 0; t < 16; ++t)
    if (t0 + t < end) dst[((size_t)(t0 + t) * a.H + h) * 128 + (tid & 127)] = f32_to_bf16_rn(acc[t]);
}

cudaError_t launch_shared_expand(const SharedExpandArgs& a, cudaStream_t stream) {
  stief_shared_expand_kernel<<<dim3((a.N + 15) / 16, a.H), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace stief
