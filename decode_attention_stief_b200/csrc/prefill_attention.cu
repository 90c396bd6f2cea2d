// prefill_attention.cu -- causal attention of ragged prompts over per-head keys and values, for
// sm_100a.  Query i of sequence b (n_q queries, n_k keys) sees keys j <= i + n_k - n_q:
//     o_i = softmax_j(scale * (q_i . k_j + q^R_i . k^R_j)) v_j.
// This kernel: one warp a query row, an online softmax in fp32.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"

namespace stief {

__global__ void __launch_bounds__(128) stief_prefill_kernel(const PrefillArgs a) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  const int q0 = a.q_start[b], nq = a.q_start[b + 1] - q0, k0 = a.kv_start[b], nk = a.kv_start[b + 1] - k0;
  if (q0 < 0 || nq < 0 || k0 < 0 || nk < 0 || q0 + nq > a.Nq || k0 + nk > a.Nkv || nq > a.max_q) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    return;
  }
  if (i >= nq) return;
  const int dq = 128 + a.dr, hk = h / (a.Hq / a.Hkv);
  const uint16_t* q = a.q + ((size_t)(q0 + i) * a.Hq + h) * dq;
  float x[6], o[4] = {}, m = -INFINITY, l = 0.f;
  for (int c = 0; c < 6; ++c) x[c] = lane + 32 * c < dq ? bf16_to_f32(q[lane + 32 * c]) * a.scale : 0.f;
  const int seen = min(nk, i + nk - nq + 1);
  for (int j = 0; j < seen; ++j) {
    const uint16_t* k = a.k + ((size_t)(k0 + j) * a.Hkv + hk) * 128;
    const uint16_t* v = a.v + ((size_t)(k0 + j) * a.Hkv + hk) * 128;
    float s = 0.f;
    for (int c = 0; c < 4; ++c) s += x[c] * bf16_to_f32(k[lane + 32 * c]);
    for (int c = 4; c < 6; ++c)
      if (lane + 32 * c < dq) s += x[c] * bf16_to_f32(a.pe[(size_t)(k0 + j) * a.dr + lane + 32 * (c - 4)]);
    for (int t = 16; t; t >>= 1) s += __shfl_xor_sync(~0u, s, t);
    const float mt = fmaxf(m, s), f = m == mt ? 1.f : __expf(m - mt), p = __expf(s - mt);
    m = mt;
    l = l * f + p;
    for (int c = 0; c < 4; ++c) o[c] = o[c] * f + p * bf16_to_f32(v[lane + 32 * c]);
  }
  for (int c = 0; c < 4; ++c)
    a.out[((size_t)(q0 + i) * a.Hq + h) * 128 + lane + 32 * c] = f32_to_bf16_rn(seen > 0 ? o[c] / l : 0.f);
}

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  stief_prefill_kernel<<<dim3((a.max_q + 3) / 4, a.Hq, a.B), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace stief
