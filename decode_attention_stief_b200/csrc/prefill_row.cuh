// prefill_row.cuh -- output rows of prompt attention by their definition, for rows that the tile's
// products cannot give.
//
// The second product adds P . V over all keys of a step, with weights of 0 for the keys that a row does
// not see; where such a key's value is NaN or infinite, 0 times it is NaN.  Such a row is known by a NaN
// in its output and computed anew, a warp a row, backwards over the keys of the tile's steps: first the
// unseen ones, which say in which dimensions the NaN may be theirs, then those it sees.  A lane scores a
// key of 32, then all lanes add the 32 values, four dimensions each.  The walk ends once no element is in
// question, or every one is NaN by a key that is seen.
//
// (Making the values of the diagonal's steps finite before their product would cost every call a look at
// them.)  All of it happens after the tile's work, from the arguments alone, so that the kernels keep no more
// than a bit a row for it: calls without a NaN take 0.1 us longer (77 tokens 6.28 -> 6.38 us, 8 prompts of 65 to
// 1500 and 8192 tokens as before).  That hangs on this form: called as a function, with a loop of its own over
// the unseen values, or with more loads in flight, it cost the kernels' main loops 2 to 5 %.  Bound by the
// latency of the rows' loads; 8192 tokens, 32 heads, position part: 0.54 ms without a NaN, 4.5 with one token
// of NaN in the middle, 5.6 with NaN from there on, 9.8 with nothing else.
#pragma once

#include "shared_latent.h"
#include "stief_device.cuh"
#include "umma.cuh"

namespace stief {

// NaN in a half of the result where that half of x, y or z is.  (Products past the largest value may
// give it too: the rows are looked at again.)
__device__ __forceinline__ uint32_t nan_of(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(y), "r"(z));
  return d;
}
__device__ __forceinline__ bool has_nan(uint32_t z) { return isnan(bf16lo(z)) || isnan(bf16hi(z)); }

__device__ __forceinline__ float dot8(uint4 x, uint4 y, float s) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(bf16hi(a[i]), bf16hi(b[i]), fmaf(bf16lo(a[i]), bf16lo(b[i]), s));
  return s;
}

// The NaN elements of the output of query row `qr` and head `h` that a value of keys [k0 + seen, k0 + walked)
// may have made, over keys [k0, k0 + seen) of KV head `hk`.  scale2: scale * log2(e), with its sign.  All
// lanes of a warp.
__device__ __forceinline__ void redo_row(const PrefillArgs& a, int qr, int h, int hk, int k0, int seen, int walked,
                                         float scale2) {
  const int lane = threadIdx.x & 31;
  uint2* at = reinterpret_cast<uint2*>(a.out + ((size_t)qr * a.Hq + h) * 128) + lane;
  const uint2 old = *at;
  float out[4] = {bf16lo(old.x), bf16hi(old.x), bf16lo(old.y), bf16hi(old.y)};
  bool odd[4], any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) any |= odd[e] = isnan(out[e]);
  if (!__any_sync(~0u, any)) return;
  const uint4* q = reinterpret_cast<const uint4*>(a.q + ((size_t)qr * a.Hq + h) * (128 + a.dr));
  float m = -1e30f, l = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f}, far[4] = {0.f, 0.f, 0.f, 0.f};  // far: of values not finite
  uint32_t unseen = 0;  // elements with an unseen value that is not finite
#pragma unroll 1
  for (int j0 = (walked - 1) / 32 * 32; j0 >= 0; j0 -= 32) {
    float s = -INFINITY;
    if (j0 + lane < seen) {
      const size_t row = (size_t)k0 + j0 + lane;
      const uint4* k = reinterpret_cast<const uint4*>(a.k + (row * a.Hkv + hk) * 128);
      float y = 0.f;
#pragma unroll 4
      for (int c = 0; c < 16; ++c) y = dot8(__ldg(q + c), __ldg(k + c), y);
      const uint4* pe = reinterpret_cast<const uint4*>(a.pe + row * a.dr);
#pragma unroll 1
      for (int c = 0; c < a.dr / 8; ++c) y = dot8(__ldg(q + 16 + c), __ldg(pe + c), y);
      s = y * scale2;
    }
    float top = fmaxf(m, s);
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float f = fast_exp2(m - top), p = fast_exp2(s - top);
    m = top;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] *= f;
#pragma unroll 1
    for (int t0 = 0; t0 < min(32, walked - j0); t0 += 8) {
      uint2 v[8];  // (loads in flight together: the walk is bound by their latency)
#pragma unroll
      for (int t = 0; t < 8; ++t)
        v[t] = __ldg(reinterpret_cast<const uint2*>(a.v + (((size_t)k0 + min(j0 + t0 + t, walked - 1)) * a.Hkv + hk) * 128) + lane);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float w = __shfl_sync(~0u, p, t0 + t);
        const float y[4] = {bf16lo(v[t].x), bf16hi(v[t].x), bf16lo(v[t].y), bf16hi(v[t].y)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (isfinite(y[e])) sum[e] = fmaf(w, y[e], sum[e]);
          else if (j0 + t0 + t < seen) far[e] += w * y[e];
          else unseen |= 1u << e;
        }
      }
    }
    bool done = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (j0 <= seen) odd[e] = odd[e] && (unseen >> e & 1u);  // (every unseen value has been looked at)
      done &= !odd[e] || isnan(far[e]) || isnan(sum[e]);
    }
    if (__all_sync(~0u, done)) break;
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (odd[e]) out[e] = isnan(sum[e]) || far[e] != 0.f ? sum[e] + far[e] : sum[e] / l;
  *at = make_uint2(pack_bf16x2_rn(out[0], out[1]), pack_bf16x2_rn(out[2], out[3]));
}

// Rows first_row + k * step of a tile (of `rows` rows, the bits k of `which`) whose outputs may hold a NaN
// that an unseen value left: the tile's number as the kernels count them, `keys` a step.
__device__ __forceinline__ void redo_rows(const PrefillArgs& a, int shift, int qtiles, unsigned tile, int rows, int keys,
                                              int first_row, int step, uint32_t which, float scale2) {
  const unsigned gb = (unsigned)((a.Hq >> shift) * a.B);
  const int groups = a.Hq >> shift, b = (int)(tile % gb) / groups, h0 = ((int)(tile % gb) % groups) << shift;
  const int begin = (qtiles - 1 - (int)(tile / gb)) * (rows >> shift), hk = h0 / (a.Hq / a.Hkv);
  const int q0 = __ldg(a.q_start + b), nq = __ldg(a.q_start + b + 1) - q0;
  const int k0 = __ldg(a.kv_start + b), n_k = __ldg(a.kv_start + b + 1) - k0;
  // keys of the tile's steps
  const long long last = min(nq, begin + (rows >> shift)) - 1 + (long long)n_k - nq + 1;
  const int walked = (int)min((long long)n_k, (last + keys - 1) / keys * keys);
#pragma unroll 1
  for (; which != 0; which &= which - 1) {
    const int row = first_row + (__ffs(which) - 1) * step, query = begin + (row >> shift);
    const int seen = (int)max(0LL, min((long long)n_k, (long long)query + n_k - nq + 1));
    if (query < nq && seen > 0 && seen < walked)
      redo_row(a, q0 + query, h0 + (row & ((1 << shift) - 1)), hk, k0, seen, walked, scale2);
  }
}

}  // namespace stief
