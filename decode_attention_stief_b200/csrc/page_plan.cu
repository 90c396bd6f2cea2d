// page_plan.cu -- block tables, slot maps and row offsets of a serving step, built on the GPU
// from the requests' lengths, for sm_100a.
//
// For sequence b with L_b cached tokens and T_b new ones (page size s, capacity C tokens):
//     q_start[b] = sum_{a<b} max(T_a, 0)
//     need_b = ceil((L_b + T_b) / s) - ceil(L_b / s)        new pages
//     P_b    = sum_{a<=b} need_a
// Page j < need_b of b is free_pages[n - 1 - (P_b - need_b + j)], n = *free_count: the top of
// the free stack first, in sequence order.  Token i of b is slot page(t / s) * s + t % s with
// t = L_b + i.  Three prefix sums over B (tokens, pages, lengths) decide everything; each
// thread then looks its own sequence up by bisection.
//
// What bounds it: latency (a few dependent loads and the scans, B <= 8192) for a decode step;
// the 4-byte slot stores for large prompts, which several CTAs share: every CTA repeats the
// scans in its own shared memory (cheaper than a second launch or a wait between CTAs) and
// writes its share of the table and the slots.  The lengths and the free count may be
// updated in place, so the last CTA to have read them (a ticket) writes the new ones.
//
// Measured: 64 sequences of one new token, 4.1 us; 512 prompts of 525,000 tokens (2.1 MB of slots),
// 8.5 us.
#include <cstdint>

#include "stief_device.cuh"
#include "shared_latent.h"

namespace stief {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kDirect = 4;  // tokens of a sequence that its own thread places
constexpr int kPer = 8;     // sequences a thread at most: 8192 over 1024 threads

// Exclusive prefix sum over the CTA (64-bit), and its total.  One barrier: every thread adds the
// sums of the warps before its own itself.  `warp_sums` is used once a kernel.
__device__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = (int)blockDim.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 8
  for (int i = 0; i < nwarps; ++i) {
    const long long w = warp_sums[i];
    if (i < warp) before += w;
    all += w;
  }
  *total = all;
  return before + incl - v;
}

__device__ __forceinline__ int sat32(long long v) { return v > 0x7fffffffLL ? 0x7fffffff : (int)v; }

// Largest i in [0, n) with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int upper_index(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) stief_page_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  __shared__ long long warp_sums[3][32];
  __shared__ int used_s, last_s;
  const int tid = threadIdx.x, nthreads = blockDim.x, B = a.B, ps = a.page_size;
  int* qs = plan_smem;        // [B] first flat token
  int* have = qs + B;         // [B] L_b, or -1 when refused
  int* first = have + B;      // [B] pages held before
  int* upto = first + B;      // [B] pages taken by the sequences before b
  int* need = upto + B;       // [B] new pages (0 when refused)
  int* tail = need + B;       // [B] page of token L_b when it is already held, else -1
  int* lead = tail + B;       // [B] first new page
  // Of several CTAs the last one writes everything but the slots, which the others share.
  const bool alone = gridDim.x == 1, clerk = blockIdx.x == gridDim.x - 1;
  const int per = (B + nthreads - 1) / nthreads, b0 = tid * per, b1 = min(B, b0 + per);  // per <= kPer
  if (tid == 0) used_s = 0;

  pdl_wait();
  pdl_launch_dependents();
  uint32_t bits = 0;
  int n = *a.free_count;
  const long long cap = (long long)a.max_pages * ps;
  // everything that the lengths alone say where to find is read before the first sum
  int T[kPer], L[kPer], page[kPer];
  auto pages_of = [&](int tokens) {  // ceil(tokens / ps), 0 <= tokens < 2^31
    const unsigned q = (unsigned)tokens / (unsigned)ps;
    return (int)q + (tokens != (int)q * ps);
  };
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (b0 + k >= b1) break;
    T[k] = a.new_tokens[b0 + k];
    L[k] = a.seq_lens[b0 + k];
  }
  long long sum = 0, total_tokens, total;
  uint32_t wanted = 0;  // bit k: the page must be there
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (b0 + k >= b1) break;
    // the page of the first new token, if it is held already
    page[k] = -1;
    if (L[k] >= 0 && L[k] < cap && T[k] > 0) {
      const int q = (int)((unsigned)L[k] / (unsigned)ps);
      if (L[k] != q * ps) {
        wanted |= 1u << k;
        page[k] = a.block_table[(size_t)(b0 + k) * a.max_pages + q];
      }
    }
    sum += T[k] > 0 ? T[k] : 0;
  }
  if (n < 0 || n > a.num_pages) {
    bits |= STIEF_DEV_BAD_LENGTH;
    n = n < 0 ? 0 : a.num_pages;
  }
  long long at = block_scan(sum, warp_sums[0], &total_tokens);
  sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (b0 + k >= b1) break;
    const int b = b0 + k;
    const bool bad = L[k] < 0 || L[k] > cap || T[k] < 0;
    qs[b] = sat32(at);
    at += T[k] > 0 ? T[k] : 0;
    const int f = bad ? 0 : pages_of(L[k]);
    bool full = !bad && ((long long)L[k] + T[k] > cap || (a.slots && at > a.max_tokens));
    if (!bad && (wanted >> k & 1u) && (page[k] < 0 || page[k] >= a.num_pages)) full = true;
    const int nd = bad || full ? 0 : pages_of(L[k] + T[k]) - f;
    if (bad) bits |= STIEF_DEV_BAD_LENGTH;
    if (full) bits |= STIEF_DEV_CAPACITY_OVERFLOW;
    have[b] = bad || full ? -1 : L[k];
    first[b] = f;
    need[b] = nd;
    tail[b] = page[k];
    sum += nd;
  }
  long long p = block_scan(sum, warp_sums[1], &total);
  int used = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (b0 + k >= b1) break;
    const int b = b0 + k;
    upto[b] = sat32(p);
    p += need[b];
    if (need[b] > 0) {
      if (p > n) {  // the free pages do not reach: refused, like every later one that needs a page
        bits |= STIEF_DEV_CAPACITY_OVERFLOW;
        have[b] = -1;
        need[b] = 0;
      } else {
        used = (int)p;
        // the first new page, which is all that most steps need
        if (clerk) {
          const int id = a.free_pages[n - 1 - upto[b]];
          lead[b] = id;  // (kept by the only CTA of a small step)
          a.block_table[(size_t)b * a.max_pages + first[b]] = id;
        }
      }
    }
  }
  if (used > 0) atomicMax(&used_s, used);
  // A decode step, a few tokens a sequence, needs nothing further: the sequence's thread places
  // them (all in its first new page or the one before).
  uint32_t work = 0;  // 1: new pages beyond the first of a sequence, 2: more tokens than that
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (b0 + k >= b1) break;
    const int b = b0 + k;
    if (need[b] > 1) work |= 1u;
    if (T[k] > kDirect) work |= 2u;
    if (a.slots && alone && T[k] > 0 && T[k] <= kDirect) {
      const int held = first[b] * ps;  // tokens up to here are in pages held before
      for (int i = 0; i < T[k]; ++i) {
        const int t = L[k] + i, pg = t < held ? tail[b] : lead[b];
        const int off = t < held ? t - (held - ps) : t - held;
        if (qs[b] < a.max_tokens - i)
          a.slots[qs[b] + i] = have[b] >= 0 && pg >= 0 && pg < a.num_pages ? pg * ps + off : -1;
      }
    }
  }
  // This CTA has read the lengths and the free count: the last one to have done so may write them.
  const bool more_pages = __syncthreads_or((int)(work & 1u)) != 0, more_tokens = __syncthreads_or((int)(work & 2u)) != 0;
  if (!alone) {
    if (tid == 0) {
      __threadfence();
      last_s = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
  }
  if (alone || last_s) {
    if (a.seq_lens_out) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (b0 + k < b1) a.seq_lens_out[b0 + k] = have[b0 + k] >= 0 ? L[k] + T[k] : L[k];
    }
    if (tid == 0) {
      *a.free_count_out = n - used_s;
      if (!alone) *a.ticket = 0u;
    }
  }
  if (clerk) {
    if (bits) report(a.dev_status, bits);
    if (a.q_start) {
      for (int b = b0; b < b1; ++b) a.q_start[b] = qs[b];
      if (tid == 0) a.q_start[B] = sat32(total_tokens);
    }
    if (a.kv_start) {
      int after[kPer];
      sum = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        after[k] = b0 + k >= b1 ? 0 : have[b0 + k] >= 0 ? L[k] + T[k] : L[k] < 0 || L[k] > cap ? 0 : L[k];
        sum += after[k];
      }
      long long kv = block_scan(sum, warp_sums[2], &total);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (b0 + k < b1) a.kv_start[b0 + k] = sat32(kv);
        kv += after[k];
      }
      if (tid == 0) a.kv_start[B] = sat32(total);
    }
  }

  // the other new table entries: one warp a sequence
  const int lane = tid & 31;
  if (more_pages)
    for (int b = (int)blockIdx.x * (nthreads >> 5) + (tid >> 5); b < B; b += (int)gridDim.x * (nthreads >> 5))
      for (int j = 1 + lane; j < need[b]; j += 32)
        a.block_table[(size_t)b * a.max_pages + first[b] + j] = a.free_pages[n - 1 - (upto[b] + j)];

  // slots: the CTA's share of the flat tokens
  if (!a.slots) return;
  if (alone && !more_tokens) {
    for (long long i = total_tokens + tid; i < a.max_tokens; i += nthreads) a.slots[i] = -1;
    return;
  }
  // (one bisection and one division for four tokens; 16-byte stores if the array allows them)
  const bool wide = (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0;
  if (!alone && clerk) return;
  const long long writers = alone ? 1 : gridDim.x - 1;
  for (long long i0 = 4LL * ((long long)blockIdx.x * nthreads + tid); i0 < a.max_tokens; i0 += 4LL * nthreads * writers) {
    int s[4] = {-1, -1, -1, -1};
    if (i0 < total_tokens) {
      int b = upper_index(qs, B, (int)i0), page = -1, at = ps;  // at: offset in the page, ps: look up
      int next = b + 1 < B ? qs[b + 1] : sat32(total_tokens), pi = 0;
      bool fresh = true;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = (int)i0 + e;
        if (i >= total_tokens || i >= a.max_tokens) break;
        while (i >= next) {  // (sequences without new tokens are passed over)
          ++b;
          next = b + 1 < B ? qs[b + 1] : sat32(total_tokens);
          fresh = true;
        }
        if (have[b] < 0) continue;
        if (fresh) {
          const int t = have[b] + (i - qs[b]);
          pi = t / ps;
          at = t - pi * ps;
        } else if (++at == ps) {
          at = 0;
          ++pi;
          fresh = true;
        }
        if (fresh)
          page = pi < first[b] ? tail[b] : a.free_pages[n - 1 - (upto[b] + pi - first[b])];
        fresh = false;
        s[e] = page >= 0 && page < a.num_pages ? page * ps + at : -1;
      }
    }
    if (wide && i0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e < a.max_tokens) a.slots[i0 + e] = s[e];
    }
  }
}

cudaError_t launch_page_plan(const PlanArgs& a, int sms, cudaStream_t stream) {
  // No more warps than the sequences need: they meet at every sum.
  const int threads = a.B <= 256 && a.max_tokens <= 1024 ? 256 : a.B <= 512 * kPer ? 512 : kPlanThreads;
  long long grid = a.slots ? (a.max_tokens + 4LL * threads - 1) / (4 * threads) : 1;
  if (grid < 1) grid = 1;
  if (grid > 2 * sms - 1) grid = 2 * sms - 1;
  if (grid > 1) ++grid;  // the one that writes the rest
  const int smem = 7 * 4 * a.B;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(stief_page_plan_kernel), a.device, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, stief_page_plan_kernel, a);
  // a decode that follows must not look a page up before this kernel has written the table
  if (e == cudaSuccess) mark_stream_compress(a.device, stream, true);
  return e;
}

}  // namespace stief
