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
#include <cstdint>

#include "stief_device.cuh"
#include "shared_latent.h"

namespace stief {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kSmallThreads = 256;

// Inclusive prefix sum over the CTA (64-bit), and its total.
__device__ long long block_scan(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = (int)blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < nwarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[nwarps - 1];
  const long long r = v + (warp > 0 ? warp_sums[warp - 1] : 0);
  __syncthreads();  // warp_sums may be reused
  return r;
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
  __shared__ long long warp_sums[32];
  __shared__ int used_s, last_s;
  const int tid = threadIdx.x, nthreads = blockDim.x, B = a.B, ps = a.page_size;
  int* qs = plan_smem;        // [B] first flat token
  int* have = qs + B;         // [B] L_b, or -1 when refused
  int* first = have + B;      // [B] pages held before
  int* upto = first + B;      // [B] pages taken by the sequences before b
  int* need = upto + B;       // [B] new pages (0 when refused)
  int* tail = need + B;       // [B] page of token L_b when it is already held, else -1
  const int per = (B + nthreads - 1) / nthreads, b0 = tid * per, b1 = min(B, b0 + per);
  if (tid == 0) used_s = 0;

  pdl_wait();
  pdl_launch_dependents();
  uint32_t bits = 0;
  int n = *a.free_count;
  if (n < 0 || n > a.num_pages) {
    bits |= STIEF_DEV_BAD_LENGTH;
    n = n < 0 ? 0 : a.num_pages;
  }
  long long sum = 0, total_tokens, total;
  for (int b = b0; b < b1; ++b) {
    const int T = a.new_tokens[b];
    if (T > 0) sum += T;
  }
  long long at = block_scan(sum, warp_sums, &total_tokens) - sum;
  const long long cap = (long long)a.max_pages * ps;
  sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int T = a.new_tokens[b], L = a.seq_lens[b];
    const bool bad = L < 0 || L > cap || T < 0;
    qs[b] = sat32(at);
    at += T > 0 ? T : 0;
    const int f = bad ? 0 : (L + ps - 1) / ps;
    int page = -1;
    bool full = !bad && ((long long)L + T > cap || (a.slots && at > a.max_tokens));
    if (!bad && !full && T > 0 && L < f * ps) {  // the first new token's page is held already
      page = a.block_table[(size_t)b * a.max_pages + f - 1];
      if (page < 0 || page >= a.num_pages) full = true;
    }
    const int nd = bad || full ? 0 : (int)(((long long)L + T + ps - 1) / ps) - f;
    if (bad) bits |= STIEF_DEV_BAD_LENGTH;
    if (full) bits |= STIEF_DEV_CAPACITY_OVERFLOW;
    have[b] = bad || full ? -1 : L;
    first[b] = f;
    need[b] = nd;
    tail[b] = page;
    sum += nd;
  }
  long long p = block_scan(sum, warp_sums, &total) - sum;
  sum = 0;
  int used = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = a.seq_lens[b];
    upto[b] = sat32(p);
    p += need[b];
    if (need[b] > 0) {
      if (p > n) {  // the free pages do not reach: refused, like every later one that needs a page
        bits |= STIEF_DEV_CAPACITY_OVERFLOW;
        have[b] = -1;
        need[b] = 0;
      } else {
        used = (int)p;
      }
    }
    sum += have[b] >= 0 ? (long long)L + a.new_tokens[b] : (L < 0 || L > cap) ? 0 : L;
  }
  if (used > 0) atomicMax(&used_s, used);
  __syncthreads();
  if (blockIdx.x == 0) {
    long long kv = block_scan(sum, warp_sums, &total) - sum;
    if (bits) report(a.dev_status, bits);
    for (int b = b0; b < b1; ++b) {
      const int L = a.seq_lens[b];
      if (a.q_start) a.q_start[b] = qs[b];
      if (a.kv_start) a.kv_start[b] = sat32(kv);
      kv += have[b] >= 0 ? (long long)L + a.new_tokens[b] : (L < 0 || L > cap) ? 0 : L;
    }
    if (tid == 0) {
      if (a.q_start) a.q_start[B] = sat32(total_tokens);
      if (a.kv_start) a.kv_start[B] = sat32(total);
    }
  }
  // Every read of the lengths and the free count of this CTA is done (the scan's barriers).
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      last_s = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
  }
  if (gridDim.x == 1 || last_s) {
    if (a.seq_lens_out)
      for (int b = b0; b < b1; ++b) {
        const int L = a.seq_lens[b];
        a.seq_lens_out[b] = have[b] >= 0 ? L + a.new_tokens[b] : L;
      }
    if (tid == 0) {
      *a.free_count_out = n - used_s;
      if (gridDim.x > 1) *a.ticket = 0u;
    }
  }

  // new table entries: one warp a sequence
  const int lane = tid & 31;
  for (int b = (int)blockIdx.x * (nthreads >> 5) + (tid >> 5); b < B; b += (int)gridDim.x * (nthreads >> 5))
    for (int j = lane; j < need[b]; j += 32)
      a.block_table[(size_t)b * a.max_pages + first[b] + j] = a.free_pages[n - 1 - (upto[b] + j)];

  // slots: the CTA's share of the flat tokens
  if (!a.slots) return;
  // (one bisection and one division for four tokens; 16-byte stores if the array allows them)
  const bool wide = (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0;
  for (long long i0 = 4LL * ((long long)blockIdx.x * nthreads + tid); i0 < a.max_tokens;
       i0 += 4LL * nthreads * gridDim.x) {
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
        if (fresh) page = pi < first[b] ? tail[b] : a.free_pages[n - 1 - (upto[b] + pi - first[b])];
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
  // a step of few sequences and tokens has little to scan: fewer warps meet sooner
  const int threads = a.B <= kSmallThreads && a.max_tokens <= 4 * kSmallThreads ? kSmallThreads : kPlanThreads;
  long long grid = a.slots ? (a.max_tokens + 4LL * threads - 1) / (4 * threads) : 1;
  if (grid < 1) grid = 1;
  if (grid > sms) grid = sms;
  const int smem = 6 * 4 * a.B;
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
