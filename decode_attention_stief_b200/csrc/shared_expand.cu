// shared_expand.cu -- the expanded form of shared latents: keys and values of every head from
// the cache rows, for sm_100a:  k[t][h] = c_t . W_K[h]^T,  v[t][h] = c_t . W_V[h]^T.
//
// A matrix product of [tokens x r] with the heads' [256 x r] weights (W_K[h] over W_V[h]).  What
// bounds it: 4 r H 128 operations a token on the tensor cores, or, for small r, the 512 H bytes
// a token that it writes.
//
// Two CTAs on neighbouring SMs work as a pair: a unit is 256 tokens (a row tile of 128 in each
// CTA) x one head, one product of M = 256, N = 256 with 256 accumulator columns in each CTA's
// TMEM, two of them in turn.  Each CTA brings half of the head's weights, the first W_K[h], the
// second W_V[h]: with both halves in one CTA (M = 128) the weights alone asked for 64 bytes a
// cycle and SM from L2, and 4096 tokens x 32 heads took 36 us.  Units are dealt out evenly, in
// order, heads innermost: a CTA keeps its rows in shared memory (two row tiles where they fit) and
// streams the weights' 64-column chunks through a ring.
//   warp 0: TMA producer; warp 1 of the first CTA: MMA issuer; warps 4-7 store the keys, warps 8-11
//   the values, through 4 KB (or 2) of shared memory each by TMA, or, where the sequence ends inside,
//   by eight lanes a token (stored by the thread that holds it, 32 bytes at a time, the weights'
//   copies waited behind the stores; all of it by eight lanes a token, r 128 took 17.8 us, by TMA
//   17.2, r 256 24.5 and 23.5).  The unit of head 0 also copies the position values.
// Row tiles begin at multiples of 128 tokens of their sequence, hence at multiples of 64 rows of
// a page: two copies bring 64 rows each.
//
// Measured: 4096 tokens x 32 heads, r 512: 36.8 us, 0.93 PFLOP/s (29 to 33 us where the 67 MB of output
// stay in L2), the tensor cores busy for 59 %; 128 heads:
// 116 us, 1.19 PFLOP/s; 3 sequences of 33 to 501 tokens, 8 heads, r 96: 7.4 us.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"
#include "umma.cuh"

namespace stief {

namespace {

constexpr int kRows = 128;                  // tokens a row tile
constexpr uint32_t kAtomA = kRows * 128;    // 128 rows x 64 columns
constexpr uint32_t kStageB = 128 * 128;     // 128 weight rows x 64 columns
constexpr int kThreads = 384;
constexpr int kMaxStages = 6;
constexpr uint32_t kTmemCols = 512;

struct Args {
  CUtensorMap mc;        // pool [rows][w], box 64 x 64
  CUtensorMap mwk, mwv;  // W [H * 128][r], box 64 x 128
  CUtensorMap mk, mv;    // outputs [N][H][128], box 64 columns x 1 x out_rows tokens
  SharedExpandArgs a;
  int chunks, na, nb;    // 64-column chunks of r, row tiles and weight chunks held
  int out_rows;          // tokens that an output warp stages at a time: 32 or 16
#ifdef STIEF_TEST_HOOKS
  uint32_t stall;     // test build: bytes expected of the first copy that none delivers
#endif
};

struct Layout {
  uint32_t b, out, bars, total;
};
__host__ __device__ constexpr Layout layout_of(int chunks, int na, int nb, int out_rows) {
  Layout l{};
  l.b = (uint32_t)(na * chunks) * kAtomA;
  l.out = l.b + (uint32_t)nb * kStageB;
  l.bars = l.out + (uint32_t)(8 * out_rows) * 128;
  l.total = l.bars + 8 * (2 * kMaxStages + 12);
  return l;
}
// One CTA an SM (it holds all of the tensor memory).  The smallest layout takes 161 KB; with fewer
// than six weight chunks another one did not fit.
static_assert(2 * (layout_of(1, 2, kMaxStages, 32).total + 1024) > 228 * 1024 &&
                  2 * (kMaxSmemPerBlock - 1024 - kStageB) > 228 * 1024,
              "two CTAs do not fit an SM");

// Rows [s0, s1) of sequence b (none if kv_start is not ascending from 0 within the outputs).
__device__ __forceinline__ void rows_of(const SharedExpandArgs& a, int b, int& s0, int& s1) {
  s0 = __ldg(a.kv_start + b);
  s1 = min(__ldg(a.kv_start + b + 1), a.N);
  if (s0 < 0 || s1 < s0) s1 = s0 = 0;
}

struct Unit {
  int b, j, h;         // sequence, row tile of it (none, for the second CTA at the end: len == 0), head
  int s0, len;         // first output row, rows of the sequence
  bool new_tile, last_of_tile;
};
// Walks a CTA's units; every warp role of both CTAs walks the same way, the second CTA one row
// tile further on.
struct Walk {
  const SharedExpandArgs& a;
  int b, j, h;
  long long left;
  bool fresh = true;
  // to the row tile `step` tiles on
  __device__ void move(int step) {
    j += step;
    while (b < a.B) {
      int s0, s1;
      rows_of(a, b, s0, s1);
      const int n = (s1 - s0 + kRows - 1) / kRows;
      if (j < n) return;
      j -= n;
      ++b;
    }
  }
  __device__ bool next(Unit& u) {
    if (left <= 0) return false;
    int s0 = 0, s1 = 0;
    if (b < a.B) rows_of(a, b, s0, s1);
    u.b = b;
    u.j = j;
    u.h = h;
    u.s0 = s0;
    u.len = s1 - s0;
    u.new_tile = fresh || h == 0;
    fresh = false;
    --left;
    if (++h == a.H) {
      h = 0;
      move(2);
    }
    u.last_of_tile = h == 0 || left == 0;
    return true;
  }
};

struct Ring {
  int n, st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) stief_shared_expand_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sum[kThreads / 32], start_b, start_j;
  const SharedExpandArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Layout lay = layout_of(p.chunks, p.na, p.nb, p.out_rows);
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  // (the full barriers and d_empty that count are the leader's; the others are each CTA's own)
  uint64_t* b_full = reinterpret_cast<uint64_t*>(smem + lay.bars);
  uint64_t* b_empty = b_full + kMaxStages;
  uint64_t* a_full = b_empty + kMaxStages;  // [2]
  uint64_t* a_empty = a_full + 2;           // [2]
  uint64_t* d_full = a_full + 4;            // [2] an accumulator is complete
  uint64_t* d_empty = a_full + 6;           // [2] it has been read
  uint64_t* drain = a_full + 8;

#ifdef STIEF_TEST_HOOKS
  const uint32_t stall = p.stall;
#else
  constexpr uint32_t stall = 0u;
#endif
  if ((smem_u32(smem) & 1023u) != 0) {  // (the same in both CTAs)
    if (tid == 0) report(a.dev_status, STIEF_DEV_SMEM_ALIGN);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], 1);
      mbar_init(&a_empty[i], 1);
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 16);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_tensormap(&p.mc);
    prefetch_tensormap(&p.mwk);
    prefetch_tensormap(&p.mwv);
    prefetch_tensormap(&p.mk);
    prefetch_tensormap(&p.mv);
  }

  // (tensor memory only after the dependency wait, and dependents only once it is held, as in
  // shared_decode.cu)
  pdl_wait();
  if (warp == 1) tmem_alloc_pair(&tmem_slot, kTmemCols);
  // where this CTA's units begin: a prefix sum of the sequences' row tiles
  const int per_thread = (a.B + kThreads - 1) / kThreads, c0 = min(a.B, tid * per_thread), c1 = min(a.B, c0 + per_thread);
  int sum = 0;
  for (int b = c0; b < c1; ++b) {
    int s0, s1;
    rows_of(a, b, s0, s1);
    sum += (s1 - s0 + kRows - 1) / kRows;
    if (blockIdx.x == 0 && (s0 != __ldg(a.kv_start + b) || s1 != __ldg(a.kv_start + b + 1)))
      report(a.dev_status, STIEF_DEV_BAD_LENGTH);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total_tiles = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == warp) incl += total_tiles;
    total_tiles += warp_sum[i];
  }
  const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
  const long long total = (long long)((total_tiles + 1) / 2) * a.H, per = (total + pairs - 1) / pairs;
  const long long u0 = (long long)pair * per;
  const long long count = u0 >= total ? 0 : min(per, total - u0);
  const int tile0 = 2 * (int)(u0 / a.H);
  if (count > 0 && tile0 >= incl - sum && tile0 < incl) {
    int at = incl - sum, b = c0;
    for (;; ++b) {
      int s0, s1;
      rows_of(a, b, s0, s1);
      const int n = (s1 - s0 + kRows - 1) / kRows;
      if (tile0 < at + n) break;
      at += n;
    }
    start_b = b;
    start_j = tile0 - at;
  }
  // (also: the barriers of both CTAs are initialised, and both have their tensor memory)
  cluster_sync();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  Walk walk{a, count > 0 ? start_b : 0, count > 0 ? start_j : 0, (int)(u0 - (long long)(tile0 / 2) * a.H), count};
  if (count > 0 && !leader) walk.move(1);
  Unit u;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    // The leader expects both CTAs' bytes on its barriers.  (The second CTA's copies may land first:
    // it asks for a slot only when the products with its last use are done, that is in the phase
    // that the leader opens.)
    if (elect_one()) {
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      Ring ra{p.na}, rb{p.nb};
      int na = 0, nb = 0;  // tiles and chunks requested
      bool ok = true;
      while (ok && walk.next(u)) {
        if (u.new_tile) {
          if (na >= p.na && !(ok = mbar_wait_bounded(&a_empty[ra.st], ra.ph ^ 1u, a.dev_status))) break;
          const uint32_t bar = in_cta(&a_full[ra.st], 0);
          if (leader) mbar_arrive_expect_tx(&a_full[ra.st], 2u * p.chunks * kAtomA + (na == 0 ? stall : 0u));
          uint8_t* dst = smem + (uint32_t)(ra.st * p.chunks) * kAtomA;
          for (int half = 0; half < 2; ++half) {
            const int pos = u.j * kRows + half * 64, pi = pos / a.page_size;
            const int page = pos < u.len && pi < a.max_pages ? __ldg(a.block_table + (size_t)u.b * a.max_pages + pi) : -1;
            // rows past the pool read as zeros: so do those of a page that is not mapped
            const int row = page >= 0 && page < a.num_pages ? page * a.page_size + pos % a.page_size
                                                            : a.num_pages * a.page_size;
            for (int c = 0; c < p.chunks; ++c)
              tma_load_2d_pair(dst + (uint32_t)c * kAtomA + half * (kAtomA / 2), &p.mc, 64 * c, row, bar, once);
          }
          ++na;
          ra.next();
        }
        for (int c = 0; c < p.chunks; ++c, ++nb, rb.next()) {
          if (nb >= p.nb && !(ok = mbar_wait_bounded(&b_empty[rb.st], rb.ph ^ 1u, a.dev_status))) break;
          uint8_t* dst = smem + lay.b + (uint32_t)rb.st * kStageB;
          const uint32_t bar = in_cta(&b_full[rb.st], 0);
          if (leader) mbar_arrive_expect_tx(&b_full[rb.st], 2 * kStageB);
          tma_load_2d_pair(dst, leader ? &p.mwk : &p.mwv, 64 * c, u.h * 128, bar, keep);
        }
      }
      // every requested copy of both CTAs lands before their shared memory is released
      for (int k = max(0, na - p.na); leader && k < na; ++k)
        mbar_wait_bounded(&a_full[k % p.na], (uint32_t)((k / p.na) & 1), nullptr);
      for (int k = max(0, nb - p.nb); leader && k < nb; ++k)
        mbar_wait_bounded(&b_full[k % p.nb], (uint32_t)((k / p.nb) & 1), nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (leader && elect_one()) {
      const uint32_t id = idesc_bf16_f32(256, 256, false, false);
      const uint32_t a_addr = smem_u32(smem), b_addr = smem_u32(smem + lay.b);
      Ring ra{p.na}, rb{p.nb};
      uint32_t d = 0, dp = 0;  // accumulator, parity of its use
      int n = 0, st_a = 0;
      bool ok = true;
      while (ok && walk.next(u)) {
        if (u.new_tile) {
          if (!(ok = mbar_wait_bounded(&a_full[ra.st], ra.ph, a.dev_status))) break;
          st_a = ra.st;
          ra.next();
        }
        if (n >= 2 && !(ok = mbar_wait_bounded(&d_empty[d], dp ^ 1u, a.dev_status))) break;
        uint64_t da = sw128_desc(a_addr + (uint32_t)(st_a * p.chunks) * kAtomA);
        for (int c = 0; c < p.chunks; ++c, rb.next(), da += kAtomA >> 4) {
          if (!(ok = mbar_wait_bounded(&b_full[rb.st], rb.ph, a.dev_status))) break;
          tc_fence_after();
          const uint64_t db = sw128_desc(b_addr + (uint32_t)rb.st * kStageB);
          const int steps = min(4, (a.r - 64 * c) / 16);
          const uint32_t acc = tmem + d * 256u;
          umma_bf16_pair(acc, da, db, id, c > 0);
          if (steps > 1) umma_bf16_pair(acc, da + 2, db + 2, id, 1);
          if (steps > 2) umma_bf16_pair(acc, da + 4, db + 4, id, 1);
          if (steps > 3) umma_bf16_pair(acc, da + 6, db + 6, id, 1);
          umma_commit_pair(&b_empty[rb.st]);
        }
        if (!ok) break;
        if (u.last_of_tile) umma_commit_pair(&a_empty[st_a]);
        umma_commit_pair(&d_full[d]);
        d ^= 1u;
        if (d == 0) dp ^= 1u;
        ++n;
      }
      // (on the normal path the end of the last product, after a timeout a bounded chance to finish)
      umma_commit_pair(drain);
      mbar_wait_bounded(drain, 0, nullptr);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- output
    const int half = (warp - 4) >> 2, quad = warp & 3;  // 0: keys, 1: values
    const uint64_t once = l2_policy_evict_first();
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    uint16_t* const base = half ? a.v : a.k;
    uint32_t d = 0, dp = 0;
    while (walk.next(u)) {
      const int t = u.j * kRows + quad * 32 + lane;  // token of the sequence
      const bool live = t < u.len;
      if (u.h == 0 && half == 0 && a.dr > 0 && live) {
        const int pi = t / a.page_size;
        const int page = pi < a.max_pages ? __ldg(a.block_table + (size_t)u.b * a.max_pages + pi) : -1;
        const bool mapped = page >= 0 && page < a.num_pages;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.pages + ((size_t)(mapped ? page : 0) * a.page_size + t % a.page_size) * (a.r + a.dr) + a.r);
        uint4* dst = reinterpret_cast<uint4*>(a.pe + (size_t)(u.s0 + t) * a.dr);
        for (int c = 0; c < a.dr / 8; ++c) dst[c] = mapped ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      }
      if (!__all_sync(~0u, mbar_wait_bounded(&d_full[d], dp, a.dev_status))) break;
      tc_fence_after();
      const uint32_t col = tmem + lanes + d * 256u + (uint32_t)half * 128u;
      uint8_t* stage = smem + lay.out + (uint32_t)((warp - 4) * p.out_rows) * 128;
      const int row0 = u.j * kRows + quad * 32, piece = lane & 7;
      uint16_t* out = base + ((size_t)(u.s0 + row0) * a.H + u.h) * 128 + piece * 8;
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        uint32_t x[2][32];
        tmem_ld32(col + c, x[0]);
        tmem_ld32(col + c + 32, x[1]);
        tmem_wait_ld();
        for (int part = 0; part < 32; part += p.out_rows) {
          bulk_wait_read_all();  // (of the lane that stores; the others have no group)
          __syncwarp();
          if ((unsigned)(lane - part) < (unsigned)p.out_rows) {
#pragma unroll
            for (int e = 0; e < 64; e += 8) {  // in the 128-byte swizzle: a row's 16-byte pieces are rotated by its number
              uint4 y;
              y.x = pack_bf16x2_rn(__uint_as_float(x[e >> 5][(e & 31)]), __uint_as_float(x[e >> 5][(e & 31) + 1]));
              y.y = pack_bf16x2_rn(__uint_as_float(x[e >> 5][(e & 31) + 2]), __uint_as_float(x[e >> 5][(e & 31) + 3]));
              y.z = pack_bf16x2_rn(__uint_as_float(x[e >> 5][(e & 31) + 4]), __uint_as_float(x[e >> 5][(e & 31) + 5]));
              y.w = pack_bf16x2_rn(__uint_as_float(x[e >> 5][(e & 31) + 6]), __uint_as_float(x[e >> 5][(e & 31) + 7]));
              *reinterpret_cast<uint4*>(stage + (lane - part) * 128 + (((e >> 3) ^ (lane & 7)) << 4)) = y;
            }
          }
          if (row0 + part + p.out_rows <= u.len) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(half ? &p.mv : &p.mk, stage, c, u.h, u.s0 + row0 + part, once);
              bulk_commit();
            }
          } else {  // (the sequence ends inside: its rows only)
            __syncwarp();
            for (int r = lane >> 3; r < p.out_rows; r += 4) {
              const uint4 y = *reinterpret_cast<const uint4*>(stage + r * 128 + ((piece ^ (r & 7)) << 4));
              if (row0 + part + r < u.len)
                __stcs(reinterpret_cast<uint4*>(out + (size_t)(part + r) * a.H * 128 + c), y);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(in_cta(&d_empty[d], 0));
      d ^= 1u;
      if (d == 0) dp ^= 1u;
    }
    bulk_wait_read_all();  // (shared memory stays until the copies have read it)
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA is read, written or signalled by the other any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

cudaError_t launch_shared_expand(const SharedExpandArgs& a, cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.chunks = (a.r + 63) / 64;
#ifdef STIEF_TEST_HOOKS
  p.stall = test_stall_bytes();
#endif
  // two row tiles where at least three weight chunks fit beside them
  constexpr uint32_t kMost = kMaxSmemPerBlock - 1024;  // the static part, rounded up
  p.nb = 3;
  p.out_rows = 32;
  p.na = layout_of(p.chunks, 2, p.nb, 32).total <= kMost ? 2 : 1;
  while (p.nb < kMaxStages && layout_of(p.chunks, p.na, p.nb + 1, 32).total <= kMost) ++p.nb;
  // With one row tile in 128 KB the ring is short, and another chunk is worth more than whole stores
  // (128 heads at r 512: 116 us against 123); with two it is not (r 256: 27.0 us against 23.5).
  if (p.na == 1 && p.nb < kMaxStages && layout_of(p.chunks, 1, p.nb + 1, 16).total <= kMost) ++p.nb, p.out_rows = 16;
  const uint32_t smem = layout_of(p.chunks, p.na, p.nb, p.out_rows).total;
  if (smem > kMost) return cudaErrorInvalidValue;
  const uint64_t w = (uint64_t)(a.r + a.dr), r = (uint64_t)a.r;
  if (!encode_tiled_bf16_2d(&p.mc, a.pages, w, (uint64_t)a.num_pages * a.page_size, w * 2, 64, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_bf16_2d(&p.mwk, a.W_K, r, (uint64_t)a.H * 128, r * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_bf16_2d(&p.mwv, a.W_V, r, (uint64_t)a.H * 128, r * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_bf16_3d(&p.mk, a.k, {128, (uint64_t)a.H, (uint64_t)a.N}, {256, (uint64_t)a.H * 256}, {64, 1, (uint32_t)p.out_rows}) ||
      !encode_tiled_bf16_3d(&p.mv, a.v, {128, (uint64_t)a.H, (uint64_t)a.N}, {256, (uint64_t)a.H * 256}, {64, 1, (uint32_t)p.out_rows}))
    return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(stief_shared_expand_kernel), a.device, (int)smem);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be units
  const long long most = 2 * (((long long)a.N / kRows + a.B + 1) / 2) * a.H;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < a.sms ? most : a.sms / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, stief_shared_expand_kernel, p);
  // (a decode that takes the keys and values for a cache must not request their rows before they are there)
  if (e == cudaSuccess) mark_stream_compress(a.device, stream, true);
  return e;
}

}  // namespace stief
