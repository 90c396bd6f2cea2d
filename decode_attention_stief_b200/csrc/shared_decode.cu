// shared_decode.cu -- absorbed attention of one query token a sequence over a cache of shared
// latent rows, for sm_100a.
//
// Every head's keys and values come from one row a token, [c_t (r values) | k^R_t (dr values)]:
// with the key and value maps folded into the query and the output projection (the absorbed
// form), head h computes
//     s_t = scale * q~_h . [c_t | k^R_t],   p = softmax(s),   o~_h = sum_t p_t c_t.
//
// What bounds it: the cache rows, 2 (r + dr) bytes a token, read once for all heads; at 128
// heads the products (2 (2 r + dr) a head and token) take as long on the tensor cores.
//
// Both products run on tcgen05 from the same shared-memory tile of 64 rows, which TMA brings in
// once: with the tile's rows in 128-byte swizzled atoms of 64 columns,
//     S [64 heads x 64 tokens]   = Q~ . tile^T        (tile K-major: k = row columns)
//     O~^T [128 dims x heads]   += tile^T . P^T       (tile MN-major: m = columns, k = tokens)
// Keeping O~ transposed makes the accumulator r / 128 tiles of one column a head: at 64 heads
// and r = 512 it takes 256 TMEM columns, half of the SM's, and the heads are the MMA's N, so
// few heads cost few cycles.  More than 64 heads are split over CTAs that run side by side and
// read the tiles through L2.
//   warp 0: TMA producer; warps 1 and 3: MMA issuers of S and of O~; warp 2: zeroes the rows past
//   the length in a sequence's last tile (they may hold NaN, and 0 * NaN is NaN); warps 4-7:
//   softmax, rescaling and the output.  S has two buffers, so the tensor cores work on the next
//   tile during a tile's softmax.
// The softmax's reference is the first tile's maximum of the head and moves only when a score
// passes it by more than 2^60 (rare: the accumulator is then rescaled in TMEM).  Weights and sums
// are floating-point numbers, so a large weight loses nothing, and the maximum of a tile, needed
// only for that test, is off the path from S to P.  Weights are rounded to bf16 once, and the sum
// l adds the rounded weights, so that a weight's rounding cancels where it dominates.  (What the
// rounding leaves, as a second bf16 operand, has no room: at 64 heads and rank 512 + 64 the queries, two
// tiles and one buffer of weights take 225 of the 227 KB.)
//
// Work: the 64-token tiles of all sequences, in order, are dealt out evenly: CTA c takes what lies
// in [c per, (c + 1) per), so ragged batches and single long sequences fill the GPU alike.  A
// sequence inside one CTA is finished there; the others leave (o~, m, l) in fp32 for a second
// kernel, launched as a programmatic dependent, which also writes the zeros of empty sequences.
//
// Measured (rank 512 + 64, outputs and caches larger than L2): one sequence of 32768 tokens, 32
// heads: 19.5 us, 1.9 TB/s over the call, of it 8 us at 4.7 TB/s for the rows (the rest is the
// start, the parts and their joining).  64 ragged sequences of up to 4096 tokens: 45 us at 32
// heads (3.8 TB/s), 49 at 64, 76 to 82 at 128.  There shared memory is what most is asked of: a tile's
// copies write 72 KB of it and its products read 240, 2500 cycles at 128 bytes a cycle, of the some
// 4000 that a tile takes with two in turn (64 heads' queries leave room for no third; the tensor
// cores are 45 % busy).  The way to memory is not: tiles brought into L2 two ahead, 77 us.  Nor is the
// softmax's length: with two warpgroups, half of a tile's tokens each, 77, and rank 96 29.0 for 28.0.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"
#include "umma.cuh"

namespace stief {

namespace {

// 64 tokens a tile (with 32, 82 against 76 us for 64 ragged sequences of up to 4096 tokens at 128
// heads, 47 against 37 us for 128 of 2000 at rank 256: a tile's fixed costs outweigh the deeper
// ring).
constexpr int kTok = 64;
constexpr uint32_t kAtom = kTok * 128;  // bytes of one 64-column atom of a tile
constexpr int kMaxHeads = 64;       // heads per CTA
constexpr int kMaxStages = 8;
constexpr int kThreads = 256;
constexpr int kSoftWarps = 4;       // warps 4..7, one per TMEM lane quadrant
constexpr int kMaxCtas = 160;       // the workspace holds two partial states for each
constexpr int kMinTiles = 2;        // tiles per CTA at least (fewer would only add merging)
constexpr uint32_t kSCol = 256;     // TMEM: O~^T at 0, S buffers at 256 and 320
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 60.f;    // log2 units a score may pass the reference by

struct Args {
  CUtensorMap mq;     // q [B * Hq][w], box 64 x heads
  CUtensorMap ma, mb; // pool rows in blocks of 64 columns: the blocks of the tile's two pieces (or
                      // one block at a time in ma, if w % 64 != 0)
  SharedDecodeArgs a;
  int w, na, sa, nm;  // row width, atoms loaded and atoms kept a tile, 128-dim tiles of o~
  int n0, m0;         // of those, the atoms and 128-dim tiles of the first piece
  int NH, groups, G;  // heads per CTA (a multiple of 16), head groups, CTAs per group
  int nstage;
  int whole_rows;     // w % 64 == 0: one copy brings a tile's atoms
  int whole;          // sequences are not split over CTAs, and there is no second kernel
  int direct;         // whole, and there is a CTA for each sequence: no sums over the lengths
  float scale2;       // |scale| * log2(e)
  int negate;         // scale < 0: the products are negated instead
#ifdef STIEF_TEST_HOOKS
  uint32_t stall;     // test build: bytes expected of the first copy that none delivers
#endif
};

struct Layout {
  uint32_t stages, p, ml, bars, total;
};
__host__ __device__ constexpr Layout layout_of(int na, int sa, int NH, int nstage) {
  Layout l{};
  l.stages = (uint32_t)na * NH * 128;  // q~ comes first
  l.p = l.stages + (uint32_t)(nstage * sa) * kAtom;
  l.ml = l.p + (uint32_t)NH * 128;
  l.bars = l.ml + 3 * kMaxHeads * 4;
  l.total = l.bars + 8 * (4 * kMaxStages + 16);
  return l;
}
// One CTA an SM (it holds all of the tensor memory).  The smallest ring of eight stages takes 133 KB;
// with fewer stages another one of at most nine atoms did not fit.
static_assert(2 * (layout_of(1, 2, 16, kMaxStages).total + 1024) > 228 * 1024 &&
                  2 * (kMaxSmemPerBlock - 1024 - 9 * kAtom) > 228 * 1024,
              "two CTAs do not fit an SM");

// Workspace: meta int2 [B] (padded to 256 bytes), (m, l) [slots][kMaxHeads], o~ [slots][NH][r].
__host__ __device__ inline size_t meta_bytes(int B) { return ((size_t)B * 8 + 255) / 256 * 256; }
__host__ __device__ inline size_t ml_bytes() { return (size_t)kMaxCtas * 2 * kMaxHeads * 8; }

__host__ __device__ inline int heads_per_cta(int Hq) {
  const int g = (Hq + kMaxHeads - 1) / kMaxHeads;
  return ((Hq + g - 1) / g + 15) / 16 * 16;
}

// Position in the ring of stages (counted up: a division by the stage count costs as much as
// several products of the pipeline it would sit in).
struct Ring {
  int n, st = 0;
  uint32_t ph = 0;  // parity of the stage's current use
  __device__ __forceinline__ void next() {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

__device__ __forceinline__ int valid_length(int L, int most) { return L < 0 || L > most ? 0 : L; }

__host__ __device__ __forceinline__ int tiles_of(int L) { return (L + kTok - 1) / kTok; }

// Tiles are dealt out by cost: a sequence counts kSegment tiles more than it has, for the query's
// copy and the output, placed before its first tile.
constexpr int kSegment = 3;
constexpr int kWholeTiles = 4, kDirectTiles = 6;  // tiles of sequences that are not split (see the launch)

// The stretch of one sequence's tiles [t0, t1) that a CTA works on.
struct Segment {
  int b, t0, t1, L;
  long long at;  // place of tile t0 on the scale by which tiles are dealt out
  bool first;    // the CTA's first
};
// Walks the CTA's tiles sequence by sequence; every warp role walks the same way.  `skip`: what is
// left of the sequence's extra cost, `off`: its next tile, `left`: what is left of the CTA's share,
// which begins at `at`.
struct Walk {
  const int32_t* lens;
  int most, B, b, off, skip;
  long long left, at;
  bool whole;    // sequences are not split: the CTA takes those that begin in its share
  bool first = true;
  __device__ bool next(Segment& s) {
    while (left > 0 && b < B) {
      const int L = valid_length(__ldg(lens + b), most), n = tiles_of(L);
      if (n == 0) {
        ++b;
        continue;
      }
      if (skip >= left && !whole) return false;
      left -= skip;
      at += skip;
      s.b = b;
      s.L = L;
      s.t0 = off;
      s.t1 = whole ? n : (int)min((long long)n, off + left);
      s.at = at;
      s.first = first;
      first = false;
      left -= s.t1 - s.t0;
      at += s.t1 - s.t0;
      ++b;
      off = 0;
      skip = kSegment;
      return true;
    }
    return false;
  }
};

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) stief_shared_decode_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t tmem_slot;
  __shared__ int warp_sum[8], start_b, start_off;
  const SharedDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = (int)blockIdx.x % p.groups, cta = (int)blockIdx.x / p.groups;
  const int h_base = group * p.NH, nheads = min(p.NH, a.Hq - h_base);
  const Layout lay = layout_of(p.na, p.sa, p.NH, p.nstage);
  float* sm_f = reinterpret_cast<float*>(smem + lay.ml);  // rescale factors
  float* sm_m = sm_f + kMaxHeads;
  float* sm_l = sm_m + kMaxHeads;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);  // [stages][2] a piece landed
  uint64_t* empty = full + 2 * kMaxStages;   // [stages][2] both products have read it
  uint64_t* q_full = empty + 2 * kMaxStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;         // [2] S of a tile is in TMEM
  uint64_t* p_full = q_full + 4;         // [2] P of a tile is in shared memory, its S has been read
  uint64_t* pv_done = q_full + 6;        // [2] O~ of a tile is added: its P and O~ are free
  uint64_t* o_free = q_full + 8;         // the segment's O~ has been read
  uint64_t* drain = q_full + 9;          // [2]
  uint64_t* partial = q_full + 11;       // a sequence's last tile is in and is not full
  uint64_t* tail = q_full + 12;          // its rows past the length are cleared
  volatile uint32_t* stop = reinterpret_cast<uint32_t*>(q_full + 13);  // the first issuer gave up

#ifdef STIEF_TEST_HOOKS
  const uint32_t stall = p.stall;
#else
  constexpr uint32_t stall = 0u;
#endif
  if ((smem_u32(smem) & 1023u) != 0) {  // swizzled operands need 1 KiB alignment
    if (tid == 0) report(a.dev_status, STIEF_DEV_SMEM_ALIGN);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2 * kMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&pv_done[i], 1);
      mbar_init(&drain[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_free, kSoftWarps);
    mbar_init(partial, 1);
    mbar_init(tail, 1);
    *stop = 0;
    fence_barrier_init();
    prefetch_tensormap(&p.mq);
    prefetch_tensormap(&p.ma);
    prefetch_tensormap(&p.mb);
  }

  // Tensor memory only after the dependency wait, and dependents only once it is held: an allocation
  // waits without a limit, and a CTA that has columns while it waits for another kernel must not
  // starve one of that kernel's.
  pdl_wait();
  if (warp == 1) tmem_alloc(&tmem_slot, kTmemCols);
  int per = 1, count = 0;  // the CTA's share begins at g0 and costs `count`
  long long g0 = 0;
  if (p.direct) {  // a CTA a sequence
    count = cta < a.B ? 1 : 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    if (count > 0 && group == 0 && tid == 64) {
      const int L = __ldg(a.seq_lens + cta);
      if (valid_length(L, a.max_seq_len) != L) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    }
  } else {
    // where this CTA's tiles begin: a prefix sum of the sequences' tile counts (warp 1, which allocates
    // meanwhile, has none of them)
    constexpr int kCounting = kThreads - 32;
    const int per_thread = (a.B + kCounting - 1) / kCounting, c0 = (warp > 1 ? tid - 32 : tid) * per_thread;
    const int c1 = warp == 1 ? c0 : min(a.B, c0 + per_thread);
    auto cost_of = [&](int b) {
      const int n = tiles_of(valid_length(__ldg(a.seq_lens + b), a.max_seq_len));
      return n > 0 ? n + kSegment : 0;
    };
    int sum = 0;
    for (int b = c0; b < c1; ++b) {
      const int L = __ldg(a.seq_lens + b);
      if (valid_length(L, a.max_seq_len) != L && blockIdx.x == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
      sum += cost_of(b);
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
    pdl_launch_dependents();
    int total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i == warp) incl += total;
      total += warp_sum[i];
    }
    per = (total + p.G - 1) / p.G;
    if (per < kMinTiles) per = kMinTiles;
    g0 = (long long)cta * per;
    count = g0 >= total ? 0 : (int)min((long long)per, total - g0);
    if (count > 0 && g0 >= incl - sum && g0 < incl) {  // one thread's sequences hold the first tile
      int at = incl - sum, b = c0;
      for (;; ++b) {
        const int n = cost_of(b);
        if (g0 < at + n) break;
        at += n;
      }
      start_b = b;
      start_off = (int)(g0 - at) - kSegment;  // negative: cost before the first tile
      if (p.whole && g0 > at) {  // that sequence is another CTA's: begin with the next
        start_b = b + 1;
        start_off = -kSegment - (at + cost_of(b) - (int)g0);
      }
    }
    __syncthreads();
  }
  const uint32_t tmem = tmem_slot;
  Walk walk{a.seq_lens, a.max_seq_len, a.B, 0, 0, 0, count, g0, p.whole != 0};
  if (p.direct) {
    walk.b = cta;
    walk.B = min(a.B, cta + 1);
  } else if (count > 0) {
    walk.b = start_b;
    walk.off = max(0, start_off);
    walk.skip = max(0, -start_off);
  }
  if (p.whole && !p.direct && count > 0) {  // (what lies before the first sequence of the share is another's)
    walk.left -= walk.skip - kSegment;
    walk.at += walk.skip - kSegment;
    walk.skip = kSegment;
  }
  Segment seg;

  const int pieces = p.n0 < p.na ? 2 : 1;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (count > 0 && elect_one()) {
      int got[2] = {0, 0};  // tiles of which the piece is requested
      const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
      int i = 0, segs = 0;
      Ring ring{p.nstage};
      bool ok = true;
      auto load_q = [&](int b, int segs) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(p.na * p.NH * 128) + (segs == 0 ? stall : 0u));
        for (int c = 0; c < p.na; ++c)
          tma_load_2d(smem + c * p.NH * 128, &p.mq, 64 * c, b * a.Hq + h_base, q_full, keep);
      };
      int page = 0;
      if (p.direct) {  // the query and the first page do not wait for the length
        page = __ldg(a.block_table + (size_t)cta * a.max_pages);
        load_q(cta, 0);
      }
      while (ok && walk.next(seg)) {
        if (segs > 0) ok = mbar_wait_ready(q_empty, (uint32_t)((segs - 1) & 1), a.dev_status);
        if (!ok) break;
        if (!p.direct) load_q(seg.b, segs);
        ++segs;
        const int32_t* entry = a.block_table + (size_t)seg.b * a.max_pages + seg.t0 * kTok / a.page_size;
        int in_page = seg.t0 * kTok % a.page_size;
        if (!p.direct) page = __ldg(entry);
        for (int t = seg.t0; t < seg.t1; ++t, ++i, ring.next()) {
          if (in_page == a.page_size) {
            in_page = 0;
            page = __ldg(++entry);
          }
          // rows past the pool read as zeros: so do those of a page that is not mapped
          const int row = page >= 0 && page < a.num_pages ? page * a.page_size + in_page
                                                          : a.num_pages * a.page_size;
          in_page += kTok;
          const int st = ring.st;
          uint8_t* dst = smem + lay.stages + (uint32_t)(st * p.sa) * kAtom;
          for (int piece = 0; piece < pieces; ++piece) {
            uint64_t* bar = &full[2 * st + piece];
            if (i >= p.nstage && !(ok = mbar_wait_ready(&empty[2 * st + piece], ring.ph ^ 1u, a.dev_status))) break;
            const int c0 = piece ? p.n0 : 0, c1 = piece ? p.na : p.n0;
            mbar_arrive_expect_tx(bar, (uint32_t)((c1 - c0) * kAtom));
            if (p.whole_rows) {
              tma_load_3d(dst + c0 * kAtom, piece ? &p.mb : &p.ma, 0, row, c0, bar, once);
            } else {
              for (int c = c0; c < c1; ++c) tma_load_2d(dst + c * kAtom, &p.ma, 64 * c, row, bar, once);
            }
            got[piece] = i + 1;
          }
          if (!ok) break;
        }
      }
      // every requested copy lands before the shared memory is released (bounded; on the normal
      // path nothing is outstanding: the MMA warp has waited for each)
      if (segs > 0 || p.direct) mbar_wait_ready(q_full, (uint32_t)(max(segs, 1) - 1) & 1u, nullptr);
      for (int piece = 0; piece < pieces; ++piece)
        for (int k = max(0, got[piece] - p.nstage); k < got[piece]; ++k)
          mbar_wait_ready(&full[2 * (k % p.nstage) + piece], (uint32_t)((k / p.nstage) & 1), nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    // (One thread runs the whole loop: under the products' shared-memory traffic every barrier
    // test, shuffle or vote between them costs 100 cycles and more.  The two products have a
    // thread each, so that neither waits for what the other one lacks.)
    if (elect_one()) {
      const uint32_t id_s = idesc_bf16_f32(64, kTok, false, false) | (p.negate ? 1u << 13 : 0u);  // (bit 13: -q~)
      const uint32_t stage0 = smem_u32(smem + lay.stages), stage_bytes = (uint32_t)p.sa * kAtom;
      const uint32_t q_step = (uint32_t)(p.NH * 128) >> 4;
      const int whole0 = min(p.n0, p.w / 64), whole1 = p.w / 64 - whole0, steps_left = p.w % 64 / 16;
      Ring ring{p.nstage};
      bool ok = true;
      int i = 0, segs = 0, tails = 0;
      while (ok && walk.next(seg)) {
        ok = mbar_wait_ready(q_full, (uint32_t)(segs & 1), a.dev_status);
        for (int t = seg.t0; ok && t < seg.t1; ++t, ++i, ring.next()) {
          const bool last = (t + 1) * kTok > seg.L;  // not full: what lies past the length is cleared first
          if (i >= 2 && !(ok = mbar_wait_ready(&p_full[i & 1], (uint32_t)((i >> 1) & 1) ^ 1u, a.dev_status))) break;
          if (!(ok = mbar_wait_ready(&full[2 * ring.st], ring.ph, a.dev_status))) break;
          if (last) {
            if (pieces > 1 && !(ok = mbar_wait_ready(&full[2 * ring.st + 1], ring.ph, a.dev_status))) break;
            mbar_arrive(partial);
            if (!(ok = mbar_wait_ready(tail, (uint32_t)(tails & 1), a.dev_status))) break;
            ++tails;
          }
          tc_fence_after();
          // (descriptors advance by additions, four steps at a time: building each one took longer
          // than its product)
          const uint32_t d = tmem + kSCol + (uint32_t)(i & 1) * kTok;
          uint64_t dq = sw128_desc(smem_u32(smem)), dt = sw128_desc(stage0 + (uint32_t)ring.st * stage_bytes);
          uint32_t acc = 0;
          auto blocks = [&](int n) {
            for (int c = 0; c < n; ++c) {
              umma_bf16(d, dq, dt, id_s, acc);
              umma_bf16(d, dq + 2, dt + 2, id_s, 1);
              umma_bf16(d, dq + 4, dt + 4, id_s, 1);
              umma_bf16(d, dq + 6, dt + 6, id_s, 1);
              dq += q_step;
              dt += kAtom >> 4;
              acc = 1;
            }
          };
          blocks(whole0);
          if (pieces > 1) {
            if (!last && !(ok = mbar_wait_ready(&full[2 * ring.st + 1], ring.ph, a.dev_status))) break;
            tc_fence_after();
            blocks(whole1);
          }
          for (int kk = 0; kk < steps_left; ++kk) {
            umma_bf16(d, dq + 2 * kk, dt + 2 * kk, id_s, acc);
            acc = 1;
          }
          umma_commit(&s_full[i & 1]);
          if (t == seg.t1 - 1) umma_commit(q_empty);  // the segment's last product with its q~
        }
        ++segs;
      }
      if (!ok) *stop = 1;
      // products left by a timeout get a bounded chance to finish; on the normal path this is the
      // end of the last one
      umma_commit(&drain[0]);
      mbar_wait_ready(&drain[0], 0u, nullptr);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- O~ issuer
    if (elect_one()) {
      const uint32_t id_o = idesc_bf16_f32(128, p.NH, true, false);
      const uint32_t stage0 = smem_u32(smem + lay.stages), stage_bytes = (uint32_t)p.sa * kAtom;
      const uint32_t p_addr = smem_u32(smem + lay.p);
      Ring ring{p.nstage};
      bool ok = true;
      int i = 0, segs = 0;
      while (ok && walk.next(seg)) {
        if (segs > 0) ok = mbar_wait_ready(o_free, (uint32_t)((segs - 1) & 1), a.dev_status);
        for (int t = seg.t0; ok && t < seg.t1; ++t, ++i, ring.next()) {
          if (!(ok = mbar_wait_ready(&p_full[i & 1], (uint32_t)((i >> 1) & 1), a.dev_status))) break;
          tc_fence_after();
          uint64_t dt = sw128_mn_desc(stage0 + (uint32_t)ring.st * stage_bytes, kAtom);
          const uint64_t dp = sw128_desc(p_addr);
          for (int m = 0; m < p.nm; ++m, dt += 2 * kAtom >> 4) {
            const uint32_t d = tmem + (uint32_t)(m * p.NH);
            umma_bf16(d, dt, dp, id_o, t > seg.t0);
            umma_bf16(d, dt + 128, dp + 2, id_o, 1);
            umma_bf16(d, dt + 256, dp + 4, id_o, 1);
            umma_bf16(d, dt + 384, dp + 6, id_o, 1);
            if (m == p.m0 - 1) umma_commit(&empty[2 * ring.st]);
          }
          if (pieces > 1) umma_commit(&empty[2 * ring.st + 1]);
          umma_commit(&pv_done[i & 1]);
        }
        ++segs;
      }
      umma_commit(&drain[1]);
      mbar_wait_ready(&drain[1], 0u, nullptr);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- rows past the length
    int i = 0, tails = 0;
    while (walk.next(seg)) {
      i += seg.t1 - seg.t0;
      const int valid = seg.L - (seg.t1 - 1) * kTok;
      if (valid >= kTok) continue;
      const int k = i - 1, st = k % p.nstage;
      // The issuer says when the tile is in (waiting on the stage itself could see an earlier
      // use), or that it gave up; the wait spans the whole segment, hence the wider limit.
      const uint64_t since = global_timer_ns();
      bool got = mbar_try_wait(partial, (uint32_t)(tails & 1));
      while (!got && *stop == 0 && global_timer_ns() - since < 32 * kWaitLimitNs)
        got = mbar_try_wait(partial, (uint32_t)(tails & 1));
      if (!__all_sync(~0u, got)) break;
      ++tails;
      uint8_t* tile = smem + lay.stages + (uint32_t)(st * p.sa) * kAtom;
      const int atoms = (a.r + 63) / 64;
      for (int e = valid * 8 + lane; e < kTok * 8; e += 32)
#pragma unroll 4
        for (int c = 0; c < atoms; ++c) *reinterpret_cast<uint4*>(tile + c * kAtom + e * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tail);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax and output
    const int quad = warp & 3, r0 = quad * 16 + (lane >> 2), col = 2 * (lane & 3);
    const bool active = quad * 16 < p.NH;        // this warp's 16 heads exist (16 * quad + ...)
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    bool bad = false;  // a wait gave up
    int i = 0;
    while (walk.next(seg)) {
      float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
      for (int t = seg.t0; t < seg.t1; ++t, ++i) {
        uint32_t v[kTok / 2], w[kTok / 4];
        float f0 = 1.f, f1 = 1.f, t0 = -1e30f, t1 = -1e30f, a0 = 0.f, a1 = 0.f;
        // weights with the references m0, m1, and their sums (of the rounded weights)
        auto weights = [&]() {
          const uint64_t sc = pack2(p.scale2, p.scale2), n0 = pack2(-m0, -m0), n1 = pack2(-m1, -m1);
          a0 = a1 = 0.f;
#pragma unroll
          for (int j = 0; j < kTok / 8; ++j) {
            const uint64_t x0 = fma2(((uint64_t)v[4 * j + 1] << 32) | v[4 * j], sc, n0);
            const uint64_t x1 = fma2(((uint64_t)v[4 * j + 3] << 32) | v[4 * j + 2], sc, n1);
            w[2 * j] = pack_bf16x2_rn(fast_exp2(lo_of(x0)), fast_exp2(hi_of(x0)));
            w[2 * j + 1] = pack_bf16x2_rn(fast_exp2(lo_of(x1)), fast_exp2(hi_of(x1)));
            a0 += bf16lo(w[2 * j]) + bf16hi(w[2 * j]);
            a1 += bf16lo(w[2 * j + 1]) + bf16hi(w[2 * j + 1]);
          }
        };
        auto over_lanes = [&]() {  // maxima of the four lanes that share a head
          t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, 1));
          t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, 1));
          t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, 2));
          t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, 2));
        };
        bool move = false;
        if (active) {
          bad |= !mbar_wait_ready(&s_full[i & 1], (uint32_t)((i >> 1) & 1), a.dev_status);
          tc_fence_after();
          tmem_ld_16x256b(tmem + lane_addr + kSCol + (uint32_t)(i & 1) * kTok, v);
          tmem_wait_ld();
          const int valid = seg.L - t * kTok;
          if (valid < kTok) {
#pragma unroll
            for (int j = 0; j < kTok / 8; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (8 * j + col + e >= valid) v[4 * j + e] = v[4 * j + 2 + e] = 0xff800000u;  // -inf
          }
          float s0 = -INFINITY, s1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < kTok / 8; ++j) {
            s0 = max3(s0, __uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]));
            s1 = max3(s1, __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          }
          // (a floor, so that a tile of -inf scores weighs 0 and not NaN)
          t0 = fmaxf(s0 * p.scale2, -1e30f);
          t1 = fmaxf(s1 * p.scale2, -1e30f);
          if (t == seg.t0) {  // the reference: the first tile's maximum
            over_lanes();
            m0 = t0;
            m1 = t1;
          }
          weights();
          move = (t0 > m0 + kRescale && r0 < nheads) || (t1 > m1 + kRescale && r0 + 8 < nheads);
        }
        if (named_bar_or(1, 128, move || bad)) {
          if (named_bar_or(1, 128, bad)) break;
          // some head's reference moves: weigh the tile again and scale its column of O~^T, once the
          // last product is in
          if (active) {
            over_lanes();
            if (t0 > m0 + kRescale) {
              f0 = fast_exp2(m0 - t0);
              m0 = t0;
            }
            if (t1 > m1 + kRescale) {
              f1 = fast_exp2(m1 - t1);
              m1 = t1;
            }
            weights();
            if ((lane & 3) == 0) {
              sm_f[r0] = f0;
              sm_f[r0 + 8] = f1;
            }
          }
          bad |= !mbar_wait_ready(&pv_done[(i - 1) & 1], (uint32_t)(((i - 1) >> 1) & 1), a.dev_status);
          if (named_bar_or(1, 128, bad)) break;
          tc_fence_after();
          for (int c = 0; c < p.nm * p.NH; c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem + lane_addr + (uint32_t)c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * lds_f32(smem_u32(sm_f + c % p.NH + e)));
            tmem_st16(tmem + lane_addr + (uint32_t)c, o);
          }
          tmem_wait_st();
        }
        l0 = l0 * f0 + a0;
        l1 = l1 * f1 + a1;
        if (active) {
          // P's buffer is free once the last tile's product is in
          if (i >= 1 && !mbar_wait_ready(&pv_done[(i - 1) & 1], (uint32_t)(((i - 1) >> 1) & 1), a.dev_status))
            bad = true;
          const uint32_t base = (uint32_t)r0 * 128u + (uint32_t)col * 2u;
#pragma unroll
          for (int j = 0; j < kTok / 8; ++j) {
            const uint32_t off = (uint32_t)((j ^ (r0 & 7)) << 4);
            *reinterpret_cast<uint32_t*>(smem + lay.p + base + off) = w[2 * j];
            *reinterpret_cast<uint32_t*>(smem + lay.p + base + 8 * 128 + off) = w[2 * j + 1];
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !bad) mbar_arrive(&p_full[i & 1]);
      }
      // the segment's sums; O~ is complete with its last tile's product
      l0 += __shfl_xor_sync(~0u, l0, 1);
      l1 += __shfl_xor_sync(~0u, l1, 1);
      l0 += __shfl_xor_sync(~0u, l0, 2);
      l1 += __shfl_xor_sync(~0u, l1, 2);
      if (active && (lane & 3) == 0) {
        sm_l[r0] = l0;
        sm_l[r0 + 8] = l1;
        sm_f[r0] = 1.f / l0;
        sm_f[r0 + 8] = 1.f / l1;
        sm_m[r0] = m0;
        sm_m[r0 + 8] = m1;
      }
      if (!bad) bad = !mbar_wait_ready(&pv_done[(i - 1) & 1], (uint32_t)(((i - 1) >> 1) & 1), a.dev_status);
      if (named_bar_or(1, 128, bad)) break;
      tc_fence_after();
      const int n = tiles_of(seg.L);
      const bool whole = seg.t0 == 0 && seg.t1 == n;
      const int dim = quad * 32 + lane;
      const int slot = ((int)blockIdx.x * 2 + (seg.first ? 0 : 1));
      uint8_t* ws = reinterpret_cast<uint8_t*>(a.workspace);
      float2* ml = reinterpret_cast<float2*>(ws + meta_bytes(a.B)) + (size_t)slot * kMaxHeads;
      float* part = reinterpret_cast<float*>(ws + meta_bytes(a.B) + ml_bytes()) + (size_t)slot * p.NH * a.r;
      if (whole) {
        // Half of the heads' 128 dims at a time, through P's memory (free until the next segment): a
        // thread has one dim of every head, and stored from there, two bytes a lane, the output took
        // 5 us at 64 heads and r = 512.
        const int hc = p.NH / 2, th = tid - 128;
        uint8_t* stage = smem + lay.p;
        for (int m = 0; m < p.nm; ++m)
          for (int c = 0; c < p.NH; c += hc) {
            uint32_t v[2][16];
            tmem_ld16(tmem + lane_addr + (uint32_t)(m * p.NH + c), v[0]);
            if (hc > 16) tmem_ld16(tmem + lane_addr + (uint32_t)(m * p.NH + c + 16), v[1]);
            float4 f[8];  // 1 / l (the last ones may lie past the heads: they are not used)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (4 * e < hc) f[e] = lds128f(smem_u32(sm_f + c + 4 * e));
            tmem_wait_ld();
            // (eight heads a branch: hc is a multiple of eight, and a test each made this ten times
            // as long)
#pragma unroll
            for (int e8 = 0; e8 < 32; e8 += 8)
              if (e8 < hc) {
#pragma unroll
                for (int e = e8; e < e8 + 8; ++e) {
                  const float4 g = f[e >> 2];
                  const float x = (e & 3) == 0 ? g.x : (e & 3) == 1 ? g.y : (e & 3) == 2 ? g.z : g.w;
                  *reinterpret_cast<uint16_t*>(stage + e * 256 + dim * 2) =
                      f32_to_bf16_rn(__uint_as_float(v[e >> 4][e & 15]) * x);
                }
              }
            named_bar_sync(1, 128);
            const int h0 = th >> 4, d = m * 128 + (th & 15) * 8;  // sixteen lanes a head
            uint16_t* o = a.out + ((size_t)seg.b * a.Hq + h_base + c + h0) * a.r + d;
            uint4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (8 * k < hc) y[k] = *reinterpret_cast<const uint4*>(stage + (8 * k + h0) * 256 + (th & 15) * 16);
#pragma unroll
            for (int k = 0; k < 4; ++k, o += 8 * (size_t)a.r)
              if (8 * k < hc && c + 8 * k + h0 < nheads && d < a.r) *reinterpret_cast<uint4*>(o) = y[k];
            named_bar_sync(1, 128);
          }
      } else {
        // 32 heads' columns at a time: one wait for two loads, then a run of stores (a warp's 32
        // neighbouring dims of one head each)
        for (int m = 0; m < p.nm; ++m) {
          const int d = m * 128 + dim;
          for (int c = 0; c < p.NH; c += 32) {
            uint32_t v[2][16];
            tmem_ld16(tmem + lane_addr + (uint32_t)(m * p.NH + c), v[0]);
            if (c + 16 < p.NH) tmem_ld16(tmem + lane_addr + (uint32_t)(m * p.NH + c + 16), v[1]);
            tmem_wait_ld();
            const int nh = d < a.r ? nheads - c : 0;  // heads to store
            float* o = part + (size_t)c * a.r + d;
#pragma unroll
            for (int e8 = 0; e8 < 32; e8 += 8, o += 8 * (size_t)a.r) {
              if (e8 + 8 <= nh) {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[(size_t)e * a.r] = __uint_as_float(v[(e8 + e) >> 4][(e8 + e) & 15]);
              } else if (e8 < nh) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (e8 + e < nh) o[(size_t)e * a.r] = __uint_as_float(v[(e8 + e) >> 4][(e8 + e) & 15]);
              }
            }
          }
        }
      }
      tc_fence_before();
      const int th = tid - 128;
      if (!whole && th < nheads) ml[th] = make_float2(sm_m[th], sm_l[th]);
      // the CTAs that hold this sequence, for the merge: written by the one with its first tile
      if (seg.t0 == 0 && th == 0 && group == 0 && !p.whole) {
        reinterpret_cast<int2*>(ws)[seg.b] =
            make_int2(cta * 2 + (seg.first ? 0 : 1), whole ? -1 : (int)((seg.at + n - 1) / per));
      }
      named_bar_sync(1, 128);  // sm_l, sm_m and O~ have been read
      if (lane == 0) mbar_arrive(o_free);
    }
    // without a second kernel the zeros of empty sequences are written here
    if (p.whole)
      for (int b = (int)blockIdx.x; b < a.B; b += (int)gridDim.x)
        if (valid_length(__ldg(a.seq_lens + b), a.max_seq_len) == 0) {
          uint4* out = reinterpret_cast<uint4*>(a.out + (size_t)b * a.Hq * a.r);
          for (int e = tid - 128; e < a.Hq * a.r / 8; e += 128) out[e] = make_uint4(0, 0, 0, 0);
        }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial states of sequences that several CTAs hold, and writes the zeros of empty
// ones.  kWarps warps share a head's parts (a CTA has one head, or eight if kWarps = 1), and a warp
// holds kVec chunks of 128 dims.  Bound by latency: the lengths and the meta word are read together,
// then everything else of up to kBatch parts.
template <int kWarps, int kVec>
__global__ void __launch_bounds__(kWarps == 1 ? 256 : 32 * kWarps) stief_shared_merge_kernel(const SharedDecodeArgs a, int NH, int groups, int G) {
  constexpr int kBatch = kVec == 4 ? 2 : 8;  // parts in flight
  __shared__ float4 acc_s[kWarps][kVec][32];
  __shared__ float2 ml_s[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int nd = (a.r + 127) / 128;
  const int h = kWarps == 1 ? (int)blockIdx.x * 8 + warp : kVec == 4 ? (int)blockIdx.x : (int)blockIdx.x / nd;
  const int d0 = (kVec == 4 ? 0 : (int)blockIdx.x % nd * 128) + lane * 4;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.workspace);
  pdl_wait();
  pdl_launch_dependents();
  const int L = valid_length(__ldg(a.seq_lens + b), a.max_seq_len);
  const int2 meta = __ldcg(reinterpret_cast<const int2*>(ws + (size_t)b * 8));  // (garbage if L == 0)
  if (L > 0 && meta.y < 0) return;  // whole: written already
  if (h >= a.Hq) return; // (kWarps > 1: never, the grid is exact)
  uint16_t* out = a.out + ((size_t)b * a.Hq + h) * a.r + d0;
  if (L == 0) {
    if (kWarps == 1 || warp == 0)
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (d0 + 128 * j < a.r) *reinterpret_cast<uint2*>(out + 128 * j) = make_uint2(0, 0);
    return;
  }
  // part k is in CTA c = meta.x / 2 + k of the head's group: slot 0 but for the first
  const int group = h / NH, hl = h % NH, c_first = meta.x >> 1, n = meta.y - c_first + 1;
  if (c_first < 0 || n < 1 || meta.y >= G) return;  // the first kernel gave up on a wait
  const float2* ml = reinterpret_cast<const float2*>(ws + meta_bytes(a.B));
  const float* part = reinterpret_cast<const float*>(ws + meta_bytes(a.B) + ml_bytes());
  float M = -INFINITY, l = 0.f;
  float4 acc[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = kWarps == 1 ? 0 : warp; k0 < n; k0 += kWarps * kBatch) {
    float2 e[kBatch];
    float4 o[kBatch][kVec];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + kWarps * i;
      e[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < kVec; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n) {
        const size_t s = (size_t)(((c_first + k) * groups + group) * 2 + (k == 0 ? (meta.x & 1) : 0));
        e[i] = __ldcg(ml + s * kMaxHeads + hl);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (d0 + 128 * j < a.r)
            o[i][j] = __ldcg(reinterpret_cast<const float4*>(part + (s * NH + hl) * a.r + d0 + 128 * j));
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, e[i].x);
    const float f0 = fast_exp2(M - top);  // (M is finite after the first batch; 2^-inf = 0 before)
    M = top;
    l *= f0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[j].x *= f0, acc[j].y *= f0, acc[j].z *= f0, acc[j].w *= f0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float f = fast_exp2(e[i].x - M);
      l += f * e[i].y;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        acc[j].x += f * o[i][j].x;
        acc[j].y += f * o[i][j].y;
        acc[j].z += f * o[i][j].z;
        acc[j].w += f * o[i][j].w;
      }
    }
  }
  if (kWarps > 1) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc_s[warp][j][lane] = acc[j];
    if (lane == 0) ml_s[warp] = make_float2(M, l);
    __syncthreads();
    if (warp >= kVec) return;  // a warp a chunk joins the warps
    for (int k = 0; k < kWarps; ++k) M = k == 0 ? ml_s[0].x : fmaxf(M, ml_s[k].x);
    l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < kWarps; ++k) {
      const float f = fast_exp2(ml_s[k].x - M);
      const float4 o = acc_s[k][warp][lane];
      l += f * ml_s[k].y;
      x.x += f * o.x;
      x.y += f * o.y;
      x.z += f * o.z;
      x.w += f * o.w;
    }
    const float inv = 1.f / l;
    if (d0 + 128 * warp < a.r)
      *reinterpret_cast<uint2*>(out + 128 * warp) = make_uint2(pack_bf16x2_rn(x.x * inv, x.y * inv), pack_bf16x2_rn(x.z * inv, x.w * inv));
    return;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (d0 + 128 * j < a.r)
      *reinterpret_cast<uint2*>(out + 128 * j) = make_uint2(pack_bf16x2_rn(acc[j].x * inv, acc[j].y * inv),
                                                            pack_bf16x2_rn(acc[j].z * inv, acc[j].w * inv));
}

size_t shared_decode_workspace_bytes(int B, int Hq, int r) {
  return meta_bytes(B) + ml_bytes() + (size_t)kMaxCtas * 2 * heads_per_cta(Hq) * r * 4;
}

cudaError_t launch_shared_decode(const SharedDecodeArgs& a, cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.w = a.r + a.dr;
  p.na = (p.w + 63) / 64;
  p.nm = (a.r + 127) / 128;
  p.sa = p.na > 2 * p.nm ? p.na : 2 * p.nm;
  p.NH = heads_per_cta(a.Hq);
  p.groups = (a.Hq + p.NH - 1) / p.NH;
  const int ctas = a.sms < kMaxCtas ? a.sms : kMaxCtas;
  p.G = ctas / p.groups;
  p.scale2 = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (p.scale2 < 1e-30f) p.scale2 = 1e-30f;  // above 0, so that a masked score stays -inf
  p.negate = a.scale < 0;
#ifdef STIEF_TEST_HOOKS
  p.stall = test_stall_bytes();
#endif
  // Short sequences are finished by one CTA each: the parts and the second kernel cost more than a
  // few further tiles.  With a CTA for each, which then needs no sums over the lengths either, up to
  // six tiles (5 sequences, 16 heads, rank 128: 6.2 us for four, 0.6 a tile more, split 8.6 to 9.2;
  // at 64 heads and rank 512 11.2 us for four, 14.4 for five, 16.8 for eight, split 14.4 to 14.7),
  // otherwise four, as whole sequences are dealt out less evenly.
  const int most_tiles = tiles_of(a.max_seq_len);
  p.direct = a.B <= p.G && most_tiles <= kDirectTiles;
  p.whole = p.direct || most_tiles <= kWholeTiles;
  constexpr uint32_t kMost = kMaxSmemPerBlock - 1024;  // the static part, rounded up
  for (p.nstage = kMaxStages; p.nstage > 2 && layout_of(p.na, p.sa, p.NH, p.nstage).total > kMost;) --p.nstage;
  const uint32_t smem = layout_of(p.na, p.sa, p.NH, p.nstage).total;
  if (smem > kMost) return cudaErrorInvalidValue;
  const uint64_t rows = (uint64_t)a.num_pages * a.page_size, pitch = (uint64_t)p.w * 2;
  p.whole_rows = p.w % 64 == 0;
  if (!encode_tiled_bf16_2d(&p.mq, a.q, (uint64_t)p.w, (uint64_t)a.B * a.Hq, pitch, 64, (uint32_t)p.NH,
                            CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // The tile comes in two pieces, split between 128-dim tiles of o~: the first half's memory is
  // free again, and its next rows under way, while the second half's product runs.
  p.m0 = (p.nm + 1) / 2;
  p.n0 = p.na < 2 * p.m0 ? p.na : 2 * p.m0;
  const uint32_t n1 = (uint32_t)(p.na - p.n0);
  if (p.whole_rows) {
    if (!encode_tiled_bf16_3d(&p.ma, a.pages, {64, rows, (uint64_t)p.na}, {pitch, 128},
                              {64, kTok, (uint32_t)p.n0}) ||
        !encode_tiled_bf16_3d(&p.mb, a.pages, {64, rows, (uint64_t)p.na}, {pitch, 128},
                              {64, kTok, n1 > 0 ? n1 : 1u}))
      return cudaErrorInvalidValue;
  } else {
    if (!encode_tiled_bf16_2d(&p.ma, a.pages, (uint64_t)p.w, rows, pitch, 64, kTok, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    p.mb = p.ma;
  }
  const auto kern = stief_shared_decode_kernel;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kern), a.device, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.G * p.groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess || p.whole) return e;
  cfg.dynamicSmemBytes = 0;
  // The warps of a CTA share a head's parts, whose number only the GPU knows: sixteen where a
  // sequence may have very many (and one wave holds the output), four otherwise, 128 dims a CTA
  // where sequences are few and the CTAs too, else all dims; with too many CTAs even so, a warp a
  // head.  (In us, a warp a head, 4 warps with 512 dims, 4 with 128, 16: 1 sequence of 32768, 32 heads,
  // 55.4, 30.1, 23.2, 19.7; 5 of 9000 to 20000, 40 heads, 45.7, 32.9, 30.2, 37.5; one of 20000 among 63
  // of 300, 32 heads, 39.1, 25.9, 33.7, 85; 64 of 511 to 4096, 128 heads, 75.7, 83, 127, 357.)
  const long long heads = (long long)a.Hq * a.B;
  if (p.G >= 64 * a.B && most_tiles >= 128 && heads * p.nm <= 4LL * a.sms) {
    cfg.blockDim = dim3(512);
    cfg.gridDim = dim3(a.Hq * p.nm, a.B);
    return cudaLaunchKernelEx(&cfg, stief_shared_merge_kernel<16, 1>, a, p.NH, p.groups, p.G);
  }
  if (p.G > 8 * a.B && heads * p.nm <= 8LL * a.sms) {
    cfg.blockDim = dim3(128);
    cfg.gridDim = dim3(a.Hq * p.nm, a.B);
    return cudaLaunchKernelEx(&cfg, stief_shared_merge_kernel<4, 1>, a, p.NH, p.groups, p.G);
  }
  if (heads <= 16LL * a.sms) {
    cfg.blockDim = dim3(128);
    cfg.gridDim = dim3(a.Hq, a.B);
    return cudaLaunchKernelEx(&cfg, stief_shared_merge_kernel<4, 4>, a, p.NH, p.groups, p.G);
  }
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3((a.Hq + 7) / 8, a.B);
  return cudaLaunchKernelEx(&cfg, stief_shared_merge_kernel<1, 4>, a, p.NH, p.groups, p.G);
}

}  // namespace stief
