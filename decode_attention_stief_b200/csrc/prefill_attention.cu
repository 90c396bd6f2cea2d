// prefill_attention.cu -- causal attention of ragged prompts over per-head keys and values, for
// sm_100a.  Query i of sequence b (n_q queries, n_k keys) sees keys j <= i + n_k - n_q:
//     o_i = softmax_j(scale * (q_i . k_j + q^R_i . k^R_j)) v_j,
// one pass over the keys with a running maximum and sum.
//
// What bounds it: the products (2 (256 + dr) operations a visible pair and head), nearly as long one
// exponential a pair (16 a cycle on an SM against 4096 multiply-adds), and nearly as long again the
// shared memory that the products read and the copies write.
//
// Two kernels; launch_prefill below chooses.  prefill_one_tile.cu: two CTAs an SM, a tile of 128
// query rows each, on its own, or, where there are few tiles, several CTAs a tile.  Here, for keys with a position part, the same two CTAs an SM, but a
// CTA and its neighbour on the next SM work as a pair on 256 query rows of one KV head: each product
// is one of M = 256 (cta_group::2), and a CTA brings half of the keys' rows and half of the values'
// columns:
//     S [256 x 64] = Q . K^T,    O [256 x 128] += P . V.
// At dr = 64 a step of 64 keys then reads 68 KB of a CTA's shared memory and writes 20, instead of 88
// and 40, and keys and values have room for three slots each, where a CTA on its own has one of keys.
// (Two tiles of queries in one CTA, steps of 128 keys and no second buffer of scores, which this
// replaces: 8192 tokens, 32 heads, dr 64, 553 us against 540; 8 chunks of 512 over 3012 keys 251
// against 219; 1 of 2048 over 6048 keys, 16 heads, 114 against 98.  Two threads a row in the softmax,
// so that twice as many warps hide each other's latencies: within 2 %.)  Without a position part
// pairs were as fast as single tiles on long prompts (8192 tokens, 32 heads over 8: 456 us both), slower
// on shorter ones (2500 tokens 66 us against 58) and faster on chunks over many keys (8 of 512 over 3012
// 216 against 239); that form is not built.
// The rest is as in prefill_one_tile.cu: S in two buffers of 64 columns, P over its S, O behind them,
// half of the tensor memory a CTA; packed heads; the reference of the softmax.
//   warp 0 of each CTA: TMA producer; warp 1 of the first: MMA issuer; warp 2: zeroes the value rows
//   past n_k in the last step (they may hold NaN, and 0 * NaN is NaN); warps 4-7: softmax, a thread a
//   row, and the output.
// CTAs start with the longest tiles of queries; a pair none of whose rows exists ends at once.
//
// Measured: 8192 tokens, 32 heads, dr 64: 540 us, 1.27 PFLOP/s (630 us, 1.09, in long runs under the
// power cap); 8 chunks of 512 over 3012 keys: 219 us, 0.94.
#include <cstdint>

#include "prefill_row.cuh"
#include "shared_latent.h"
#include "stief_device.cuh"
#include "umma.cuh"

namespace stief {

namespace {

constexpr int kRows = 128;                 // query rows a tile
constexpr int kKeys = 64;                  // keys a step
constexpr uint32_t kAtom = kRows * 128;    // bytes of 128 rows x 64 columns
constexpr uint32_t kBlock = kKeys / 2 * 128;  // bytes of 32 key rows x 64 columns
constexpr uint32_t kValue = kKeys * 128;   // bytes of 64 value rows x 64 columns
constexpr int kThreads = 256;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kOCol = 128;            // S at 0 and 64, O at 128
constexpr float kRescale = 60.f;           // log2 units a score may pass the reference by
constexpr float kFloor = -1e30f;

struct Args {
  CUtensorMap mq;   // q [Nq][Hq][128], box 64 columns x pack heads x 128 / pack queries
  CUtensorMap mk;   // k [Nkv] rows in blocks of 64 columns, box 64 x 32 x 2
  CUtensorMap mv;   // v, same, box 64 x 64 x 1
  CUtensorMap mp;   // k_pe [Nkv][dr], box 64 x 32
  PrefillArgs a;
  int pack;         // heads of a tile: its row r is query r / pack, head r % pack (pack divides 128)
  int shift;        // log2(pack)
  int qtiles;       // tiles of the longest sequence
  float scale2;     // |scale| * log2(e)
  int negate;       // scale < 0: the products are negated instead
#ifdef STIEF_TEST_HOOKS
  uint32_t stall;   // test build: bytes expected of the first copy that none delivers
  uint32_t apart;   // test build: the pair's tensor memory is taken not to match
#endif
};

constexpr int kBlocks = 3;                 // of 64 columns in a query or key row
constexpr int kSlots = 3;                  // of keys and of values
constexpr uint32_t kKeyBytes = kBlocks * kBlock;
constexpr uint32_t kSmemK = kBlocks * kAtom, kSmemV = kSmemK + kSlots * kKeyBytes, kSmemBars = kSmemV + kSlots * kValue;
constexpr uint32_t kSmem = kSmemBars + 8 * (4 * kSlots + 12);
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs share an SM");

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 2) stief_prefill_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const PrefillArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  // (the full barriers of copies, p_full and tail that count are the leader's; the others are each
  // CTA's own)
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kSmemBars);  // [kSlots]
  uint64_t* k_empty = k_full + kSlots;   // [kSlots]
  uint64_t* v_full = k_empty + kSlots;   // [kSlots]
  uint64_t* v_empty = v_full + kSlots;   // [kSlots]
  uint64_t* s_full = v_empty + kSlots;   // [2] S of a step is in TMEM
  uint64_t* p_full = s_full + 2;         // [2] P of a step is, in both CTAs
  uint64_t* pv_done = s_full + 4;        // [2] O of a step is added
  uint64_t* q_full = s_full + 6;
  uint64_t* o_full = s_full + 7;         // O is complete
  uint64_t* partial = s_full + 8;        // the last values are in and are not 64
  uint64_t* tail = s_full + 9;           // their rows past n_k are cleared, in both CTAs
  uint64_t* drain = s_full + 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 11);
#ifdef STIEF_TEST_HOOKS
  const uint32_t stall = p.stall, apart = p.apart;
#else
  constexpr uint32_t stall = 0u, apart = 0u;
#endif
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) report(a.dev_status, STIEF_DEV_SMEM_ALIGN);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 4 * kSlots; ++i) mbar_init(&k_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(o_full, 1);
    mbar_init(partial, 1);
    mbar_init(tail, 2);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  const int groups = a.Hq >> p.shift, gb = groups * a.B, rest = (int)(blockIdx.x / 2 % (unsigned)gb);
  const int qt = p.qtiles - 1 - (int)(blockIdx.x / 2 / (unsigned)gb);
  const int b = rest / groups, h0 = (rest % groups) << p.shift, hk = h0 / (a.Hq / a.Hkv);

  pdl_wait();
  const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
  const int k0 = __ldg(a.kv_start + b), k1 = __ldg(a.kv_start + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.Nq || k0 < 0 || k1 < k0 || k1 > a.Nkv || q1 - q0 > a.max_q) {
    if (tid == 0 && leader && h0 == 0 && qt == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    return;
  }
  // first query of the pair and of this CTA (which has none, where the second tile is missing)
  const int nq = q1 - q0, n_k = k1 - k0, queries = kRows >> p.shift, begin = qt * 2 * queries;
  if (begin >= nq) return;  // (both CTAs)
  const int first = begin + (int)rank * queries;
  // steps of keys that the pair's last query sees
  const int last = min(nq, begin + 2 * queries) - 1;
  const long long most = (long long)last + n_k - nq + 1;
  int n = most > 0 ? (int)((min(most, (long long)n_k) + kKeys - 1) / kKeys) : 0;

  // (only after the dependency wait, and before this kernel's own dependents may start: a CTA that
  // holds tensor memory while it waits for another kernel must not starve one of that kernel's)
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs have their barriers and their tensor memory
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  // A product takes both CTAs' operands and results from the same columns.  The two allocate together,
  // and with other kernels' CTAs on one of the two SMs their columns have not been seen to differ, but
  // nothing documented promises it: if they do, nothing is computed and no row is written.
  const bool paired = load_cluster(in_cta(tmem_slot, rank ^ 1u)) == tmem + apart;
  if (!paired) {
    if (tid == 0) report(a.dev_status, STIEF_DEV_TMEM_PAIR);
    n = 0;
  }
  uint32_t nan = 0, which = 0;  // NaN among a row's outputs, and the warp's rows with one

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (n > 0 && elect_one()) {
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      int nk = 0, nv = 0;
      // The leader expects both CTAs' bytes on its barriers.  (The second CTA's copies may land first: it
      // asks for a slot only when the products with its last use are done, that is in the phase
      // that the leader opens.)
      auto load_k = [&](int j) -> bool {
        const int slot = j % kSlots;
        if (j >= kSlots && !mbar_wait_ready(&k_empty[slot], (uint32_t)((j / kSlots) & 1) ^ 1u, a.dev_status)) return false;
        uint8_t* at = smem + kSmemK + (uint32_t)slot * kKeyBytes;
        const uint32_t bar = in_cta(&k_full[slot], 0);
        const int row = k0 + j * kKeys + (int)rank * (kKeys / 2);
        if (leader) mbar_arrive_expect_tx(&k_full[slot], 2 * kKeyBytes);
        tma_load_3d_pair(at, &p.mk, 0, row, hk * 2, bar, keep);
        tma_load_2d_pair(at + 2 * kBlock, &p.mp, 0, row, bar, keep);
        return true;
      };
      auto load_v = [&](int j) -> bool {
        const int slot = j % kSlots;
        if (j >= kSlots && !mbar_wait_ready(&v_empty[slot], (uint32_t)((j / kSlots) & 1) ^ 1u, a.dev_status)) return false;
        if (leader) mbar_arrive_expect_tx(&v_full[slot], 2 * kValue);
        tma_load_3d_pair(smem + kSmemV + (uint32_t)slot * kValue, &p.mv, 0, k0 + j * kKeys, hk * 2 + (int)rank,
                         in_cta(&v_full[slot], 0), keep);
        return true;
      };
      if (leader) mbar_arrive_expect_tx(q_full, 2 * kBlocks * kAtom + stall);
      for (int c = 0; c < kBlocks; ++c)
        tma_load_3d_pair(smem + (uint32_t)c * kAtom, &p.mq, 64 * c, h0, q0 + first, in_cta(q_full, 0), once);
      bool ok = load_k(nk++);
      // (the keys of a step are free again one step before its values)
      for (int j = 0; ok && j < n; ++j) {
        if (nk < n) {
          if (!(ok = load_k(nk))) break;
          ++nk;
        }
        ok = load_v(nv);
        if (ok) ++nv;
      }
      // every requested copy of both CTAs lands before their shared memory is released
      if (leader) {
        mbar_wait_ready(q_full, 0, nullptr);
        for (int j = max(0, nk - kSlots); j < nk; ++j)
          mbar_wait_ready(&k_full[j % kSlots], (uint32_t)((j / kSlots) & 1), nullptr);
        for (int j = max(0, nv - kSlots); j < nv; ++j)
          mbar_wait_ready(&v_full[j % kSlots], (uint32_t)((j / kSlots) & 1), nullptr);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (n > 0 && leader && elect_one()) {
      const uint32_t id_s = idesc_bf16_f32(256, kKeys, false, false) | (p.negate ? 1u << 13 : 0u);
      const uint32_t id_o = idesc_bf16_f32(256, 128, false, true);
      const uint64_t dq = sw128_desc(smem_u32(smem)), dk0 = sw128_desc(smem_u32(smem + kSmemK));
      const uint64_t dv0 = sw128_mn_desc(smem_u32(smem + kSmemV), kValue);  // (64 columns a CTA: one block)
      const int pe_steps = a.dr / 16;
      auto wait_k = [&](int j) -> bool {
        return mbar_wait_ready(&k_full[j % kSlots], (uint32_t)((j / kSlots) & 1), a.dev_status);
      };
      auto issue_s = [&](int j) {
        tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((uint32_t)(j % kSlots) * (kKeyBytes >> 4));
        const uint32_t d = tmem + (uint32_t)(j & 1) * kKeys;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16_pair(d, dq + (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2, dk + (kk >> 2) * (kBlock >> 4) + (kk & 3) * 2,
                         id_s, kk > 0);
        for (int kk = 0; kk < pe_steps; ++kk)
          umma_bf16_pair(d, dq + 2 * (kAtom >> 4) + 2 * kk, dk + 2 * (kBlock >> 4) + 2 * kk, id_s, 1);
        umma_commit_pair(&s_full[j & 1]);
        umma_commit_pair(&k_empty[j % kSlots]);
      };
      bool ok = mbar_wait_ready(q_full, 0, a.dev_status);
      for (int j = 0; j < 2 && j < n && ok; ++j) {
        ok = wait_k(j);
        if (ok) issue_s(j);
      }
      for (int j = 0; ok && j < n; ++j) {
        // (what has long arrived is waited for first: a test of a barrier takes some 250 cycles next
        // to the products' shared-memory traffic)
        if (!(ok = mbar_wait_ready(&v_full[j % kSlots], (uint32_t)((j / kSlots) & 1), a.dev_status))) break;
        if (j == n - 1 && n * kKeys > n_k) {  // rows past n_k must not be NaN
          mbar_arrive_cluster(in_cta(partial, 0));
          mbar_arrive_cluster(in_cta(partial, 1));
          if (!(ok = mbar_wait_ready(tail, 0, a.dev_status))) break;
        }
        if (j + 2 < n && !(ok = wait_k(j + 2))) break;
        if (!(ok = mbar_wait_ready(&p_full[j & 1], (uint32_t)((j >> 1) & 1), a.dev_status))) break;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((uint32_t)(j % kSlots) * (kValue >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_ts_pair(tmem + kOCol, tmem + (uint32_t)(j & 1) * kKeys + kk * 8, dv + kk * 128, id_o, j > 0 || kk > 0);
        umma_commit_pair(&v_empty[j % kSlots]);
        umma_commit_pair(&pv_done[j & 1]);
        if (j + 2 < n) issue_s(j + 2);  // into the buffer that P has left
      }
      if (ok) umma_commit_pair(o_full);
      // products left by a timeout get a bounded chance to finish; on the normal path this is the
      // end of the last one
      umma_commit_pair(drain);
      mbar_wait_ready(drain, 0, nullptr);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- value rows past n_k
    if (n > 0 && n * kKeys > n_k) {
      const uint64_t since = global_timer_ns();
      bool got = mbar_try_wait(partial, 0);
      while (!got && global_timer_ns() - since < 8 * kWaitLimitNs) got = mbar_try_wait(partial, 0);
      if (__all_sync(~0u, got)) {
        uint8_t* v = smem + kSmemV + (uint32_t)((n - 1) % kSlots) * kValue;
        for (int e = (n_k - (n - 1) * kKeys) * 8 + lane; e < kKeys * 8; e += 32)
          *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_cta(tail, 0));
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax and output
    const int quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16, o_col = tmem + lanes + kOCol;
    const int r0 = quad * 32, query = first + ((r0 + lane) >> p.shift);  // the thread's row
    const int seen = (int)max(0LL, min((long long)n_k, (long long)query + n_k - nq + 1));  // keys it sees
    const int all = __shfl_sync(~0u, seen, 0);  // keys that every row of the warp sees
    const uint64_t scale2 = pack2(p.scale2, p.scale2);
    float m = kFloor;
    uint64_t l0 = 0, l1 = 0;
    bool ok = paired;
    for (int j = 0; j < n; ++j) {
      ok = __all_sync(~0u, mbar_wait_ready(&s_full[j & 1], (uint32_t)((j >> 1) & 1), a.dev_status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t s_col = tmem + lanes + (uint32_t)(j & 1) * kKeys;
      uint32_t s[2][32];
      tmem_ld32(s_col, s[0]);
      tmem_ld32(s_col + 32, s[1]);
      tmem_wait_ld();
      if (all < (j + 1) * kKeys) {  // some row of the warp does not see the whole step
        const int lim = seen - j * kKeys;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e >= lim) s[c][e] = 0xff800000u;  // -inf
      }
      float t0 = kFloor, t1 = kFloor;
      auto maximum = [&](int c) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          t0 = max3(t0, __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
          t1 = max3(t1, __uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3]));
        }
      };
      if (j == 0) {  // the reference: the first step's maximum
        maximum(0);
        maximum(1);
        m = fmaxf(fmaxf(t0, t1) * p.scale2, kFloor);
      }
      // the weights of 32 keys, their sums added to l0 and l1
      auto weights = [&](int c) {
        const uint64_t m2 = pack2(-m, -m);
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t x = fma2(((uint64_t)s[c][2 * e + 1] << 32) | s[c][2 * e], scale2, m2);
          const float lo = fast_exp2(lo_of(x)), hi = fast_exp2(hi_of(x));
          if (e & 1) l1 = add2(l1, pack2(lo, hi));
          else l0 = add2(l0, pack2(lo, hi));
          w[e] = pack_bf16x2_rn(lo, hi);
        }
        tmem_st16(s_col + 16 * c, w);
      };
      const uint64_t before0 = l0, before1 = l1;
      weights(0);
      if (j > 0) maximum(0);
      weights(1);
      if (j > 0) maximum(1);
      const float top = fmaxf(t0, t1) * p.scale2;
      if (__any_sync(~0u, top > m + kRescale)) {  // (never in the first step)
        ok = __all_sync(~0u, mbar_wait_ready(&pv_done[(j - 1) & 1], (uint32_t)(((j - 1) >> 1) & 1), a.dev_status));
        if (!ok) break;
        tc_fence_after();
        const bool move = top > m + kRescale;
        const float f = move ? fast_exp2(m - top) : 1.f;
        if (move) m = top;
        l0 = fma2(before0, pack2(f, f), 0);
        l1 = fma2(before1, pack2(f, f), 0);
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          uint32_t v[16];
          tmem_ld16(o_col + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
          tmem_st16(o_col + c, v);
        }
        weights(0);
        weights(1);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(in_cta(&p_full[j & 1], 0));
    }
    // the output: zeros for a row that sees no key
    if (ok && n > 0) ok = __all_sync(~0u, mbar_wait_ready(o_full, 0, a.dev_status));
    if (ok) {
      tc_fence_after();
      const uint64_t ls = add2(l0, l1);
      const float inv = seen > 0 ? 1.f / (lo_of(ls) + hi_of(ls)) : 0.f;
      // The rows go through the warp's part of the queries' memory (their last product is done), so
      // that half a warp stores a whole row.  A row's 16-byte pieces are rotated by its number.
      uint8_t* stage = smem + (uint32_t)quad * 32 * 256;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t v[32];
        if (n > 0) {
          tmem_ld32(o_col + c, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (seen > 0) {
            x.x = pack_bf16x2_rn(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv);
            x.y = pack_bf16x2_rn(__uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv);
            x.z = pack_bf16x2_rn(__uint_as_float(v[e + 4]) * inv, __uint_as_float(v[e + 5]) * inv);
            x.w = pack_bf16x2_rn(__uint_as_float(v[e + 6]) * inv, __uint_as_float(v[e + 7]) * inv);
          }
          nan = nan_of(x.x, x.y, nan_of(x.z, x.w, nan));
          *reinterpret_cast<uint4*>(stage + lane * 256 + ((((c + e) >> 3) ^ (lane & 15)) << 4)) = x;
        }
      }
      __syncwarp();
      const int piece = lane & 15;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4), qr = first + ((r0 + r) >> p.shift), h = h0 + ((r0 + r) & (p.pack - 1));
        const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 256 + ((piece ^ (r & 15)) << 4));
        if (qr < nq) *reinterpret_cast<uint4*>(a.out + ((size_t)(q0 + qr) * a.Hq + h) * 128 + piece * 8) = x;
      }
      which = __ballot_sync(~0u, has_nan(nan));
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA is read, written or signalled by the other any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  if (__builtin_expect(which != 0, 0)) {
    __syncwarp();
    redo_rows(a, p.shift, p.qtiles, blockIdx.x / 2, 2 * kRows, kKeys, (int)rank * kRows + (warp & 3) * 32, 1, which,
              p.negate ? -p.scale2 : p.scale2);
  }
}

namespace {

cudaError_t launch_pair(const PrefillArgs& a, int pack, cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.pack = pack;
  while ((1 << p.shift) < p.pack) ++p.shift;
  const int queries = kRows / p.pack;
  p.qtiles = (int)((a.max_q + 2LL * queries - 1) / (2 * queries));
  p.scale2 = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (p.scale2 < 1e-30f) p.scale2 = 1e-30f;  // above 0, so that a masked score stays -inf
  p.negate = a.scale < 0;
#ifdef STIEF_TEST_HOOKS
  p.stall = test_stall_bytes();
  p.apart = test_tmem_apart();
#endif
  const long long blocks = 2LL * p.qtiles * (a.Hq / p.pack) * a.B;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const uint64_t rows = a.Nkv > 0 ? a.Nkv : 1, dk = (uint64_t)a.Hkv * 128;  // (no keys: the maps are never used)
  const int dq = 128 + a.dr;
  const void* k = a.Nkv > 0 ? a.k : a.q;
  const void* v = a.Nkv > 0 ? a.v : a.q;
  if (!encode_tiled_bf16_3d(&p.mq, a.q, {(uint64_t)dq, (uint64_t)a.Hq, (uint64_t)a.Nq}, {(uint64_t)dq * 2, (uint64_t)a.Hq * dq * 2},
                            {64, (uint32_t)p.pack, (uint32_t)queries}) ||
      !encode_tiled_bf16_3d(&p.mk, k, {64, rows, dk / 64}, {dk * 2, 128}, {64, kKeys / 2, 2}) ||
      !encode_tiled_bf16_3d(&p.mv, v, {64, rows, dk / 64}, {dk * 2, 128}, {64, kKeys, 1}) ||
      !encode_tiled_bf16_2d(&p.mp, a.Nkv > 0 ? a.pe : a.q, (uint64_t)a.dr, rows, (uint64_t)a.dr * 2, 64, kKeys / 2,
                            CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(stief_prefill_kernel), a.device, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, stief_prefill_kernel, p);
}

// CTAs that share the keys of a tile (prefill_one_tile.cu).  A split saves part of the walk, some 0.6
// us a step of 64 keys, and costs 2 to 3 us where tiles have all their rows.  It pays while all CTAs
// are resident, two an SM (clusters of four and eight leave some places empty), and the walk is long
// enough: 8 steps with an SM for each CTA, else 16, or 64 for eight CTAs a tile.  In us, with 1, 2, 4
// and 8 CTAs a tile and no position part:
//   1 query over 2001 keys, 4 heads          24.5  15.5  10.5   8.0
//   500 tokens, 4 heads                      10.2  11.4   8.9  10.6
//   8 chunks of 17 over 17 to 989, 4 heads   14.9  11.4   9.2  10.4
//   128 queries over 8256 keys, 32 heads     92.4  54.9  35.1  32.8
//   300 over 3300, 24 heads                  39.0  27.9  35.0  43.0
//   1500 tokens, 8 heads                     20.7  18.2  22.5  36.5
//   2 prompts of 500, 8 heads                10.3  11.7  11.6  24.1
// Below 8 steps a tile is not split, although four CTAs would save 1.3 us in the second row: the steps
// are a guess from the arrays' sizes, and a split of fewer costs as much as it saves elsewhere.  The
// worst case known of the rule is 128 queries over 2128 keys, 128 heads: 35 us with two, 34 with one.
int split_of(const PrefillArgs& a, int pack) {
  const long long queries = kRows / pack, groups = a.Hq / pack;
  // No more tiles than this, and about so many steps in the longest walk: the lengths are on the GPU,
  // and those of several sequences are taken to differ.
  const long long each = a.B * ((a.max_q + queries - 1) / queries), all = a.Nq / queries + a.B;
  const long long tiles = (each < all ? each : all) * groups, steps = (a.B > 1 ? a.Nkv * 3LL / 2 : a.Nkv) / kKeys / a.B;
  if (steps < 8) return 1;
  auto fits = [&](int c) { return 4 * c * tiles <= 7LL * a.sms; };
  if (16 * tiles <= a.sms || (8 * tiles <= a.sms && steps >= 16) || (fits(8) && steps >= 64)) return 8;
  if (fits(4) && (4 * tiles <= a.sms || steps >= 16)) return 4;
  return tiles <= a.sms && steps >= 16 ? 2 : 1;
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  // Query heads that share a KV head go into the rows of one tile (8 prompts of 65 to 1500 queries,
  // 32 heads over 8: 84.9 us against 109.5 with a head a tile and steps of 128 keys).
  const int group = a.Hq / a.Hkv, pack = group <= kRows && (group & (group - 1)) == 0 ? group : 1;
  // With a position part: a pair starts later and shares the later tile's keys, so the walk over them
  // has to be long (1000 tokens, 32 heads: single tiles 23.2 us, pairs 24.4; 8 prompts of 65 to 1500,
  // 105 and 113, over 500 cached tokens each, 193 and 185).  Where the rows of a prompt fill one tile
  // at most, half of a pair has nothing to do, which matters once there are more tiles than SMs (8
  // chunks of 128 over 4128 keys, 32 heads: 111 and 163 us; 1 of 128 over 8128 keys, 128 heads: 194
  // and 159).
  const bool spare = (long long)a.max_q * pack <= kRows && (long long)a.B * (a.Hq / pack) > a.sms;
  const bool pair = a.dr > 0 && a.Nkv > 1024LL * a.B && !spare && (a.max_q / kRows + 2LL) * a.B * a.Hq < (1LL << 31);
  const int split = split_of(a, pack);
  if (split > 1) return launch_prefill_one_tile(a, pack, split, stream);
  return pair ? launch_pair(a, pack, stream) : launch_prefill_one_tile(a, pack, 1, stream);
}

}  // namespace stief
