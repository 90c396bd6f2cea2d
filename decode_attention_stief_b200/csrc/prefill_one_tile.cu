// prefill_one_tile.cu -- causal attention of ragged prompts over per-head keys and values, for sm_100a:
// two CTAs an SM, a tile of 128 query rows each (prefill_attention.cu has the formula, the form in
// which two CTAs share the keys, and the rule between them).
//
// A CTA walks the keys in steps of 64; both products run on tcgen05:
//     S [128 x 64] = Q . K^T,    O [128 x 128] += P . V,
// P in tensor memory over its S, V MN-major as it lies in memory.  S has two buffers of 64 columns,
// so that the next step's scores are there when a step's softmax ends, and the softmax warps never
// wait for a product; with O that is half of the tensor memory, and the other CTA of the SM has the
// other half: one's products, start and end overlap the other's exponentials.  (Steps of 128 keys
// have room for one buffer, and each step's scores wait for the last step's product: 2500 tokens,
// 32 heads, 63.8 us against 58.5; 8 chunks of 512 over 3012 keys, 260 against 245.)
// The rows of a tile are (query, head) pairs of the heads that share a KV head where their number
// divides 128: short chunks leave fewer rows empty, and fewer tiles cross the diagonal (32 single
// queries over 4001 keys, 32 heads over 8: 252 us a head a tile, 82 packed).
// With a position part a query row is 192 columns and one slot of keys fits instead of two: the
// slot whose successor is needed latest, because scores are computed a step ahead (two slots of keys
// and one of values: 1 chunk of 128 over 8128 keys, 128 heads, 200 us; this way 182).
// Where tiles are few and walks long (split_of in prefill_attention.cu), the CTAs of a cluster share a
// tile's keys: each walks its part, leaves its rows of O, m and l in fp32 in its shared memory, and
// joins its share of the rows from all of them (a part counts if the row sees a key of it, so that a NaN
// reaches the row as in the other forms).  1 query over 8001 keys, 8 heads over 1: 15.5 us
// against 82; over 32001: 45 against 313; 8 chunks of 17 over 989, 4 heads: 9.2 against 14.9.
//   warp 0: TMA producer; warp 1: MMA issuer; warp 2: zeroes the value rows past n_k in the last step
//   (they may hold NaN, and 0 * NaN is NaN); warps 4-7: softmax, a thread a row, and the output.
// The softmax's reference is the first step's maximum of the row and moves only when a score passes
// it by more than 2^60 (weights and sums are floating-point numbers: a large weight loses nothing);
// the warp then rescales its rows of O, once the last product is done.  Weights are rounded to bf16 for
// the second product (the tensor cores take both operands in one type, and a second product with what
// the rounding leaves would make the products half as many again); the sum l adds them unrounded: with rounded ones
// the error against 64 bits is 2 % smaller and the time 1 to 3 % larger.
//
// What bounds it: shared memory.  A step's products read 64 KB of it (the queries for every 64 keys
// anew) and its copies write 32: 768 cycles at 128 bytes a cycle, where the products alone would take
// 512 and the exponentials, 16 a cycle on an SM, another 512 beside them.  Of the some 1900 cycles that
// a step of both CTAs takes that is 80 %; the tensor cores are busy for 47 % (chunks) of the time.
// (Pairs of CTAs, each with half of the keys and values, ask less of it: 8 chunks of 512 over 3012 keys
// 216 us against 239; but 2500 tokens 66 against 58, and 8192, 32 heads over 8, 456 both.  Not built.)
// Measured: 8192 tokens, 32 heads over 8: 456 us, 1.21 PFLOP/s (535 us in long runs under the power cap);
// 8 prompts of 65 to 1500: 80 to 85 us, 0.74 PFLOP/s (its diagonal tiles compute twice what is counted);
// 5 prompts of up to 64: 5.7 us.
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
constexpr uint32_t kBlock = kKeys * 128;   // bytes of 64 key or value rows x 64 columns
constexpr int kThreads = 256;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kOCol = 128;            // S at 0 and 64, O at 128
constexpr float kRescale = 60.f;           // log2 units a score may pass the reference by
constexpr float kFloor = -1e30f;
constexpr int kMaxSplit = 8;                // a cluster of any GPU

struct Args {
  CUtensorMap mq;   // q [Nq][Hq][128], box 64 columns x pack heads x 128 / pack queries
  CUtensorMap mk;   // k [Nkv] rows in blocks of 64 columns, box 64 x 64 x 2
  CUtensorMap mv;   // v, same
  CUtensorMap mp;   // k_pe [Nkv][dr], box 64 x 64
  PrefillArgs a;
  int pack;         // heads of a tile: its row r is query r / pack, head r % pack (pack divides 128)
  int shift;        // log2(pack)
  int qtiles;       // tiles of the longest sequence
  int split;        // CTAs (a cluster) that share a tile's keys: 1, 2, 4 or 8
  float scale2;     // |scale| * log2(e)
  int negate;       // scale < 0: the products are negated instead
#ifdef STIEF_TEST_HOOKS
  uint32_t stall;   // test build: bytes expected of the first copy that none delivers
#endif
};

template <bool kPe>
struct Form {
  static constexpr int kBlocks = kPe ? 3 : 2;  // of 64 columns in a query or key row
  static constexpr int kKSlots = kPe ? 1 : 2;
  static constexpr uint32_t kKeyBytes = kBlocks * kBlock, kValueBytes = 2 * kBlock;
  static constexpr uint32_t kK = kBlocks * kAtom, kV = kK + kKSlots * kKeyBytes, kBars = kV + 2 * kValueBytes;
  static constexpr uint32_t kTotal = kBars + 8 * 20;
};
static_assert(2 * (Form<true>::kTotal + 1024) <= 228 * 1024, "two CTAs share an SM");
// The parts of a split tile: its rows of O in fp32, then (m, l) of each, over what the queries, keys
// and values took.
constexpr uint32_t kPartRow = 512, kPartMl = kRows * kPartRow;
static_assert(kPartMl + kRows * 8 <= Form<false>::kBars, "the parts fit");

}  // namespace

template <bool kPe, bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) stief_prefill_one_tile_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using F = Form<kPe>;
  constexpr int kKSlots = F::kKSlots;
  const PrefillArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + F::kBars);  // [2]
  uint64_t* k_empty = k_full + 2;   // [2]
  uint64_t* v_full = k_full + 4;    // [2]
  uint64_t* v_empty = k_full + 6;   // [2]
  uint64_t* s_full = k_full + 8;    // [2] S of a step is in TMEM
  uint64_t* p_full = k_full + 10;   // [2] P of a step is
  uint64_t* pv_done = k_full + 12;  // [2] O of a step is added
  uint64_t* q_full = k_full + 14;
  uint64_t* o_full = k_full + 15;   // O is complete
  uint64_t* partial = k_full + 16;  // the last values are in and are not 64
  uint64_t* tail = k_full + 17;     // their rows past n_k are cleared
  uint64_t* drain = k_full + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 19);
#ifdef STIEF_TEST_HOOKS
  const uint32_t stall = p.stall;
#else
  constexpr uint32_t stall = 0u;
#endif
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) report(a.dev_status, STIEF_DEV_SMEM_ALIGN);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(&k_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 14; i < 19; ++i) mbar_init(&k_full[i], 1);
    fence_barrier_init();
  }
  const unsigned tile = kSplit ? blockIdx.x / (unsigned)p.split : blockIdx.x;
  const int rank = kSplit ? (int)cluster_rank() : 0;
  const int groups = a.Hq >> p.shift, gb = groups * a.B, rest = (int)(tile % (unsigned)gb);
  const int qt = p.qtiles - 1 - (int)(tile / (unsigned)gb);
  const int b = rest / groups, h0 = (rest % groups) << p.shift, hk = h0 / (a.Hq / a.Hkv);

  pdl_wait();
  const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
  int k0 = __ldg(a.kv_start + b);
  const int k1 = __ldg(a.kv_start + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.Nq || k0 < 0 || k1 < k0 || k1 > a.Nkv || q1 - q0 > a.max_q) {
    if (tid == 0 && rank == 0 && h0 == 0 && qt == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    return;
  }
  const int nq = q1 - q0, n_all = k1 - k0, first = qt * (kRows >> p.shift);  // first query
  if (first >= nq) return;
  // steps of keys that the tile's last query sees
  const int last = min(nq, first + (kRows >> p.shift)) - 1;
  const long long most = (long long)last + n_all - nq + 1;
  int n = most > 0 ? (int)((min(most, (long long)n_all) + kKeys - 1) / kKeys) : 0;
  int n_k = n_all, before = 0;  // keys from k0 on, and those of the CTAs before this one
  const int per = kSplit ? (n + p.split - 1) / p.split : n;  // steps of a CTA
  if (kSplit) {
    const int js = min(n, rank * per);
    n = min(per, n - js);
    before = js * kKeys;
    k0 += before;
    n_k = min(n_all - before, n * kKeys);
  }

  // (only after the dependency wait, and before this kernel's own dependents may start: a CTA that
  // holds tensor memory while it waits for another kernel must not starve one of that kernel's)
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  uint32_t nan = 0, which = 0;  // NaN among a row's outputs, and the warp's rows with one

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (n > 0 && elect_one()) {
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      int nk = 0, nv = 0;
      auto load_k = [&](int j) -> bool {
        const int slot = j % kKSlots;
        if (j >= kKSlots && !mbar_wait_ready(&k_empty[slot], (uint32_t)((j / kKSlots) & 1) ^ 1u, a.dev_status)) return false;
        uint8_t* at = smem + F::kK + (uint32_t)slot * F::kKeyBytes;
        mbar_arrive_expect_tx(&k_full[slot], F::kKeyBytes);
        tma_load_3d(at, &p.mk, 0, k0 + j * kKeys, hk * 2, &k_full[slot], keep);
        if (kPe) tma_load_2d(at + 2 * kBlock, &p.mp, 0, k0 + j * kKeys, &k_full[slot], keep);
        return true;
      };
      auto load_v = [&](int j) -> bool {
        if (j >= 2 && !mbar_wait_ready(&v_empty[j & 1], (uint32_t)((j >> 1) & 1) ^ 1u, a.dev_status)) return false;
        mbar_arrive_expect_tx(&v_full[j & 1], F::kValueBytes);
        tma_load_3d(smem + F::kV + (uint32_t)(j & 1) * F::kValueBytes, &p.mv, 0, k0 + j * kKeys, hk * 2, &v_full[j & 1], keep);
        return true;
      };
      mbar_arrive_expect_tx(q_full, F::kBlocks * kAtom + stall);
      for (int c = 0; c < F::kBlocks; ++c) tma_load_3d(smem + (uint32_t)c * kAtom, &p.mq, 64 * c, h0, q0 + first, q_full, once);
      // (with two slots of keys a step's are requested one step before its values: theirs are free first)
      bool ok = true;
      if (kKSlots == 2) ok = load_k(nk++);
      for (int j = 0; ok && j < n; ++j) {
        if (nk < n) {
          if (!(ok = load_k(nk))) break;
          ++nk;
        }
        ok = load_v(nv);
        if (ok) ++nv;
      }
      // every requested copy lands before the shared memory is released
      mbar_wait_ready(q_full, 0, nullptr);
      for (int j = max(0, nk - kKSlots); j < nk; ++j)
        mbar_wait_ready(&k_full[j % kKSlots], (uint32_t)((j / kKSlots) & 1), nullptr);
      for (int j = max(0, nv - 2); j < nv; ++j) mbar_wait_ready(&v_full[j & 1], (uint32_t)((j >> 1) & 1), nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (n > 0 && elect_one()) {
      const uint32_t id_s = idesc_bf16_f32(128, kKeys, false, false) | (p.negate ? 1u << 13 : 0u);
      const uint32_t id_o = idesc_bf16_f32(128, 128, false, true);
      const uint64_t dq = sw128_desc(smem_u32(smem)), dk0 = sw128_desc(smem_u32(smem + F::kK));
      const uint64_t dv0 = sw128_mn_desc(smem_u32(smem + F::kV), kBlock);
      const int pe_steps = a.dr / 16;
      auto wait_k = [&](int j) -> bool { return mbar_wait_ready(&k_full[j % kKSlots], (uint32_t)((j / kKSlots) & 1), a.dev_status); };
      auto issue_s = [&](int j) {
        tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((j % kKSlots) * (F::kKeyBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16(tmem + (uint32_t)(j & 1) * kKeys, dq + (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2,
                    dk + (kk >> 2) * (kBlock >> 4) + (kk & 3) * 2, id_s, kk > 0);
        if (kPe)
          for (int kk = 0; kk < pe_steps; ++kk)
            umma_bf16(tmem + (uint32_t)(j & 1) * kKeys, dq + 2 * (kAtom >> 4) + 2 * kk, dk + 2 * (kBlock >> 4) + 2 * kk,
                      id_s, 1);
        umma_commit(&s_full[j & 1]);
        umma_commit(&k_empty[j % kKSlots]);
      };
      bool ok = mbar_wait_ready(q_full, 0, a.dev_status);
      for (int j = 0; j < 2 && j < n && ok; ++j) {
        ok = wait_k(j);
        if (ok) issue_s(j);
      }
      for (int j = 0; ok && j < n; ++j) {
        // (what has long arrived is waited for first: a test of a barrier takes some 250 cycles next
        // to the products' shared-memory traffic)
        if (!(ok = mbar_wait_ready(&v_full[j & 1], (uint32_t)((j >> 1) & 1), a.dev_status))) break;
        if (j == n - 1 && n * kKeys > n_k) {  // rows past n_k must not be NaN
          mbar_arrive(partial);
          if (!(ok = mbar_wait_ready(tail, 0, a.dev_status))) break;
        }
        if (kKSlots == 2 && j + 2 < n && !(ok = wait_k(j + 2))) break;
        if (!(ok = mbar_wait_ready(&p_full[j & 1], (uint32_t)((j >> 1) & 1), a.dev_status))) break;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((j & 1) * (F::kValueBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_ts(tmem + kOCol, tmem + (uint32_t)(j & 1) * kKeys + kk * 8, dv + kk * 128, id_o, j > 0 || kk > 0);
        umma_commit(&v_empty[j & 1]);
        umma_commit(&pv_done[j & 1]);
        if (j + 2 < n) {
          if (kKSlots == 1 && !(ok = wait_k(j + 2))) break;
          issue_s(j + 2);  // into the buffer that P has left
        }
      }
      if (ok) umma_commit(o_full);
      // products left by a timeout get a bounded chance to finish; on the normal path this is the
      // end of the last one
      umma_commit(drain);
      mbar_wait_ready(drain, 0, nullptr);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- value rows past n_k
    if (n > 0 && n * kKeys > n_k) {
      const uint64_t since = global_timer_ns();
      bool got = mbar_try_wait(partial, 0);
      while (!got && global_timer_ns() - since < 8 * kWaitLimitNs) got = mbar_try_wait(partial, 0);
      if (__all_sync(~0u, got)) {
        uint8_t* v = smem + F::kV + (uint32_t)((n - 1) & 1) * F::kValueBytes;
        for (int c = 0; c < 2; ++c)
          for (int e = (n_k - (n - 1) * kKeys) * 8 + lane; e < kKeys * 8; e += 32)
            *reinterpret_cast<uint4*>(v + c * kBlock + e * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(tail);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax and output
    const int quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16, o_col = tmem + lanes + kOCol;
    const int r0 = quad * 32, query = first + ((r0 + lane) >> p.shift);  // the thread's row
    const int sees = (int)max(0LL, min((long long)n_all, (long long)query + n_all - nq + 1));  // keys it sees
    const int seen = sees - before;  // (at or below 0: none of this CTA's)
    const int all = __shfl_sync(~0u, seen, 0);  // keys that every row of the warp sees
    const uint64_t scale2 = pack2(p.scale2, p.scale2);
    float m = kFloor;
    uint64_t l0 = 0, l1 = 0;
    bool ok = true;
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
      if (lane == 0) mbar_arrive(&p_full[j & 1]);
    }
    // the output: zeros for a row that sees no key
    if (ok && n > 0) ok = __all_sync(~0u, mbar_wait_ready(o_full, 0, a.dev_status));
    if (kSplit && ok) {
      // this CTA's part; a row's 16-byte pieces are rotated by its number
      tc_fence_after();
      const uint64_t ls = add2(l0, l1);
      uint8_t* part = smem + (uint32_t)(r0 + lane) * kPartRow;
      *reinterpret_cast<float2*>(smem + kPartMl + (uint32_t)(r0 + lane) * 8) = make_float2(m, lo_of(ls) + hi_of(ls));
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t v[32] = {};
        if (n > 0) {
          tmem_ld32(o_col + c, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<uint4*>(part + ((((c + e) >> 2) ^ lane) << 4)) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    if (!kSplit && ok) {
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
  if (kSplit) cluster_sync();  // every CTA's part is in its shared memory
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (kSplit) {
    // each CTA joins its share of the rows, a warp a row
    const int rows = kRows / p.split;
    for (int i = warp; i < rows; i += kThreads / 32) {
      const int r = rank * rows + i, query = first + (r >> p.shift), h = h0 + (r & (p.pack - 1));
      if (query >= nq) break;
      float2 ml[kMaxSplit];
      float4 o[kMaxSplit];
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < p.split) {
          const uint32_t at = in_cta(smem, (uint32_t)k);
          ml[k] = load_cluster_f2(at + kPartMl + (uint32_t)r * 8);
          o[k] = load_cluster_f4(at + (uint32_t)r * kPartRow + (uint32_t)((lane ^ (r & 31)) << 4));
        }
      // A part counts if the row sees a key of it, whatever its sum: a NaN must reach the row, and a row
      // whose scores are all -inf is 0 / 0, as in a tile that is not split.
      const int sees = (int)max(0LL, min((long long)n_all, (long long)query + n_all - nq + 1));
      float top = kFloor, l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < p.split && k * per * kKeys < sees) top = fmaxf(top, ml[k].x);
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k)
        if (k < p.split && k * per * kKeys < sees) {
          const float f = fast_exp2(ml[k].x - top);
          l += f * ml[k].y;
          x.x += f * o[k].x;
          x.y += f * o[k].y;
          x.z += f * o[k].z;
          x.w += f * o[k].w;
        }
      const float inv = sees > 0 ? 1.f / l : 0.f;  // (zeros for a row that sees no key)
      const uint2 y = make_uint2(pack_bf16x2_rn(x.x * inv, x.y * inv), pack_bf16x2_rn(x.z * inv, x.w * inv));
      *reinterpret_cast<uint2*>(a.out + ((size_t)(q0 + query) * a.Hq + h) * 128 + lane * 4) = y;
      if (__any_sync(~0u, has_nan(nan_of(y.x, y.y, 0)))) which |= 1u << (i / (kThreads / 32));
    }
    __syncwarp();
    cluster_sync();  // no part is read any more
  }
  if (__builtin_expect(which != 0, 0)) {
    __syncwarp();
    const int first_row = kSplit ? rank * (kRows / p.split) + warp : (warp & 3) * 32;
    redo_rows(a, p.shift, p.qtiles, tile, kRows, kKeys, first_row, kSplit ? kThreads / 32 : 1, which,
              p.negate ? -p.scale2 : p.scale2);
  }
}

namespace {

template <bool kPe, bool kSplit>
cudaError_t launch(const PrefillArgs& a, int pack, int split, cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.pack = pack;
  p.split = split;
  while ((1 << p.shift) < p.pack) ++p.shift;
  const int queries = kRows / p.pack;
  p.qtiles = (int)((a.max_q + (long long)queries - 1) / queries);
  p.scale2 = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (p.scale2 < 1e-30f) p.scale2 = 1e-30f;  // above 0, so that a masked score stays -inf
  p.negate = a.scale < 0;
#ifdef STIEF_TEST_HOOKS
  p.stall = test_stall_bytes();
#endif
  const long long blocks = (long long)p.qtiles * (a.Hq / p.pack) * a.B * split;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const uint64_t rows = a.Nkv > 0 ? a.Nkv : 1, dk = (uint64_t)a.Hkv * 128;  // (no keys: the maps are never used)
  const int dq = 128 + a.dr;
  const void* k = a.Nkv > 0 ? a.k : a.q;
  const void* v = a.Nkv > 0 ? a.v : a.q;
  if (!encode_tiled_bf16_3d(&p.mq, a.q, {(uint64_t)dq, (uint64_t)a.Hq, (uint64_t)a.Nq}, {(uint64_t)dq * 2, (uint64_t)a.Hq * dq * 2},
                            {64, (uint32_t)p.pack, (uint32_t)queries}) ||
      !encode_tiled_bf16_3d(&p.mk, k, {64, rows, dk / 64}, {dk * 2, 128}, {64, kKeys, 2}) ||
      !encode_tiled_bf16_3d(&p.mv, v, {64, rows, dk / 64}, {dk * 2, 128}, {64, kKeys, 2}) ||
      (kPe && !encode_tiled_bf16_2d(&p.mp, a.Nkv > 0 ? a.pe : a.q, (uint64_t)a.dr, rows, (uint64_t)a.dr * 2, 64, kKeys,
                                    CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(stief_prefill_one_tile_kernel<kPe, kSplit>), a.device, (int)Form<kPe>::kTotal);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Form<kPe>::kTotal;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, stief_prefill_one_tile_kernel<kPe, kSplit>, p);
}

}  // namespace

cudaError_t launch_prefill_one_tile(const PrefillArgs& a, int pack, int split, cudaStream_t stream) {
  if (split > 1) return a.dr > 0 ? launch<true, true>(a, pack, split, stream) : launch<false, true>(a, pack, split, stream);
  return a.dr > 0 ? launch<true, false>(a, pack, 1, stream) : launch<false, false>(a, pack, 1, stream);
}

}  // namespace stief
