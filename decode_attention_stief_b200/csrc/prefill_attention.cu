// prefill_attention.cu -- causal attention of ragged prompts over per-head keys and values, for
// sm_100a.  Query i of sequence b (n_q queries, n_k keys) sees keys j <= i + n_k - n_q:
//     o_i = softmax_j(scale * (q_i . k_j + q^R_i . k^R_j)) v_j,
// one pass over the keys with a running maximum and sum.
//
// What bounds it: the products (2 (256 + dr) operations a visible pair and head) and, nearly as
// long, one exponential a pair: 16 a cycle on an SM against 4096 multiply-adds.
//
// Two kernels.  Without a position part, prefill_one_tile.cu: two CTAs an SM, a tile of 128 query
// rows each.  With one a CTA's rows are half as long again and two such CTAs have room for one step
// of 64 keys each: the products with 64 keys read shared memory for longer than they compute, and
// what is in flight does not cover the way to memory.  So this file's kernel takes two tiles of
// queries that share steps of 128 keys (launch_prefill below has the rule and both sides of it).
// 8192 tokens, 32 heads, dr 64: 550 us, 1.25 PFLOP/s, the tensor cores busy for 63 % of it (1.20
// PFLOP/s under the power cap of a long run).
//
// A CTA takes 256 queries of one head as two tiles of 128 and walks the keys in tiles of 128;
// both products run on tcgen05 with M = N = 128:
//     S_w = Q_w . K^T      (Q, K in shared memory, K-major, 128-byte swizzle)
//     O_w += P_w . V       (P in tensor memory, V MN-major as it lies in memory)
// TMEM holds S_0, S_1, O_0, O_1, 128 columns each: all of it.  P_w overwrites S_w, whose row a
// thread holds in registers meanwhile.  The tensor cores work for one tile of queries while the
// softmax of the other runs.
//   warp 0: TMA producer; warps 1 and 3: MMA issuers of the two tiles; warp 2: zeroes the value
//   rows past n_k in the last tile (they may hold NaN, and 0 * NaN is NaN); warps 4-7 and 8-11:
//   softmax of the two tiles, one thread a query row, and the output.
// The reference of the running maximum moves only when a score passes it by more than 2^60
// (weights and sums are floating-point numbers: a large weight loses nothing): a warp then rescales
// its own rows of O_w, whose last product is complete when S_w of the next tile is, because the
// products run in order.
// CTAs start with the longest tiles of queries; a tile of queries none of whose rows exists ends
// at once.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"
#include "umma.cuh"

namespace stief {

namespace {

constexpr int kRows = 128;                 // queries a tile, keys a tile
constexpr uint32_t kAtom = kRows * 128;    // bytes of 128 rows x 64 columns
constexpr float kRescale = 60.f;           // log2 units a score may pass the reference by
constexpr float kFloor = -1e30f;
constexpr int kAtoms = 3;                  // of 64 columns in a query row
// Slots of 64 value rows: what fits.  (Not above 4: a tile's barrier, one of two in turn, is armed again
// only after a wait for the halves of two tiles before.)
constexpr int kHalves = 3;
constexpr uint32_t kKeys = 2 * kAtom;      // bytes of a key tile without the position part
constexpr uint32_t kHalf = kAtom;          // bytes of 64 value rows (two atoms of 64 columns)

struct Args {
  CUtensorMap mq;   // q [Nq][Hq * (128 + dr)], box 64 x 128 (dr > 0)
  CUtensorMap mk;   // k [Nkv] rows in blocks of 64 columns, box 64 x 128 x 2
  CUtensorMap mv;   // v, box 64 x 64 x 2
  CUtensorMap mp;   // k_pe [Nkv][dr], box 64 x 128
  PrefillArgs a;
  int qtiles;       // tiles of 256 queries of the longest sequence
  float scale2;     // |scale| * log2(e)
  int negate;       // scale < 0: the products are negated instead
#ifdef STIEF_TEST_HOOKS
  uint32_t stall;     // test build: bytes expected of the first copy that none delivers
#endif
};

// Two tiles of queries, two slots of keys, one of position parts, slots of 64 value rows.  A key tile's
// position part is wanted between its two products only, so one slot of it is enough, and what
// that saves holds a third half tile of values: with two, the next one arrived too late.
constexpr uint32_t kSmemK = 2 * kAtoms * kAtom, kSmemPe = kSmemK + 2 * kKeys, kSmemV = kSmemPe + kAtom;
constexpr uint32_t kSmemBars = kSmemV + kHalves * kHalf, kSmem = kSmemBars + 8 * (6 + kHalves + 12);
static_assert(kSmem <= kMaxSmemPerBlock - 1024, "one CTA's shared memory, beside the static part");

}  // namespace

__global__ void __launch_bounds__(384, 1) stief_prefill_kernel(const __grid_constant__ Args p) {
  constexpr uint32_t kTmemCols = 512;  // S_w at 128 w, O_w at 256 + 128 w
  constexpr uint32_t kOCol = 256;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t tmem_slot;
  const PrefillArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kSmemBars);  // [2]
  uint64_t* k_empty = k_full + 2;           // [2]
  uint64_t* v_full = k_full + 4;            // [2] both halves of a value tile, tiles in turn
  uint64_t* v_empty = k_full + 6;           // [kHalves]
  uint64_t* q_full = v_empty + kHalves;     // [2]
  uint64_t* s_full = q_full + 2;            // [2] S_w of a tile is in TMEM (and O_w before it)
  uint64_t* p_full = q_full + 4;            // [2] P_w of a tile is
  uint64_t* o_full = q_full + 6;            // [2] O_w is complete
  uint64_t* partial = q_full + 8;           // the last value tile is in and is not full
  uint64_t* tail = q_full + 9;              // its rows past n_k are cleared
  uint64_t* drain = q_full + 10;            // [2]

#ifdef STIEF_TEST_HOOKS
  const uint32_t stall = p.stall;
#else
  constexpr uint32_t stall = 0u;
#endif
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) report(a.dev_status, STIEF_DEV_SMEM_ALIGN);
    return;
  }
  const int hb = a.Hq * a.B, rest = (int)(blockIdx.x % (unsigned)hb);
  const int qt = p.qtiles - 1 - (int)(blockIdx.x / (unsigned)hb);
  const int b = rest / a.Hq, h = rest % a.Hq, hk = h / (a.Hq / a.Hkv);

  pdl_wait();
  const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
  const int k0 = __ldg(a.kv_start + b), k1 = __ldg(a.kv_start + b + 1);
  const bool bad_rows = q0 < 0 || q1 < q0 || q1 > a.Nq || k0 < 0 || k1 < k0 || k1 > a.Nkv || q1 - q0 > a.max_q;
  if (bad_rows) {
    if (tid == 0 && h == 0 && qt == 0) report(a.dev_status, STIEF_DEV_BAD_LENGTH);
    return;
  }
  const int nq = q1 - q0, n_k = k1 - k0, first = qt * 2 * kRows;
  if (first >= nq) return;
  // key tiles that each tile of queries sees: up to its last row's last key
  int nt[2] = {0, 0};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int begin = first + w * kRows, last = min(nq, begin + kRows) - 1;  // last row
    const long long seen = begin < nq ? (long long)last + n_k - nq + 1 : 0;
    nt[w] = seen > 0 ? (int)((min(seen, (long long)n_k) + kRows - 1) / kRows) : 0;
  }
  const int tiles = max(nt[0], nt[1]);

  if (tid == 0 && tiles > 0) {
    // a slot is empty when both tiles of queries have read it.  (Where one of them sees a key tile
    // less, that is the last one, whose slot nobody waits for.)
    const uint32_t users = (nt[0] > 0) + (nt[1] > 0);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], users);
    }
    for (int i = 0; i < kHalves; ++i) mbar_init(&v_empty[i], users);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&v_full[w], 1);
      mbar_init(&q_full[w], 1);
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&o_full[w], 1);
      mbar_init(&drain[w], 1);
    }
    mbar_init(partial, (nt[0] == tiles) + (nt[1] == tiles));
    mbar_init(tail, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now: a kernel that starts while this CTA has no tensor memory yet could take all of it
  // and then wait for this kernel to end.
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;

  if (warp < 4) {
    // (the shares add up to what the block was launched with: 3 x 168)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      if (elect_one()) {
        const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
        const int dq = 128 + a.dr;
        int nkl = 0, nvl = 0;  // key tiles and value halves requested
        const bool half[2] = {nt[0] > 0, nt[1] > 0};
        auto load_q = [&](int w) {
          mbar_arrive_expect_tx(&q_full[w], (uint32_t)kAtoms * kAtom + stall);
          for (int c = 0; c < kAtoms; ++c)
            tma_load_2d(smem + (uint32_t)(w * kAtoms + c) * kAtom, &p.mq, h * dq + 64 * c, q0 + first + w * kRows,
                        &q_full[w], once);
        };
        int vs = 0;
        uint32_t vp = 0;  // parity of the half's current use
        bool ok = true;
        for (int i = 0; ok && i < tiles; ++i) {
          const int row = k0 + i * kRows, ks = i % 2;
          if (i == 0 && half[0]) load_q(0);
          if (i >= 2 && !(ok = mbar_wait_ready(&k_empty[ks], (uint32_t)(i / 2 & 1) ^ 1u, a.dev_status))) break;
          mbar_arrive_expect_tx(&k_full[ks], kKeys + kAtom);
          tma_load_3d(smem + kSmemK + (uint32_t)ks * kKeys, &p.mk, 0, row, hk * 2, &k_full[ks], keep);
          ++nkl;
          // (the one slot of position parts is free when the last tile's keys are)
          if (i > 0) ok = mbar_wait_ready(&k_empty[(i - 1) % 2], (uint32_t)((i - 1) / 2 & 1), a.dev_status);
          tma_load_2d(smem + kSmemPe, &p.mp, 0, row, &k_full[ks], keep);  // (after a timeout too: it is expected)
          if (!ok) break;
          if (i == 0 && half[1]) load_q(1);
          for (int c = 0; c < 2; ++c) {
            if (nvl >= kHalves && ok) ok = mbar_wait_ready(&v_empty[vs], vp ^ 1u, a.dev_status);
            if (!ok && c == 0) break;
            if (c == 0) mbar_arrive_expect_tx(&v_full[i & 1], 2 * kHalf);
            tma_load_3d(smem + kSmemV + (uint32_t)vs * kHalf, &p.mv, 0, row + 64 * c, hk * 2, &v_full[i & 1], keep);
            ++nvl;
            if (++vs == kHalves) vs = 0, vp ^= 1u;
          }
        }
        // every requested copy lands before the shared memory is released
        if (tiles > 0) {
          for (int w = 0; w < 2; ++w)
            if (half[w]) mbar_wait_ready(&q_full[w], 0, nullptr);
          for (int j = max(0, nkl - 2); j < nkl; ++j)
            mbar_wait_ready(&k_full[j % 2], (uint32_t)(j / 2 & 1), nullptr);
          for (int j = max(0, nvl / 2 - 2); j < nvl / 2; ++j)
            mbar_wait_ready(&v_full[j & 1], (uint32_t)((j >> 1) & 1), nullptr);
        }
      }
    } else if (warp == 1 || warp == 3) {
      // -------------------------------------------------------------- MMA issuers, one a query tile
      // (one thread for both spent a third of its time testing barriers, which costs hundreds of
      // cycles while the products read shared memory, and kept the other tile's products waiting)
      const int w = warp >> 1, n = w ? nt[1] : nt[0];
      if (n > 0 && elect_one()) {
        const uint32_t id_s = idesc_bf16_f32(128, 128, false, false) | (p.negate ? 1u << 13 : 0u);
        const uint32_t id_o = idesc_bf16_f32(128, 128, false, true);
        const uint32_t k_addr = smem_u32(smem + kSmemK), v_addr = smem_u32(smem + kSmemV);
        const uint32_t s_col = tmem + (uint32_t)w * 128u, o_col = s_col + kOCol;
        const uint64_t dq = sw128_desc(smem_u32(smem) + (uint32_t)(w * kAtoms) * kAtom);
        const uint64_t dp = sw128_desc(smem_u32(smem + kSmemPe));
        const int pe_steps = a.dr / 16;
        int va = 0;
        auto wait_k = [&](int i) -> bool {
          return mbar_wait_ready(&k_full[i % 2], (uint32_t)(i / 2 & 1), a.dev_status);
        };
        auto issue_s = [&](int i) {
          tc_fence_after();
          const uint64_t dk = sw128_desc(k_addr + (uint32_t)(i % 2) * kKeys);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(s_col, dq + (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2, dk + (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2,
                      id_s, kk > 0);
          for (int kk = 0; kk < pe_steps; ++kk)
            umma_bf16(s_col, dq + 2 * (kAtom >> 4) + 2 * kk, dp + 2 * kk, id_s, 1);
          umma_commit(&s_full[w]);
          umma_commit(&k_empty[i % 2]);
        };
        bool ok = mbar_wait_ready(&q_full[w], 0, a.dev_status) && wait_k(0);
        // (the second tile starts when the first has its weights: half a turn behind it)
        if (w == 1 && nt[0] > 0 && ok) ok = mbar_wait_ready(&p_full[0], 0, a.dev_status);
        if (ok) issue_s(0);
        for (int i = 0; ok && i < n; ++i) {
          const int vb = va + 1 == kHalves ? 0 : va + 1;
          if (!(ok = mbar_wait_ready(&v_full[i & 1], (uint32_t)((i >> 1) & 1), a.dev_status))) break;
          if (i == tiles - 1 && (i + 1) * kRows > n_k) {  // rows past n_k must not be NaN
            mbar_arrive(partial);
            if (!(ok = mbar_wait_ready(tail, 0, a.dev_status))) break;
          }
          const uint64_t dva = sw128_mn_desc(v_addr + (uint32_t)va * kHalf, kHalf / 2);
          const uint64_t dvb = sw128_mn_desc(v_addr + (uint32_t)vb * kHalf, kHalf / 2);
          if (!(ok = mbar_wait_ready(&p_full[w], (uint32_t)(i & 1), a.dev_status))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_bf16_ts(o_col, s_col + kk * 8, dva + kk * 128, id_o, i > 0 || kk > 0);
          umma_commit(&v_empty[va]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma_bf16_ts(o_col, s_col + 32 + kk * 8, dvb + kk * 128, id_o, 1);
          umma_commit(&v_empty[vb]);
          if (i + 1 < n) {
            if (!(ok = wait_k(i + 1))) break;
            issue_s(i + 1);
          } else {
            umma_commit(&o_full[w]);
          }
          va = vb + 1 == kHalves ? 0 : vb + 1;
        }
        // products left by a timeout get a bounded chance to finish; on the normal path this is
        // the end of the last one
        umma_commit(&drain[w]);
        mbar_wait_ready(&drain[w], 0, nullptr);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- value rows past n_k
      if (tiles > 0 && tiles * kRows > n_k) {
        const uint64_t since = global_timer_ns();
        bool got = mbar_try_wait(partial, 0);
        while (!got && global_timer_ns() - since < 8 * kWaitLimitNs) got = mbar_try_wait(partial, 0);
        if (__all_sync(~0u, got)) {
          const int valid = n_k - (tiles - 1) * kRows;
          for (int half = 0; half < 2; ++half) {
            uint8_t* v = smem + kSmemV + (uint32_t)((2 * tiles - 2 + half) % kHalves) * kHalf;
            for (int c = 0; c < 2; ++c)
              for (int e = max(0, valid - 64 * half) * 8 + lane; e < 64 * 8; e += 32)
                *reinterpret_cast<uint4*>(v + c * (kHalf / 2) + e * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(tail);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + lanes + (uint32_t)w * 128u, o_col = tmem + lanes + kOCol + (uint32_t)w * 128u;
    const int row = first + w * kRows + quad * 32 + lane;  // the thread's query
    const int shift = n_k - nq;
    const int seen = (int)max(0LL, min((long long)n_k, (long long)row + shift + 1));  // keys it sees
    // keys that every row of the warp sees (rows past n_q see no fewer)
    const int all = __shfl_sync(~0u, seen, 0);
    const uint64_t scale2 = pack2(p.scale2, p.scale2);
    float m = kFloor;
    uint64_t l0 = 0, l1 = 0;
    bool ok = true;
    for (int i = 0; i < nt[w]; ++i) {
      ok = __all_sync(~0u, mbar_wait_ready(&s_full[w], (uint32_t)(i & 1), a.dev_status));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, s[c]);
      tmem_wait_ld();
      const int lim = seen - i * kRows;
      if (all < (i + 1) * kRows) {  // some row of the warp does not see the whole tile
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e >= lim) s[c][e] = 0xff800000u;  // -inf
      }
      float t[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        t[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2) t[c] = max3(t[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
      }
      const float top = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * p.scale2, kFloor);
      if (i == 0) {
        m = top;
      } else {
        const bool move = top > m + kRescale;
        if (__any_sync(~0u, move)) {  // rescale this warp's rows of O
          const float f = move ? fast_exp2(m - top) : 1.f;
          if (move) m = top;
          const uint64_t f2 = pack2(f, f);
          l0 = fma2(l0, f2, 0);
          l1 = fma2(l1, f2, 0);
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tmem_ld16(o_col + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_st16(o_col + c, v);
          }
        }
      }
      const uint64_t m2 = pack2(-m, -m);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w16[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t x =
              fma2(((uint64_t)s[c][2 * e + 1] << 32) | s[c][2 * e], scale2, m2);
          const float lo = fast_exp2(lo_of(x)), hi = fast_exp2(hi_of(x));
          if (e & 1) l1 = add2(l1, pack2(lo, hi));
          else l0 = add2(l0, pack2(lo, hi));
          w16[e] = pack_bf16x2_rn(lo, hi);
        }
        tmem_st16(s_col + 16 * c, w16);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[w]);
    }
    // the output: zeros for a row that sees no key
    if (ok && nt[w] > 0) ok = __all_sync(~0u, mbar_wait_ready(&o_full[w], 0, a.dev_status));
    if (ok) {
      tc_fence_after();
      const uint64_t ls = add2(l0, l1);
      const float inv = seen > 0 ? 1.f / (lo_of(ls) + hi_of(ls)) : 0.f;
      // The rows go through the warp's part of the queries' memory (their last product is done), so
      // that half a warp stores a whole row: stored by the thread that holds it, in pieces of 16
      // bytes, a row took five times as long.  A row's 16-byte pieces are rotated by its number.
      uint8_t* stage = smem + (uint32_t)(w * kAtoms) * kAtom + (uint32_t)quad * 32 * 256;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t v[32];
        if (nt[w] > 0) {
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
          *reinterpret_cast<uint4*>(stage + lane * 256 + ((((c + e) >> 3) ^ (lane & 15)) << 4)) = x;
        }
      }
      __syncwarp();
      const int row0 = row - lane, piece = lane & 15;
      uint16_t* out = a.out + ((size_t)(q0 + row0) * a.Hq + h) * 128 + piece * 8;
#pragma unroll
      for (int r = lane >> 4; r < 32; r += 2) {
        const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 256 + ((piece ^ (r & 15)) << 4));
        if (row0 + r < nq) *reinterpret_cast<uint4*>(out + (size_t)r * a.Hq * 128) = x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

namespace {

cudaError_t launch_two_tiles(const PrefillArgs& a, cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.qtiles = (int)((a.max_q + 2LL * kRows - 1) / (2 * kRows));
  p.scale2 = (a.scale < 0 ? -a.scale : a.scale) * 1.4426950408889634f;
  if (p.scale2 < 1e-30f) p.scale2 = 1e-30f;  // above 0, so that a masked score stays -inf
  p.negate = a.scale < 0;
#ifdef STIEF_TEST_HOOKS
  p.stall = test_stall_bytes();
#endif
  const long long blocks = (long long)p.qtiles * a.Hq * a.B;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const uint64_t rows = a.Nkv > 0 ? a.Nkv : 1;  // (no keys: the maps are never used)
  const void* k = a.Nkv > 0 ? a.k : a.q;
  const void* v = a.Nkv > 0 ? a.v : a.q;
  const void* pe = a.Nkv > 0 ? a.pe : a.q;
  const uint64_t dq = (uint64_t)a.Hq * (128 + a.dr), dk = (uint64_t)a.Hkv * 128, dp = a.dr;
  if (!encode_tiled_bf16_2d(&p.mq, a.q, dq, (uint64_t)a.Nq, dq * 2, 64, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_bf16_3d(&p.mk, k, {64, rows, dk / 64}, {dk * 2, 128}, {64, kRows, 2}) ||
      !encode_tiled_bf16_3d(&p.mv, v, {64, rows, dk / 64}, {dk * 2, 128}, {64, kRows / 2, 2}) ||
      !encode_tiled_bf16_2d(&p.mp, pe, dp, rows, dp * 2, 64, kRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(stief_prefill_kernel), a.device, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(384);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, stief_prefill_kernel, p);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  // Query heads that share a KV head go into the rows of one tile (8 prompts of 65 to 1500 queries,
  // 32 heads over 8: 84.9 us against 109.5 with a head a tile and steps of 128 keys).
  const int group = a.Hq / a.Hkv, pack = group <= kRows && (group & (group - 1)) == 0 ? group : 1;
  // With a position part one tile of queries a CTA is for prompts that do not fill more than one:
  // 8 chunks of 128 over 4128 keys, 32 heads, 116 us against 150; but 8 of 256, 229 against 182.  And
  // then only if there are more CTAs than SMs or few keys: 1 chunk of 128 over 8128 keys, 128 heads,
  // 182 us against 132; 5 prompts of up to 64, 6.0 against 7.9.
  const bool small = (long long)a.max_q * pack <= kRows &&
                     ((long long)a.B * (a.Hq / pack) > a.sms || a.Nkv <= 512LL * a.B);
  return a.dr == 0 || small ? launch_prefill_one_tile(a, pack, stream) : launch_two_tiles(a, stream);
}

}  // namespace stief
