// Parts of the shared prefix on the 5th-generation tensor cores (tcgen05) for
// d = 64 and 128: two units of 128 query rows on each SM.
//
// A unit is 128 query rows with two score tiles S, the weights P written over
// them, and an accumulator O, all in tensor memory:
//   S[row][token]  = Q (sigma c)^T            TN = 64 tokens at a time;
//   P[row][token]  = 2^7 e^{x - ref}, fp16, written over S;
//   O[row][coord] += P (sigma c).
// The scores of a unit's next tile are formed while its four warps take the
// exponentials of this one. Two forms:
//   shared   the units are 256 different rows over the same tokens: a token's
//            codes are decoded once for both (bf16 outputs, more than 128 rows);
//   split    the units are the same rows over alternate tiles, two parts of the
//            softmax (up to 128 rows, and fp16 outputs).
//
// Warps 0-3 and 4-7: softmax of unit 0 and 1, a query row per thread. Warps
// 8-11 and 12-15: codes of keys and of values to fp16 tiles (swizzled, sigma c
// rounded once: kLargeScale). Warps 16 and 17:
// issue the units' products. Warps 18 and 19: copy codes and scales of a tile
// each in turn into a ring of raw stages, so that memory latency is hidden by
// depth, not by registers. O is rescaled only when a row's maximum grows by more
// than 2^8 over the reference its weights use (the weights stay below 2^15; the
// final quotient does not see the reference).
//
// The query row is scaled by a power of two to [2^13, 2^14) and rounded to
// fp16. For fp16 outputs (EXACT) queries, keys and weights are split into an
// fp16 value and its rest; the scores take the three products that matter, the
// values the two of the weights. What remains is the rounding of the values, half
// a step of fp16, like the output's own. For bf16 outputs, with steps 8 times as
// wide, one product each is enough.
//
// What bounds it: 128 rows x 64 tokens are 512 clocks of the special function
// units and, at d = 128, 512 of the tensor cores; two units could keep both busy.
// What it reaches is the chain of a tile: decode, scores, exponentials, values,
// each handed on through a barrier. 128 sequences x 8 queries x 8 heads of d = 128
// over 32768 int4 tokens, bf16: 168 us, against 80 of the products at the measured
// dense rate. 16 x 8 x 8 over 131072 int8 tokens: 141 us the whole call, 39 of
// products, 47 of memory; without the decoding of the two int8 tiles it took 43
// less. On a small case ncu shows 28 % of the tensor pipe, 29 % of the special
// function units and 36 % of the issue slots.
#pragma once

#include "prefix_mma.cuh"

namespace srftq {

template <int D, int BITS, int G, bool EXACT, bool SHARED>
struct PrefixPair {
  static_assert(!(EXACT && SHARED), "fp16 outputs take the split form");
  static constexpr int TN = 64;
  static constexpr int CB = D * BITS / 8, NG = D / G, SB = 2 * NG;
  static constexpr int kPieces = D / 64;
  static constexpr int kTPiece = TN * 128, kT = kPieces * kTPiece;
  static constexpr int kKT = kT * (EXACT ? 2 : 1);
  static constexpr int kQTile = kPieces * kMmaRows * 128 * (EXACT ? 2 : 1);
  static constexpr int kQ = kQTile * (SHARED ? 2 : 1);
  static constexpr int kSlots = EXACT ? 2 : BITS == 8 ? (SHARED ? 2 : 3) : SHARED ? 3 : 4;
  static constexpr int kSlot = kKT + kT;                            // a decoded tile
  // a raw stage: rows of K, rows of V, scale rows of K, of V (4 bytes at least)
  static constexpr int SBS = SB < 4 ? 4 : SB;
  static constexpr int kRawV = TN * CB, kRawKS = 2 * TN * CB, kRawVS = kRawKS + TN * SBS;
  static constexpr int kRawStage = kRawVS + TN * SBS;
  static constexpr int kRaws = BITS == 4 ? 6 : EXACT ? 3 : 4;
  static constexpr int kSlotOff = kQ;
  static constexpr int kRawOff = kSlotOff + kSlots * kSlot;
  static constexpr int kOnOff = kRawOff + kRaws * kRawStage;        // uint32 [raws][2], [16][2]
  static constexpr int kBarOff = kOnOff + 8 * (kRaws + 16);
  static constexpr int kBars = 2 * kRaws + 4 * kSlots + 13;
  static constexpr int kBytes = kBarOff + 8 * kBars + 16;
  static constexpr int kSmem = kBytes + 1024;                       // slack to start on 1024 bytes
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr int kThreads = 640;
  static constexpr int kQPiece = kMmaRows * 128;                    // a piece of a query tile
  // tensor memory columns: score tiles (two of each unit), accumulators
  static constexpr int kSCol = 0, kOCol = 256;
  static constexpr uint32_t kIdescS = f16_idesc<128, TN>();
  static constexpr uint32_t kIdescO = f16_idesc<128, D>() | (1u << 16);   // B is MN-major
};

// Arrives on `bar` when this thread's cp.async copies so far have landed (the
// arrival is one of the barrier's count).
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

template <int D, int BITS, int G, bool EXACT, bool SHARED>
__global__ void __launch_bounds__(640, 1) prefix_pair_kernel(const PrefixArgs a) {
  using L = PrefixPair<D, BITS, G, EXACT, SHARED>;
  constexpr int TN = L::TN, CB = L::CB, NG = L::NG, NS = L::kSlots, NR = L::kRaws;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_a = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((0u - raw_a) & 1023u);
  const uint32_t sm = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the same in the warp's lanes
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t *rfull = bars, *rempty = rfull + NR, *kfull = rempty + NR, *kempty = kfull + NS;
  uint64_t *vfull = kempty + NS, *vempty = vfull + NS;
  // scores and weights by unit and tile (2 u + buffer), values by unit
  uint64_t *sfull = vempty + NS, *pfull = sfull + 4, *odone = pfull + 4, *qfull = odone + 2;
  uint64_t* all_done = qfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(all_done + 2);
  int* first_bad = reinterpret_cast<int*>(all_done + 2) + 1;
  volatile uint32_t* on_raw = reinterpret_cast<volatile uint32_t*>(smem + L::kOnOff);
  volatile uint32_t* on_ring = on_raw + 2 * NR;   // by tile, 16 of them

  // this block's head, rows and tokens
  constexpr int ROWS = SHARED ? 2 * kMmaRows : kMmaRows;
  const int g = a.q_per_kv, M = a.n_seq * g;
  const int blocks = (M + ROWS - 1) / ROWS, tiles = (M + kMmaRows - 1) / kMmaRows;
  const int rt = int(blockIdx.x) % blocks, sh = int(blockIdx.x) / blocks;
  const int h = sh % a.heads, part_i = sh / a.heads;
  const int t0 = part_i * a.prefix_per, t1 = range_end(t0, a.prefix_per, a.prefix_len);
  const int n = (t1 - t0 + TN - 1) / TN;                           // tiles of 64 tokens
  // units with rows: both, or (shared, an odd last tile of rows) the first
  const int units = SHARED && 2 * rt + 1 >= tiles ? 1 : 2;

  if (tid == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&rfull[i], 33);
      mbar_init(&rempty[i], 8);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kfull[i], 4);
      mbar_init(&kempty[i], SHARED ? units : 1);   // an arrival of each unit that reads it
      mbar_init(&vfull[i], 4);
      mbar_init(&vempty[i], SHARED ? units : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
    }
    for (int u = 0; u < 2; ++u) mbar_init(&odone[u], 1);
    for (int u = 0; u < 2; ++u) mbar_init(&qfull[u], 1);
    mbar_init(all_done, 2);
    *abort_flag = 0;
    *first_bad = INT_MAX;
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  grid_dependency_wait();   // the query tiles
  const uint32_t tmem = *tmem_slot;

  if (warp == 16 || warp == 17) {
    // ---------------- MMA issuers, one for each unit ----------------
    // The whole warp runs this and every operand is the same in its lanes, so
    // addresses and descriptors stay in uniform registers; one elected lane
    // issues. (From a branch of one lane each product waits for its operands to
    // be moved there: 131072 int8 tokens for 128 rows took 239 instead of 157 us.)
    {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok =
            __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, a.guard));
        tc_fence_after();
        return ok;
      };
      // S of unit u = Q K^T of the tile in slot sl, the unit's m-th
      const uint64_t q0 = sw128_desc(sm);
      auto scores = [&](int u, int sl, int m) {
        const uint32_t dt = tm + L::kSCol + 128 * u + 64 * (m & 1);
        const uint64_t qd = q0 + (SHARED ? u * (L::kQTile >> 4) : 0);
        const uint64_t k0 = sw128_desc(sm + L::kSlotOff + sl * L::kSlot);
#pragma unroll
        for (int pc = 0; pc < L::kPieces; ++pc)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t qk = qd + ((pc * L::kQPiece + 32 * ks) >> 4);
            const uint64_t kd = k0 + ((pc * L::kTPiece + 32 * ks) >> 4);
            tc_mma_f16_elect(dt, qk, kd, L::kIdescS, (pc | ks) != 0 ? 1u : 0u);
            if constexpr (EXACT) {
              tc_mma_f16_elect(dt, qk + (L::kPieces * L::kQPiece >> 4), kd, L::kIdescS, 1u);
              tc_mma_f16_elect(dt, qk, kd + (L::kT >> 4), L::kIdescS, 1u);
            }
          }
        tc_commit_elect(&sfull[2 * u + (m & 1)]);
      };
      // O of unit u += P V of the tile in slot sl, the unit's m-th
      auto values = [&](int u, int sl, int m) {
        const uint32_t pt = tm + L::kSCol + 128 * u + 64 * (m & 1), ot = tm + L::kOCol + 128 * u;
        const uint64_t v0 =
            sw128_mn_desc(sm + L::kSlotOff + sl * L::kSlot + L::kKT, L::kTPiece);
#pragma unroll
        for (int ks = 0; ks < TN / 16; ++ks) {
          const uint64_t bd = v0 + ((2048 * ks) >> 4);
          tc_mma_f16_ts_elect(ot, pt + 8 * ks, bd, L::kIdescO, (m | ks) != 0 ? 1u : 0u);
          if constexpr (EXACT)
            tc_mma_f16_ts_elect(ot, pt + TN / 2 + 8 * ks, bd, L::kIdescO, 1u);
        }
        tc_commit_elect(&odone[u]);
      };
      const int u = warp - 16;
      const int n_mine = u < units ? (SHARED ? n : (n + 1 - u) / 2) : 0;
      uint64_t* my_q = &qfull[SHARED ? u : 0];
      if (lane == 0 && (SHARED ? u < units : u == 0)) {
        const int64_t tile = int64_t(h) * tiles + (SHARED ? 2 * rt + u : rt);
        mbar_arrive_expect_tx(my_q, L::kQTile);
        bulk_load(smem + (SHARED ? u * L::kQTile : 0), a.q_image + tile * L::kQTile, L::kQTile, my_q);
      }
      __syncwarp();
      bool ok = n_mine == 0 || wait(my_q, 0);
      // the scores run a tile ahead of the values
      for (int m = 0; m <= n_mine && ok; ++m) {
        if (m < n_mine) {
          const int j = SHARED ? m : 2 * m + u, sl = j % NS;
          ok = wait(&kfull[sl], (j / NS) & 1);
          if (!ok) break;
          scores(u, sl, m);
          tc_commit_elect(&kempty[sl]);
        }
        if (m > 0) {
          const int i = m - 1, j = SHARED ? i : 2 * i + u, sl = j % NS;
          ok = wait(&vfull[sl], (j / NS) & 1) && wait(&pfull[2 * u + (i & 1)], (i >> 1) & 1);
          if (!ok) break;
          values(u, sl, i);
          tc_commit_elect(&vempty[sl]);
        }
      }
      tc_commit_elect(all_done);   // every product is done before tensor memory is freed
      (void)mbar_wait_bounded(all_done, 0);
      __syncwarp();
    }
  } else if (warp > 17) {
    // ---------------- loaders: tile j by warp 18 + j % 2 ----------------
    constexpr int PPT = CB / 16, NK = TN * PPT / 32;   // pieces of a row, of a lane
    int32_t page[2];
    auto look_up = [&](int j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = t0 + j * TN + lane + 32 * k;
        page[k] = j < n && t < t1 && a.dbg_token(true, t)
                      ? __ldg(a.prefix_table + a.map.page.div(uint32_t(t)))
                      : -1;
      }
    };
    look_up(warp - 18);
    for (int j = warp - 18; j < n; j += 2) {
      const int st = j % NR;
      int32_t row[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t t = uint32_t(t0 + j * TN + lane + 32 * k);
        row[k] = uint32_t(page[k]) < uint32_t(a.map.n_pages)
                     ? int32_t(uint32_t(page[k]) * a.map.page.d + (t - a.map.page.div(t) * a.map.page.d))
                     : -1;
        if (row[k] >= 0 && !a.dbg_row(row[k])) row[k] = -1;
      }
      look_up(j + 2);
      if (j >= NR && !__all_sync(0xffffffffu, wait_or_abort(&rempty[st], ((j / NR) & 1) ^ 1,
                                                            abort_flag, a.guard)))
        break;
      const uint32_t rb = sm + L::kRawOff + st * L::kRawStage;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int p = lane + 32 * i, tok = p / PPT, pc = p % PPT;
        const int32_t r = __shfl_sync(0xffffffffu, row[(32 * i) / PPT / 32], tok & 31);
        const int64_t at = (int64_t(r < 0 ? 0 : r) * a.heads + h) * CB + pc * 16;
        copy16(rb + p * 16, a.k_codes + at, r >= 0);
        copy16(rb + L::kRawV + p * 16, a.v_codes + at, r >= 0);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t vec = int64_t(row[k] < 0 ? 0 : row[k]) * a.heads + h;
        const uint16_t *ks = a.k_scales + vec * NG, *vs = a.v_scales + vec * NG;
        const uint32_t dk = rb + L::kRawKS + (lane + 32 * k) * L::SBS, dv = dk + TN * L::SBS;
        if constexpr (L::SB >= 16) {
          copy16(dk, ks, row[k] >= 0);
          copy16(dv, vs, row[k] >= 0);
        } else if constexpr (L::SB >= 4) {
          copy_small<L::SB>(dk, ks, row[k] >= 0);
          copy_small<L::SB>(dv, vs, row[k] >= 0);
        } else {   // one scale: 2 bytes, below the smallest asynchronous copy
          const uint32_t x = row[k] >= 0 ? __ldg(ks) : 0u, y = row[k] >= 0 ? __ldg(vs) : 0u;
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(dk), "r"(x) : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(dv), "r"(y) : "memory");
        }
      }
      const uint32_t on0 = __ballot_sync(0xffffffffu, row[0] >= 0);
      const uint32_t on1 = __ballot_sync(0xffffffffu, row[1] >= 0);
      copies_arrive(&rfull[st]);
      __syncwarp();
      if (lane == 0) {
        on_raw[2 * st] = on0;
        on_raw[2 * st + 1] = on1;
        __threadfence_block();
        mbar_arrive(&rfull[st]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 8) {
    // ---------------- codes to fp16 tiles: warps 8-11 keys, 12-15 values ----------------
    // Neighbouring threads take the 16-byte pieces of one row.
    constexpr int PPT = CB / 16, RPP = 128 / PPT;        // pieces of a row, rows per pass
    constexpr int NK = TN / RPP, CC = 128 / BITS;        // pieces of a thread, coordinates of one
    constexpr bool TWO = CC > G;                         // two scales to a piece
    const bool keys = warp < 12;
    const int dt = tid & 127, pc = dt % PPT, tr = dt / PPT;
    const uint32_t h_lo = in_register(0x64086408u, a.zero);
    const uint32_t h_hi = in_register(0x64806480u, a.zero);
    uint64_t *full = keys ? kfull : vfull, *empty = keys ? kempty : vempty;
    const uint32_t codes = sm + L::kRawOff + (keys ? 0 : L::kRawV) + dt * 16;
    const uint32_t scales = sm + L::kRawOff + (keys ? L::kRawKS : L::kRawVS) + tr * L::SBS +
                            pc * CC / G * 2;
    const uint32_t tiles_at = sm + L::kSlotOff + (keys ? 0 : L::kKT);
    for (int j = 0; j < n; ++j) {
      const int st = j % NR, sl = j % NS;
      if (!__all_sync(0xffffffffu,
                      wait_or_abort(&rfull[st], (j / NR) & 1, abort_flag, a.guard)))
        break;
      uint4 w[NK];
      uint32_t s[NK];
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        w[k] = lds128(codes + st * L::kRawStage + 2048 * k);
        const uint32_t sa = scales + st * L::kRawStage + k * RPP * L::SBS;
        if constexpr (TWO) {
          s[k] = lds32(sa);
        } else {
          uint16_t x;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(sa));
          s[k] = x;
        }
      }
      drop_large<BITS>(s, first_bad, [&](int k) { return t0 + j * TN + tr + k * RPP; });
      // an entry of the ring is written again 16 tiles on, long after the
      // softmax of this tile: at most the slots' tiles lie between
      if (tid == 256) {
        on_ring[2 * (j & 15)] = on_raw[2 * st];
        on_ring[2 * (j & 15) + 1] = on_raw[2 * st + 1];
        __threadfence_block();
      }
      if (j >= NS && !__all_sync(0xffffffffu, wait_or_abort(&empty[sl], ((j / NS) & 1) ^ 1,
                                                            abort_flag, a.guard)))
        break;
      if (EXACT && keys)
        decode_pieces<D, BITS, G, TN, EXACT, NK>(tiles_at + sl * L::kSlot, L::kT, pc, tr, w, s, h_lo,
                                                 h_hi);
      else
        decode_pieces<D, BITS, G, TN, false, NK>(tiles_at + sl * L::kSlot, 0, pc, tr, w, s, h_lo,
                                                 h_hi);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[sl]);
        mbar_arrive(&rempty[st]);
      }
    }
  } else {
    // ---------------- softmax: a query row per thread ----------------
    const int u = warp >> 2, r = tid & 127;
    const int tile_i = SHARED ? 2 * rt + u : rt;         // 128-row tile of the head
    const int r0 = tile_i * kMmaRows;
    const int n_mine = SHARED ? n : (n + 1 - u) / 2;     // tiles of this unit
    if (u < units) {
      const uint32_t tl = tmem + (uint32_t(warp & 3) << 21);
      const uint32_t tO = tl + L::kOCol + 128 * u;
      const int64_t tile = int64_t(h) * tiles + tile_i;
      bool ok = true;
      const int rr = min(r0 + r, M - 1);
      const int lim = a.len(rr / g);
      const float f = a.q_factor[tile * kMmaRows + r];
      float ref = -INFINITY, l = 0.0f;       // the reference of the weights, their sum
      for (int m = 0; m < n_mine; ++m) {
        const int j = SHARED ? m : 2 * m + u;
        const uint32_t tS = tl + L::kSCol + 128 * u + 64 * (m & 1);
        if (!__all_sync(0xffffffffu, wait_or_abort(&sfull[2 * u + (m & 1)], (m >> 1) & 1,
                                                   abort_flag, a.guard))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[2][32];
        tmem_ld32(tS, s[0]);
        tmem_ld32(tS + 32, s[1]);
        const int tk = t0 + j * TN;
        const uint32_t on[2] = {on_ring[2 * (j & 15)], on_ring[2 * (j & 15) + 1]};
        tmem_wait_ld(s[0], s[1]);
        // a row that ends before this tile needs no mask: its weights are 0 below
        const bool past = lim <= tk;
        if (!__all_sync(0xffffffffu,
                        (on[0] & on[1]) == 0xffffffffu && (past || tk + TN <= lim))) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((on[k] >> i) & 1u) || tk + 32 * k + i >= lim) s[k][i] = 0xff800000u;
        }
        float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            mx = max3(mx, __uint_as_float(s[k][i]), __uint_as_float(s[k][i + 1]));
            mx1 = max3(mx1, __uint_as_float(s[k][i + 2]), __uint_as_float(s[k][i + 3]));
          }
        mx = past ? -INFINITY : fmaxf(mx, mx1) * f;   // f > 0
        const bool grow = mx > ref + 8.0f || (ref == -INFINITY && mx > -INFINITY);
        const float nref = grow ? mx : ref;
        const float cc = !grow ? 1.0f : ref == -INFINITY ? 0.0f : ex2(ref - nref);
        l *= cc;
        ref = nref;
        // P = 2^7 e^{x - ref} (0 while the row has seen no token)
        const float b = past ? -INFINITY : 7.0f - (ref == -INFINITY ? 0.0f : ref);
        float2 sum = make_float2(0.0f, 0.0f), sum1 = sum;
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // 32 tokens at a time, to free their scores
          uint32_t ph[16], pl[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(s[k][i]), __uint_as_float(s[k][i + 1])),
                make_float2(f, f), make_float2(b, b));
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            if (i & 2) sum1 = __fadd2_rn(sum1, p);
            else sum = __fadd2_rn(sum, p);
            const uint32_t hh = pack_half2(p.x, p.y);
            ph[i / 2] = hh;
            if constexpr (EXACT) pl[i / 2] = half2_rest(p.x, p.y, hh);
          }
          tmem_st16(tS + 16 * k, ph);
          if constexpr (EXACT) tmem_st16(tS + 32 + 16 * k, pl);
        }
        l += (sum.x + sum.y) + (sum1.x + sum1.y);
        // O follows the reference. These scores were issued after the values of
        // tile m - 2, so the phase that tells of tile m - 1 is the next or the last.
        if (m > 0 && __any_sync(0xffffffffu, grow)) {
          if (!__all_sync(0xffffffffu,
                          wait_or_abort(&odone[u], (m - 1) & 1, abort_flag, a.guard))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            tmem_ld32(tO + k, o);
            tmem_wait_ld1(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * cc);
            tmem_st32(tO + k, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * u + (m & 1)]);
      }
      if (ok && __all_sync(0xffffffffu, wait_or_abort(all_done, 0, abort_flag, a.guard))) {
        tc_fence_after();
        // the decoders' last arrivals, for what they have found
        if (n > 0) {
          const int sl = (n - 1) % NS, ph = ((n - 1) / NS) & 1;
          (void)wait_or_abort(&kfull[sl], ph, abort_flag, a.guard);
          (void)wait_or_abort(&vfull[sl], ph, abort_flag, a.guard);
        }
        if (lim > *first_bad) l = NAN;
        const int64_t part = (int64_t(SHARED ? part_i : 2 * part_i + u) * a.heads + h) * M + r0 + r;
        const bool live = r0 + r < M && a.dbg_part(true, part);
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t o[32];
          if (n_mine > 0) {
            tmem_ld32(tO + k, o);
            tmem_wait_ld1(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (live) {
            float y[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              y[(i & ~7) + decoded_coord<BITS>(i & 7)] = __uint_as_float(o[i]) * 0x1p-7f;
            float4* dst = reinterpret_cast<float4*>(a.pre_acc + part * D + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
        if (live) a.pre_ml[part] = make_float2(ref, l * 0x1p-7f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace srftq
