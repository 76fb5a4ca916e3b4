// The decoding of packed codes into fp16 tiles for tcgen05, and the parts of the
// shared prefix for d = 256, for batches with many query rows per KV head.
//
// A block takes 128 query rows (of all sequences) of one head and a range of
// the prefix's tokens, TN at a time:
//   S[row][token]  = Q (sigma c)^T            both operands in shared memory;
//   P[row][token]  = 2^7 e^{x - ref}, fp16, written over S in tensor memory;
//   O[row][coord] += P (sigma c)              P from tensor memory.
// Warps 4-7 turn packed codes into swizzled fp16 tiles (sigma c, rounded once:
// kLargeScale), warp 8 issues the products, warps 0-3 hold a query row per thread:
// its maximum and sum need no exchange. Two score buffers let the tensor cores
// form the next scores while the exponentials of these are taken. O is rescaled
// only when a row's maximum grows by more than 2^8 over the reference its weights
// use (the weights then stay below 2^15 in fp16; the final quotient does not see
// the reference).
//
// The query row is scaled by a power of two to [2^13, 2^14) and rounded to
// fp16. For fp16 outputs (EXACT) that is not enough: queries, keys and weights
// are each split into an fp16 value and its rest, and the scores take the three
// products that matter, the values the two of the weights; the remaining
// rounding is that of the values, half a step of fp16, like the output's own.
// For bf16 outputs, with steps 8 times as wide, one product each is enough.
//
// One such unit fills an SM at d = 256: the queries (64 KB, 128 KB with their
// rests) and two stages of keys and values leave no shared memory, O and two
// score buffers no tensor memory for a second. For d = 64 and 128, where two
// units fit, prefix_pair.cuh puts them into one block that decodes each tile
// once for both.
//
// What bounds it: per 128 rows and 64 tokens the two products take 1024 clocks
// of the tensor cores and the exponentials 512 of the special function units;
// the decoding, by four warps, is next to them and not hidden behind another
// unit's products: 28672 tokens, 4 heads, up to 128 rows 69 us a call with bf16
// outputs, 104 with fp16 (twice the products, and 32 tokens at a time).
#pragma once

#include "paged_attention.cuh"
#include "tc.cuh"

namespace srftq {

constexpr int kMmaRows = 128;

template <int BITS, int G, bool EXACT>
struct PrefixMma {
  static constexpr int D = 256;
  static constexpr int TN = EXACT ? 32 : 64;                  // tokens per step
  static constexpr int CB = D * BITS / 8, NG = D / G;
  static constexpr int kPieces = D / 64;                      // 128-byte columns of a row
  static constexpr int kQPiece = kMmaRows * 128, kQ = kPieces * kQPiece;
  static constexpr int kTPiece = TN * 128, kT = kPieces * kTPiece;   // a K or V tile
  static constexpr int kKT = kT * (EXACT ? 2 : 1);            // keys (and their rests)
  static constexpr int kStages = 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQ * (EXACT ? 2 : 1);
  static constexpr int kVOff = kKOff + kStages * kKT;
  static constexpr int kOnOff = kVOff + kStages * kT;         // uint8 [4 steps][TN]: tokens there
  static constexpr int kBarOff = kOnOff + 4 * TN;
  static constexpr int kBytes = kBarOff + 8 * 20 + 16;
  static constexpr int kSmem = kBytes + 1024;                 // slack to start on 1024 bytes
  static constexpr int kThreads = 288;
  static constexpr int kSCols = TN;                           // a score buffer
  static constexpr int kOCol = 2 * TN;
  static constexpr int kTmemCols = 512;                       // a power of two >= kOCol + D
  static constexpr uint32_t kIdescS = f16_idesc<128, TN>();
  static constexpr uint32_t kIdescO = f16_idesc<128, D>() | (1u << 16);   // B is MN-major
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Position p of 8 consecutive coordinates in the decoded order: the code pairs
// that one AND isolates. int4: (0, 4), (1, 5), (2, 6), (3, 7); int8, two words of
// 4: (0, 2), (1, 3) each.
template <int BITS>
__host__ __device__ constexpr int decoded_coord(int p) {
  return BITS == 4 ? (p & 1) * 4 + (p >> 1) : (p & 4) + 2 * (p & 1) + ((p >> 1) & 1);
}

// 8 codes (1 or 2 words) to sigma c in decoded order: v rounded to fp16, rest what
// that left (exact: a product has 18 bits at most). h_lo, h_hi: the magic numbers
// 1024 + u and 1024 + 16 u (int8: 1024 + u) in registers.
template <int BITS, bool REST>
__device__ __forceinline__ void decode_chunk(const uint32_t* w, uint32_t sg2, uint32_t h_lo,
                                             uint32_t h_hi, uint4& v, uint4& rest) {
  constexpr uint32_t k1 = 0x3C003C00u, k16 = 0x2C002C00u;                       // 1, 2^-4
  constexpr uint32_t o8 = 0xE408E408u, o72 = 0xD480D480u, o128 = 0xE480E480u;   // -1032, -72, -1152
  uint32_t c[4];
  if constexpr (BITS == 4) {
    const uint32_t y = w[0] >> 8;
    c[0] = hfma2((w[0] & 0x000F000Fu) ^ h_lo, k1, o8);
    c[1] = hfma2((w[0] & 0x00F000F0u) ^ h_hi, k16, o72);
    c[2] = hfma2((y & 0x000F000Fu) ^ h_lo, k1, o8);
    c[3] = hfma2((y & 0x00F000F0u) ^ h_hi, k16, o72);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[2 * i] = hfma2((w[i] & 0x00FF00FFu) ^ h_hi, k1, o128);
      c[2 * i + 1] = hfma2(((w[i] >> 8) & 0x00FF00FFu) ^ h_hi, k1, o128);
    }
  }
  v = make_uint4(hmul2(c[0], sg2), hmul2(c[1], sg2), hmul2(c[2], sg2), hmul2(c[3], sg2));
  if constexpr (REST) {
    rest = make_uint4(hfma2(c[0], sg2, v.x ^ 0x80008000u), hfma2(c[1], sg2, v.y ^ 0x80008000u),
                      hfma2(c[2], sg2, v.z ^ 0x80008000u), hfma2(c[3], sg2, v.w ^ 0x80008000u));
  }
}

// A thread's NK pieces (16 bytes of codes, piece pc of rows tr, tr + RPP, ...) as
// fp16 into a tile at `base` (rest_at > 0: their rests that far behind it). Chunks
// of one row in different 128-byte columns share banks, so the threads of a store
// start at different chunks (order j ^ rot).
template <int D, int BITS, int G, int TN, bool REST, int NK>
__device__ __forceinline__ void decode_pieces(uint32_t base, uint32_t rest_at, int pc, int tr,
                                              const uint4 (&w)[NK], const uint32_t (&s)[NK],
                                              uint32_t h_lo, uint32_t h_hi) {
  constexpr int PPT = D * BITS / 128, RPP = 128 / PPT, NC = 16 / BITS;
  constexpr bool TWO = 128 / BITS > G;   // two scales to a piece
  const int rot = BITS == 4 ? (PPT == 4 ? (pc >> 1) * 2 : PPT == 8 ? pc >> 1 : 0)
                            : (PPT >= 8 ? (pc >> 2) & 1 : 0);
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const int tok = tr + k * RPP;
    uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    uint32_t s0 = (TWO ? s[k] & 0xFFFFu : s[k]) * 0x10001u;
    uint32_t s1 = TWO ? (s[k] >> 16) * 0x10001u : s0;
    if (BITS == 8 ? rot & 1 : rot & 2) {
      const uint32_t y0 = x[0], y1 = x[1], z = s0;
      x[0] = x[2];
      x[1] = x[3];
      x[2] = y0;
      x[3] = y1;
      s0 = s1;
      s1 = z;
    }
    if (BITS == 4 && (rot & 1)) {
      const uint32_t y0 = x[0], y2 = x[2];
      x[0] = x[1];
      x[1] = y0;
      x[2] = x[3];
      x[3] = y2;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = pc * NC + (j ^ rot);
      const uint32_t at = base + (c >> 3) * (TN * 128) + tok * 128 + (((c & 7) ^ (tok & 7)) << 4);
      uint4 v, r;
      decode_chunk<BITS, REST>(x + j * 4 / NC, 2 * j < NC ? s0 : s1, h_lo, h_hi, v, r);
      sts128(at, v);
      if constexpr (REST) sts128(at + rest_at, r);
    }
  }
}

// Large scales (kLargeScale) may belong to tokens behind the end of some rows, whose
// weights there are 0 and would still make NaN of them. So they enter the products as
// 0, and the first token that has one goes to shared memory; the rows that reach it
// take NaN for their sum at the end (each attends to all tokens below its length, so
// the first is enough), and the join does them anew.
template <int BITS, int NK, class Tok>
__device__ __forceinline__ void drop_large(uint32_t (&s)[NK], int* first_bad, Tok token) {
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < NK; ++k) any |= large_halves<BITS>(s[k]);
  if (any) {
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const uint32_t bad = large_halves<BITS>(s[k]);
      if (bad) {
        s[k] &= ~((bad >> 15) * 0xFFFFu);
        atomicMin(first_bad, token(k));
      }
    }
  }
}

template <int BITS, int G, bool EXACT>
__global__ void __launch_bounds__(PrefixMma<BITS, G, EXACT>::kThreads, 1)
    prefix_mma_kernel(const PrefixArgs a) {
  using L = PrefixMma<BITS, G, EXACT>;
  constexpr int D = L::D, TN = L::TN, CB = L::CB, NG = L::NG;   // tokens per step, code bytes, scales
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_a = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((0u - raw_a) & 1023u);
  const uint32_t sm = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6;
  uint64_t *sfull = bars + 8, *pfull = bars + 10, *odone = bars + 12, *drain = bars + 13;   // drain: all products done
  uint64_t* qfull = bars + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);
  int* first_bad = reinterpret_cast<int*>(bars + 16) + 1;
  volatile uint8_t* on_sh = smem + L::kOnOff;

  // this block's head, rows and tokens
  const int g = a.q_per_kv, hq = a.heads * g, M = a.n_seq * g;
  const int tiles = (M + kMmaRows - 1) / kMmaRows;
  const int rt = int(blockIdx.x) % tiles, sh = int(blockIdx.x) / tiles;
  const int h = sh % a.heads, part_i = sh / a.heads;
  const int r0 = rt * kMmaRows;
  const int t0 = part_i * a.prefix_per, t1 = range_end(t0, a.prefix_per, a.prefix_len);
  const int n = (t1 - t0 + TN - 1) / TN;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 4);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 4);
      mbar_init(&vempty[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
    }
    mbar_init(odone, 1);
    mbar_init(drain, 1);
    mbar_init(qfull, 1);
    *abort_flag = 0;
    *first_bad = INT_MAX;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  grid_dependency_wait();   // the query tiles
  const uint32_t tmem = *tmem_slot;
  const int64_t tile = int64_t(h) * tiles + rt;

  if (warp == 8) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t kQBytes = L::kQ * (EXACT ? 2 : 1);
      mbar_arrive_expect_tx(qfull, kQBytes);
      bulk_load(smem + L::kQOff, a.q_image + tile * kQBytes, kQBytes, qfull);
      bool ok = wait_or_abort(qfull, 0, abort_flag, a.guard);
      auto values = [&](int i) {   // O += P(i) V(i)
        const int st = i & 1;
        if (!wait_or_abort(&vfull[st], (i >> 1) & 1, abort_flag, a.guard) ||
            !wait_or_abort(&pfull[st], (i >> 1) & 1, abort_flag, a.guard))
          return false;
        tc_fence_after();
        const uint32_t vb = sm + L::kVOff + st * L::kT, pt = tmem + st * L::kSCols;
#pragma unroll
        for (int ks = 0; ks < TN / 16; ++ks) {
          const uint64_t bd = sw128_mn_desc(vb + 2048u * ks, L::kTPiece);
          tc_mma_f16_ts(tmem + L::kOCol, pt + 8 * ks, bd, L::kIdescO, (i | ks) != 0 ? 1u : 0u);
          if constexpr (EXACT)
            tc_mma_f16_ts(tmem + L::kOCol, pt + TN / 2 + 8 * ks, bd, L::kIdescO, 1u);
        }
        tc_commit(&vempty[st]);
        tc_commit(odone);
        return true;
      };
      for (int i = 0; i < n && ok; ++i) {
        const int st = i & 1;
        if (!wait_or_abort(&kfull[st], (i >> 1) & 1, abort_flag, a.guard)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t qa = sm + L::kQOff, kb = sm + L::kKOff + st * L::kKT;
        const uint32_t dt = tmem + st * L::kSCols;
#pragma unroll
        for (int pc = 0; pc < L::kPieces; ++pc)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t qd = sw128_desc(qa + pc * L::kQPiece + 32u * ks);
            const uint64_t kd = sw128_desc(kb + pc * L::kTPiece + 32u * ks);
            tc_mma_f16(dt, qd, kd, L::kIdescS, (pc | ks) != 0 ? 1u : 0u);
            if constexpr (EXACT) {
              tc_mma_f16(dt, sw128_desc(qa + L::kQ + pc * L::kQPiece + 32u * ks), kd, L::kIdescS, 1u);
              tc_mma_f16(dt, qd, sw128_desc(kb + L::kT + pc * L::kTPiece + 32u * ks), L::kIdescS, 1u);
            }
          }
        tc_commit(&kempty[st]);
        tc_commit(&sfull[st]);
        if (i > 0) ok = values(i - 1);
      }
      if (ok && n > 0) (void)values(n - 1);
      tc_commit(drain);   // every product is done before tensor memory is freed
      (void)mbar_wait_bounded(drain, 0);
    }
  } else if (warp >= 4) {
    // ---------------- codes to fp16 tiles ----------------
    // Neighbouring threads take the 16-byte pieces of one row, so a load of a
    // warp touches few lines; piece -> 16-byte chunks of 8 decoded coordinates.
    constexpr int PPT = CB / 16, RPP = 128 / PPT;        // pieces of a row, rows per pass
    constexpr int NK = TN / RPP;                         // pieces of a thread
    constexpr int CC = 128 / BITS;                       // coordinates of a piece
    constexpr int GC = CC > G ? CC / G : 1;              // its scales (1 or 2)
    static_assert(TN % RPP == 0 && GC <= 2, "pieces");
    const int dt = tid - 128;
    const int pc = dt % PPT, tr = dt / PPT;
    const uint32_t h_lo = in_register(0x64086408u, a.zero);
    const uint32_t h_hi = in_register(0x64806480u, a.zero);
    uint4 kw[NK], vw[NK];
    uint32_t ks[NK], vs[NK];
    int32_t page[NK], row[NK], next[NK];   // table entry two steps on; rows of this step, the next
    auto token = [&](int i, int k) { return t0 + i * TN + tr + k * RPP; };
    auto look_up = [&](int i, int k) {
      const int t = token(i, k);
      return i < n && t < t1 && a.dbg_token(true, t)
                 ? __ldg(a.prefix_table + a.map.page.div(uint32_t(t)))
                 : -1;
    };
    auto row_at = [&](int i, int k, int32_t p) {
      const uint32_t t = uint32_t(token(i, k));
      return uint32_t(p) < uint32_t(a.map.n_pages)
                 ? int32_t(uint32_t(p) * a.map.page.d + (t - a.map.page.div(t) * a.map.page.d))
                 : -1;
    };
    auto load = [&](const int32_t (&r)[NK], const uint8_t* codes, const uint16_t* scales,
                    uint4 (&w)[NK], uint32_t (&s)[NK]) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int64_t vec = int64_t(r[k] < 0 ? 0 : r[k]) * a.heads + h;
        const uint16_t* sp = scales + vec * NG + pc * CC / G;
        w[k] = make_uint4(0, 0, 0, 0);
        s[k] = 0;
        if (r[k] >= 0 && a.dbg_row(r[k])) {
          w[k] = __ldg(reinterpret_cast<const uint4*>(codes + vec * CB) + pc);
          s[k] = GC == 2 ? __ldg(reinterpret_cast<const uint32_t*>(sp)) : uint32_t(__ldg(sp));
        }
      }
    };
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      row[k] = row_at(0, k, look_up(0, k));
      next[k] = row_at(1, k, look_up(1, k));
    }
    load(row, a.k_codes, a.k_scales, kw, ks);
    load(row, a.v_codes, a.v_scales, vw, vs);
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
#pragma unroll
      for (int k = 0; k < NK; ++k) page[k] = look_up(i + 2, k);
      if (i >= 2 && !__all_sync(0xffffffffu, wait_or_abort(&kempty[st], ((i >> 1) & 1) ^ 1,
                                                           abort_flag, a.guard)))
        break;
      // which tokens are there: bytes, written again four steps on, after the
      // scores of step i + 2, which follow the weights of this step
      if (pc == 0) {
#pragma unroll
        for (int k = 0; k < NK; ++k) on_sh[(i & 3) * TN + tr + k * RPP] = row[k] >= 0 ? 1 : 0;
      }
      drop_large<BITS>(ks, first_bad, [&](int k) { return token(i, k); });
      decode_pieces<D, BITS, G, TN, EXACT, NK>(sm + L::kKOff + st * L::kKT, L::kT, pc, tr, kw, ks, h_lo,
                                           h_hi);
      __threadfence_block();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[st]);
      load(next, a.k_codes, a.k_scales, kw, ks);
      if (i >= 2 && !__all_sync(0xffffffffu, wait_or_abort(&vempty[st], ((i >> 1) & 1) ^ 1,
                                                           abort_flag, a.guard)))
        break;
      drop_large<BITS>(vs, first_bad, [&](int k) { return token(i, k); });
      decode_pieces<D, BITS, G, TN, false, NK>(sm + L::kVOff + st * L::kT, 0, pc, tr, vw, vs, h_lo,
                                           h_hi);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&vfull[st]);
      load(next, a.v_codes, a.v_scales, vw, vs);
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        row[k] = next[k];
        next[k] = row_at(i + 2, k, page[k]);
      }
    }
  } else {
    // ---------------- softmax: a query row per thread ----------------
    const int r = tid;                       // row of the tile, lane of tensor memory
    const int rr = min(r0 + r, M - 1);
    const int lim = a.len(rr / g);
    const float f = a.q_factor[tile * kMmaRows + r];
    const uint32_t tl = tmem + (uint32_t(warp) << 21);   // lanes 32 warp ..
    float ref = -INFINITY, l = 0.0f;         // the reference of the weights, their sum
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      if (!__all_sync(0xffffffffu,
                      wait_or_abort(&sfull[st], (i >> 1) & 1, abort_flag, a.guard))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[TN / 32][32];
#pragma unroll
      for (int k = 0; k < TN / 32; ++k) tmem_ld32(tl + st * L::kSCols + 32 * k, s[k]);
      if constexpr (TN == 64) tmem_wait_ld(s[0], s[TN / 32 - 1]);
      else tmem_wait_ld1(s[0]);
      const int tk = t0 + i * TN;
      // bit j of on[k]: token 32 k + j of the step is there
      uint32_t on[TN / 32];
      const bool past = lim <= tk;   // the row ends before: its weights are 0 below
      bool all = past || tk + TN <= lim;
#pragma unroll
      for (int k = 0; k < TN / 32; ++k) {
        on[k] = __ballot_sync(0xffffffffu, on_sh[(i & 3) * TN + 32 * k + lane] != 0);
        all = all && on[k] == 0xffffffffu;
      }
      if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
        for (int k = 0; k < TN / 32; ++k)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((on[k] >> j) & 1u) || tk + 32 * k + j >= lim) s[k][j] = 0xff800000u;
      }
      float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int k = 0; k < TN / 32; ++k)
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          mx = max3(mx, __uint_as_float(s[k][j]), __uint_as_float(s[k][j + 1]));
          mx1 = max3(mx1, __uint_as_float(s[k][j + 2]), __uint_as_float(s[k][j + 3]));
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
      uint32_t ph[32];
      uint32_t pl[EXACT ? 32 : 1];
#pragma unroll
      for (int k = 0; k < TN / 32; ++k)
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(s[k][j]), __uint_as_float(s[k][j + 1])),
              make_float2(f, f), make_float2(b, b));
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          if (j & 2) sum1 = __fadd2_rn(sum1, p);
          else sum = __fadd2_rn(sum, p);
          const uint32_t hh = pack_half2(p.x, p.y);
          ph[16 * k + j / 2] = hh;
          if constexpr (EXACT) pl[16 * k + j / 2] = half2_rest(p.x, p.y, hh);
        }
      l += (sum.x + sum.y) + (sum1.x + sum1.y);
      if constexpr (TN == 64) {
        tmem_st32(tl + st * L::kSCols, ph);
        if constexpr (EXACT) tmem_st32(tl + st * L::kSCols + 32, pl);
      } else {   // TN = 32: 16 columns each
        if constexpr (EXACT) {
#pragma unroll
          for (int j = 0; j < 16; ++j) ph[16 + j] = pl[j];
        }
        tmem_st32(tl + st * L::kSCols, ph);
      }
      // O follows the reference (it is complete up to step i - 1 by then)
      if (i > 0 && __any_sync(0xffffffffu, grow)) {
        if (!__all_sync(0xffffffffu, wait_or_abort(odone, (i - 1) & 1, abort_flag, a.guard))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t o[32];
          tmem_ld32(tl + L::kOCol + k, o);
          tmem_wait_ld1(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * cc);
          tmem_st32(tl + L::kOCol + k, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[st]);
    }
    // The end has a barrier of its own: two phases of odone may pass between a
    // warp's looks at it here, and a parity cannot tell them apart.
    if (ok && __all_sync(0xffffffffu, wait_or_abort(drain, 0, abort_flag, a.guard))) {
      tc_fence_after();
      // the decoders' last arrival, for what they have found
      if (n > 0) (void)wait_or_abort(&vfull[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, a.guard);
      if (lim > *first_bad) l = NAN;
      const int64_t part = (int64_t(part_i) * a.heads + h) * M + r0 + r;
      const bool live = r0 + r < M && a.dbg_part(true, part);
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        tmem_ld32(tl + L::kOCol + k, o);
        tmem_wait_ld1(o);
        if (live) {
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            y[(j & ~7) + decoded_coord<BITS>(j & 7)] = __uint_as_float(o[j]) * 0x1p-7f;
          float4* dst = reinterpret_cast<float4*>(a.pre_acc + part * D + k);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
      }
      if (live) a.pre_ml[part] = make_float2(ref, l * 0x1p-7f);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, L::kTmemCols);
}

}  // namespace srftq
