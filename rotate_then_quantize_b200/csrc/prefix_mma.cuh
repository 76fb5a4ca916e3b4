// Parts of the shared prefix on the 5th-generation tensor cores (tcgen05), for
// batches with many query rows per KV head.
//
// A block takes 128 query rows (of all sequences) of one head and a range of
// the prefix's tokens, TN at a time:
//   S[row][token]  = Q (sigma c / 128)^T      both operands in shared memory;
//   P[row][token]  = 2^7 e^{x - ref}, fp16, written over S in tensor memory;
//   O[row][coord] += P (sigma c / 128)        P from tensor memory.
// Warps 4-7 turn packed codes into swizzled fp16 tiles (sigma c / 128, rounded
// once: at most |sigma|, so it cannot overflow), warp 8 issues the products,
// warps 0-3 hold a query row per thread: its maximum and sum need no exchange.
// Two score buffers let the tensor cores form the next scores while the
// exponentials of these are taken. O is rescaled only when a row's maximum
// grows by more than 2^8 over the reference its weights use (the weights then
// stay below 2^15 in fp16; the final quotient does not see the reference).
//
// The query row is scaled by a power of two to [2^13, 2^14) and rounded to
// fp16. For fp16 outputs (EXACT) that is not enough: queries, keys and weights
// are each split into an fp16 value and its rest, and the scores take the three
// products that matter, the values the two of the weights; the remaining
// rounding is that of the values, half a step of fp16, like the output's own.
// For bf16 outputs, with steps 8 times as wide, one product each is enough.
//
// What bounds it: per 128 rows and 64 tokens at d = 128 the two products take
// 512 clocks of the tensor cores and the exponentials 512 of the special
// function units; two blocks per SM overlap them with the decoding.
#pragma once

#include "paged_attention.cuh"
#include "tc.cuh"

namespace srftq {

constexpr int kMmaRows = 128;

template <int D, int BITS, int G, bool EXACT>
struct PrefixMma {
  static constexpr int TN = D == 256 && EXACT ? 32 : 64;      // tokens per step
  static constexpr int CB = D * BITS / 8, NG = D / G;
  static constexpr int kPieces = D / 64;                      // 128-byte columns of a row
  static constexpr int kQPiece = kMmaRows * 128, kQ = kPieces * kQPiece;
  static constexpr int kTPiece = TN * 128, kT = kPieces * kTPiece;   // a K or V tile
  static constexpr int kKT = kT * (EXACT ? 2 : 1);            // keys (and their rests)
  static constexpr int kStages = 2;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQ * (EXACT ? 2 : 1);
  static constexpr int kVOff = kKOff + kStages * kKT;
  static constexpr int kRowOff = kVOff + kStages * kT;        // float [128]: score factors
  static constexpr int kOnOff = kRowOff + 4 * kMmaRows;       // uint32 [4 steps][2]: tokens there
  static constexpr int kBarOff = kOnOff + 8 * 4;
  static constexpr int kBytes = kBarOff + 8 * 20 + 16;
  static constexpr int kSmem = kBytes + 1024;                 // slack to start on 1024 bytes
  static constexpr int kThreads = 288;
  static constexpr int kSCols = TN;                           // a score buffer
  static constexpr int kOCol = 2 * TN < 64 ? 64 : 2 * TN;
  static constexpr int kTmemCols = kOCol + D <= 128 ? 128 : kOCol + D <= 256 ? 256 : 512;
  // blocks per SM: shared memory and tensor memory both allow them
  static constexpr int kBlocks =
      2 * (kSmem + 1024) <= 227 * 1024 && 2 * kTmemCols <= 512 ? 2 : 1;
  static constexpr uint32_t kIdescS = f16_idesc<128, TN>();
  static constexpr uint32_t kIdescO = f16_idesc<128, D>() | (1u << 16);   // B is MN-major
};

// Position p of 8 consecutive coordinates in the decoded order: the code pairs
// that one AND isolates. int4: (0, 4), 16 (1, 5), (2, 6), 16 (3, 7); int8, two
// words of 4: (0, 2), (1, 3) each.
template <int BITS>
__host__ __device__ constexpr int decoded_coord(int p) {
  return BITS == 4 ? (p & 1) * 4 + (p >> 1) : (p & 4) + 2 * (p & 1) + ((p >> 1) & 1);
}
template <int BITS>
__host__ __device__ constexpr bool decoded_times16(int p) {
  return BITS == 4 && ((p >> 1) & 1);
}

// 8 codes (1 or 2 words) to sigma c / 128 in decoded order: v rounded to fp16,
// rest what that left (exact, but for subnormals).
template <int BITS, bool REST>
__device__ __forceinline__ void decode_chunk(const uint32_t* w, uint32_t sg2, uint4& v, uint4& rest) {
  constexpr uint32_t k128 = 0x20002000u;                     // 2^-7
  constexpr uint32_t o8 = 0xC808C808u, o128 = 0xC880C880u;   // -1032 / 128, -1152 / 128
  uint32_t c[4];
  if constexpr (BITS == 4) {
    const uint32_t y = w[0] >> 8;
    c[0] = hfma2((w[0] & 0x000F000Fu) ^ 0x64086408u, k128, o8);
    c[1] = hfma2((w[0] & 0x00F000F0u) ^ 0x64806480u, k128, o128);
    c[2] = hfma2((y & 0x000F000Fu) ^ 0x64086408u, k128, o8);
    c[3] = hfma2((y & 0x00F000F0u) ^ 0x64806480u, k128, o128);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[2 * i] = hfma2((w[i] & 0x00FF00FFu) ^ 0x64806480u, k128, o128);
      c[2 * i + 1] = hfma2(((w[i] >> 8) & 0x00FF00FFu) ^ 0x64806480u, k128, o128);
    }
  }
  v = make_uint4(hmul2(c[0], sg2), hmul2(c[1], sg2), hmul2(c[2], sg2), hmul2(c[3], sg2));
  if constexpr (REST) {
    rest = make_uint4(hfma2(c[0], sg2, v.x ^ 0x80008000u), hfma2(c[1], sg2, v.y ^ 0x80008000u),
                      hfma2(c[2], sg2, v.z ^ 0x80008000u), hfma2(c[3], sg2, v.w ^ 0x80008000u));
  }
}

template <int D, int BITS, int G, bool EXACT>
__global__ void __launch_bounds__(PrefixMma<D, BITS, G, EXACT>::kThreads,
                                  PrefixMma<D, BITS, G, EXACT>::kBlocks)
    prefix_mma_kernel(const PrefixArgs a) {
  using L = PrefixMma<D, BITS, G, EXACT>;
  constexpr int TN = L::TN, CB = L::CB, NG = L::NG;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_a = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((0u - raw_a) & 1023u);
  const uint32_t sm = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6;
  uint64_t *sfull = bars + 8, *pfull = bars + 10, *odone = bars + 12, *drain = bars + 13;   // drain: all products done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 15);
  float* row_f = reinterpret_cast<float*>(smem + L::kRowOff);
  volatile uint32_t* on_sh = reinterpret_cast<volatile uint32_t*>(smem + L::kOnOff);

  // this block's head, rows and tokens
  const int g = a.q_per_kv, hq = a.heads * g, M = a.n_seq * g;
  const int tiles = (M + kMmaRows - 1) / kMmaRows;
  const int rt = int(blockIdx.x) % tiles, sh = int(blockIdx.x) / tiles;
  const int h = sh % a.heads, part_i = sh / a.heads;
  const int r0 = rt * kMmaRows;
  const int t0 = part_i * a.prefix_per, t1 = min(t0 + a.prefix_per, a.prefix_len);
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
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  // queries: a warp per row in turn, lane l its columns 4 l .. (+ 128 i)
  for (int r = warp; r < kMmaRows; r += 9) {
    const int rr = min(r0 + r, M - 1);
    const float* qv = a.qrot + (int64_t(rr / g) * hq + h * g + rr % g) * D;
    // decoded position 4 l .. 4 l + 3: half of a chunk of 8 coordinates
    constexpr int NV = (D + 127) / 128;
    float x[NV][4];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int base = (128 * i + 4 * lane) & ~7, half = lane & 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c0 = decoded_coord<BITS>(k), c1 = decoded_coord<BITS>(4 + k);
        x[i][k] = 128 * i + 4 * lane < D ? __ldg(qv + base + (half ? c1 : c0)) : 0.0f;
        amax = fmaxf(amax, fabsf(x[i][k]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int ex = int((__float_as_uint(amax) >> 23) & 255u);
    const int e = ex > 0 && ex < 255 ? min(max(140 - ex, -100), 100) : 0;
    const float up = __uint_as_float(uint32_t(e + 127) << 23);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 128 * i + 4 * lane;
      if (col >= D) continue;
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = x[i][k] * up * (decoded_times16<BITS>(k) ? 0.0625f : 1.0f);
      const uint2 hi = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
      // row r of piece col / 64: 16-byte chunk (col % 64) / 8, XOR-swizzled
      const uint32_t at = sm + L::kQOff + (col >> 6) * L::kQPiece + r * 128 +
                          ((((col & 63) >> 3) ^ (r & 7)) << 4) + (col & 4) * 2;
      sts64(at, hi);
      if constexpr (EXACT)
        sts64(at + L::kQ, make_uint2(half2_rest(y[0], y[1], hi.x), half2_rest(y[2], y[3], hi.y)));
    }
    if (lane == 0) row_f[r] = __uint_as_float(uint32_t(127 - e) << 23) * 128.0f;
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      bool ok = true;
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
    constexpr int TH = 128 / TN;                 // threads per token
    constexpr int C = D / TH;                    // coordinates of a thread
    constexpr int NB = C * BITS / 8, NV = NB / 16;
    constexpr int GP = C > G ? C / G : 1;        // its scales
    static_assert(NB % 16 == 0, "whole 16-byte pieces");
    const int dt = tid - 128;
    const int tok = dt % TN, part = dt / TN;     // token of the step, part of the row
    const int sgi = part * C / G;
    uint4 kw[NV], vw[NV];
    uint16_t ks[GP], vs[GP];
    auto row_at = [&](int i) {
      const int t = t0 + i * TN + tok;
      return i < n && t < t1 ? a.map.row(a.prefix_table, uint32_t(t)) : int64_t(-1);
    };
    auto load = [&](int64_t row, const uint8_t* codes, const uint16_t* scales, uint4 (&w)[NV],
                    uint16_t (&s)[GP]) {
      const int64_t vec = (row < 0 ? 0 : row) * a.heads + h;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        w[k] = row < 0 ? make_uint4(0, 0, 0, 0)
                       : __ldg(reinterpret_cast<const uint4*>(codes + vec * CB + part * NB) + k);
#pragma unroll
      for (int k = 0; k < GP; ++k) s[k] = row < 0 ? uint16_t(0) : __ldg(scales + vec * NG + sgi + k);
    };
    // 16-byte chunk j of this thread's C coordinates in row `tok` of a tile
    auto chunk_at = [&](uint32_t tile, int j) {
      const int c = part * (C / 8) + j;
      return tile + (c >> 3) * L::kTPiece + tok * 128 + (((c & 7) ^ (tok & 7)) << 4);
    };
    int64_t row = row_at(0), next = row_at(1);
    if (n > 0) {
      load(row, a.k_codes, a.k_scales, kw, ks);
      load(row, a.v_codes, a.v_scales, vw, vs);
    }
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const int64_t after = row_at(i + 2);
      if (i >= 2 && !__all_sync(0xffffffffu, wait_or_abort(&kempty[st], ((i >> 1) & 1) ^ 1,
                                                           abort_flag, a.guard)))
        break;
      const uint32_t on = __ballot_sync(0xffffffffu, row >= 0);
      // a slot is written again four steps on, after the scores of step i + 2,
      // which follow the weights of this step
      if (part == 0 && lane == 0) {
        on_sh[2 * (i & 3) + (tok >> 5)] = on;
        __threadfence_block();
      }
      const uint32_t kt = sm + L::kKOff + st * L::kKT;
#pragma unroll
      for (int j = 0; j < C / 8; ++j) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(kw) + j * BITS / 4;
        const uint32_t s = ks[8 * j / G];
        uint4 v, r;
        decode_chunk<BITS, EXACT>(w, s | (s << 16), v, r);
        sts128(chunk_at(kt, j), v);
        if constexpr (EXACT) sts128(chunk_at(kt + L::kT, j), r);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[st]);
      if (i + 1 < n) load(next, a.k_codes, a.k_scales, kw, ks);
      if (i >= 2 && !__all_sync(0xffffffffu, wait_or_abort(&vempty[st], ((i >> 1) & 1) ^ 1,
                                                           abort_flag, a.guard)))
        break;
      const uint32_t vt = sm + L::kVOff + st * L::kT;
#pragma unroll
      for (int j = 0; j < C / 8; ++j) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(vw) + j * BITS / 4;
        const uint32_t s = vs[8 * j / G];
        uint4 v, r;
        decode_chunk<BITS, false>(w, s | (s << 16), v, r);
        sts128(chunk_at(vt, j), v);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&vfull[st]);
      if (i + 1 < n) load(next, a.v_codes, a.v_scales, vw, vs);
      row = next;
      next = after;
    }
  } else {
    // ---------------- softmax: a query row per thread ----------------
    const int r = tid;                       // row of the tile, lane of tensor memory
    const int rr = min(r0 + r, M - 1);
    const int lim = a.len(rr / g);
    const float f = row_f[r];
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
      const uint32_t on0 = on_sh[2 * (i & 3)];
      const uint32_t on1 = TN == 64 ? on_sh[2 * (i & 3) + 1] : 0xffffffffu;
      if (!__all_sync(0xffffffffu, (on0 & on1) == 0xffffffffu && tk + TN <= lim)) {
#pragma unroll
        for (int k = 0; k < TN / 32; ++k)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(((k ? on1 : on0) >> j) & 1u) || tk + 32 * k + j >= lim) s[k][j] = 0xff800000u;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < TN / 32; ++k)
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          mx = fmaxf(mx, fmaxf(__uint_as_float(s[k][j]), __uint_as_float(s[k][j + 1])));
      mx *= f;                               // f > 0
      const bool grow = mx > ref + 8.0f || (ref == -INFINITY && mx > -INFINITY);
      const float nref = grow ? mx : ref;
      const float cc = !grow ? 1.0f : ref == -INFINITY ? 0.0f : ex2(ref - nref);
      l *= cc;
      ref = nref;
      // P = 2^7 e^{x - ref} (0 while the row has seen no token)
      const float b = 7.0f - (ref == -INFINITY ? 0.0f : ref);
      float sum = 0.0f, sum1 = 0.0f;
      uint32_t ph[32];
      uint32_t pl[EXACT ? 32 : 1];
#pragma unroll
      for (int k = 0; k < TN / 32; ++k)
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float p0 = ex2(fmaf(__uint_as_float(s[k][j]), f, b));
          const float p1 = ex2(fmaf(__uint_as_float(s[k][j + 1]), f, b));
          sum += p0;
          sum1 += p1;
          const uint32_t hh = pack_half2(p0, p1);
          ph[16 * k + j / 2] = hh;
          if constexpr (EXACT) pl[16 * k + j / 2] = half2_rest(p0, p1, hh);
        }
      l += sum + sum1;
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
      const int64_t part = (int64_t(part_i) * a.heads + h) * M + r0 + r;
      const bool live = r0 + r < M;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        tmem_ld32(tl + L::kOCol + k, o);
        tmem_wait_ld1(o);
        if (live) {
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)   // 128 / 2^7 = 1
            y[(j & ~7) + decoded_coord<BITS>(j & 7)] =
                __uint_as_float(o[j]) * (decoded_times16<BITS>(j & 7) ? 0.0625f : 1.0f);
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
