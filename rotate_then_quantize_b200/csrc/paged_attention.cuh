// Decode attention over a paged quantised cache for a batch that shares a
// prefix: the shared tokens are read once for all sequences, every sequence's
// own tokens once for its query heads.
//
// For sequence b, query head h g + j (KV head h) and the tokens t < len_b:
//   out = sum_t p_t vhat_t,  p = softmax_t(scale q . khat_t),
// with khat, vhat the dequantised rows. As in attention.cuh the work is done
// in the rotated domain (R is orthogonal: "When Quantization Is Free",
// Methodology 1): with c the codes and sigma the group scales,
//   q . khat_t = (lambda_K * R_K (s_K q)) . (sigma c)_t,
//   out = s_V * R_V^T (lambda_V * sum_t p_t (sigma c)_t).
// The softmax splits over tokens: a part with scores x_t has the state
//   m = max x_t,  l = sum e^{x_t - m},  a = sum e^{x_t - m} (sigma c)_t,
// and parts join as m = max m_i, l = sum l_i e^{m_i - m}, a likewise. Tokens
// below prefix_len are one part (or several) whose rows are the queries of all
// sequences; the rest of each sequence are parts of its own.
//
// Three launches on the caller's stream (four with prefix_mma.cuh), each but the
// first a programmatic one:
//   prefix_prepare_kernel   a warp per query: lambda_K * R_K (s_K q) * scale *
//                           log2 e into the workspace; block 0 also plans the
//                           split of the sequences' own tokens;
//   prefix_tile_kernel      the parts, each (m, l, a) into the workspace;
//   prefix_merge_kernel     1, 4 or 16 warps per query head: joins its parts,
//                           applies lambda_V / l, R_V^T and s_V, rounds once. A
//                           head whose sums are not finite, for a scale too large
//                           for the parts' fp16 (kLargeScale), is done anew there.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "pages.cuh"
#include "ptx.cuh"
#include "token_plan.cuh"
#include "warp_rotate.cuh"

namespace srftq {

constexpr int kPrefixRows = 8;        // query rows of one item
constexpr float kLog2e = 1.4426950408889634f;

// Plan of the own tokens, in the workspace: header, then start[n_seq + 1], the
// first chunk of every sequence (chunk c of sequence b covers the own tokens
// [c chunk, (c + 1) chunk)).
struct PrefixPlan {
  int32_t n_chunks;   // chunks of all sequences
  int32_t taken;      // items that blocks have taken beyond their first
};

struct PrefixArgs {
  int32_t n_seq, heads, q_per_kv, lg_group;
  int32_t prefix_len, max_pages;
  int32_t prefix_splits, prefix_per;   // parts of the prefix and tokens of each
  int32_t chunk_goal;                  // chunks that the plan aims for
  PageMap map;
  const void* q;                       // [n_seq][heads q_per_kv][d] fp16 or bf16
  bool bf16;
  const uint8_t* k_codes;              // pool rows of [heads][d bits / 8]
  const uint16_t* k_scales;            // pool rows of [heads][d / group]
  const int8_t* k_signs;
  const float* k_lambda;
  const uint8_t* v_codes;
  const uint16_t* v_scales;
  const int8_t* v_signs;
  const float* v_lambda;
  const int32_t* prefix_table;
  const int32_t* block_table;          // [n_seq][max_pages]
  const int32_t* seq_lens;
  float scale;
  void* out;                           // like q
  float* lse;                          // [n_seq][heads q_per_kv] or null
  bool pre_mma;                        // the prefix's parts come from a tcgen05 kernel
  bool pre_shared;                     // whose two units are different rows (prefix_pair.cuh)
  int32_t bits;
  uint32_t zero;                       // 0 (in_register)
  float* qrot;                         // workspace: rotated queries
  uint8_t* q_image;                    // pre_mma: the rows' fp16 tiles, [heads][tiles] of them
  float* q_factor;                     // and the rows' score factors, [heads][tiles * 128]
  PrefixPlan* plan;
  int32_t* chunk_start;
  int4* chunk_of;                      // of each chunk: sequence, first token, end, 0
  float2* pre_ml;                      // [splits][heads][n_seq q_per_kv]
  float* pre_acc;                      // the same rows of d
  float2* own_ml;                      // [chunks][heads][q_per_kv]
  float* own_acc;
  unsigned* guard;

  // tokens of sequence b: all, those of its own
  __device__ __forceinline__ int32_t len(int b) const {
    const int64_t cap = int64_t(max_pages) * map.page.d;
    const int64_t most = cap > prefix_len ? cap : prefix_len;
    const int32_t n = seq_lens[b];
    return n < 0 ? 0 : n > most ? int32_t(most) : n;
  }
  __device__ __forceinline__ int32_t own(int b) const { return max(len(b) - prefix_len, 0); }

  // Index checks of the debug build: a token's table entry (the prefix's table or a
  // sequence's), a row of the pool, a query head, a chunk record, a row of the parts.
  __device__ __forceinline__ bool dbg_token(bool pre, int64_t t) const {
    return dbg_ok(t >= 0 && t < (pre ? int64_t(prefix_len) : int64_t(max_pages) * map.page.d), guard);
  }
  __device__ __forceinline__ bool dbg_row(int64_t row) const {
    return dbg_ok(row >= 0 && row < int64_t(map.n_pages) * map.page.d, guard);
  }
  __device__ __forceinline__ bool dbg_query(int64_t v) const {
    return dbg_ok(v >= 0 && v < int64_t(n_seq) * heads * q_per_kv, guard);
  }
  __device__ __forceinline__ bool dbg_chunk(int64_t c) const {
    return dbg_ok(c >= 0 && c < int64_t(chunk_goal) + n_seq, guard);
  }
  __device__ __forceinline__ bool dbg_part(bool pre, int64_t part) const {
    const int64_t chunks = int64_t(chunk_goal) + n_seq, rows = int64_t(n_seq) * q_per_kv;
    return dbg_ok(part >= 0 && part < heads * (pre ? prefix_splits * rows : chunks * q_per_kv), guard);
  }
  // Pool row of token t, -1 when it has none.
  __device__ __forceinline__ int64_t pool_row(bool pre, const int32_t* table, uint32_t t) const {
    if (!dbg_token(pre, t)) return -1;
    const int64_t row = map.row(table, t);
    return row < 0 || dbg_row(row) ? row : -1;
  }
};

__device__ __forceinline__ float lo_f32(uint32_t w, bool bf16) {
  return bf16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half(uint16_t(w)));
}
__device__ __forceinline__ float hi_f32(uint32_t w, bool bf16) {
  return bf16 ? __uint_as_float(w & 0xFFFF0000u) : __half2float(__ushort_as_half(uint16_t(w >> 16)));
}

// Programmatic launches (launch_after): the next grid may start from here on;
// the grids before this one are complete from here on. So a grid may be resident
// while the one before still writes the workspace: what it finds there it reads
// with ordinary loads, never through the read-only path (__ldg), which may return
// what a line held before. The caller's inputs are complete before the first
// launch starts.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Block-wide scan of the chunk counts (all threads of a block of 256).
__device__ inline void plan_own_tokens(const PrefixArgs& a) {
  __shared__ int64_t total_sh[8];
  __shared__ int32_t wsum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  int64_t total = 0;
  for (int b = tid; b < a.n_seq; b += nt) total += a.own(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) total_sh[warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < nt / 32; ++w) total += total_sh[w];
  // chunks of at least 128 tokens (a tile for each warp), few enough that
  // sum ceil(own / chunk) <= goal + n_seq
  const int32_t chunk = chunk_tokens(total, a.chunk_goal);
  int32_t carry = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += nt) {
    const int b = b0 + tid;
    const int32_t n = b < a.n_seq ? chunks_of(a.own(b), chunk) : 0;
    int32_t v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    int32_t before = carry, all = carry;
    for (int w = 0; w < nt / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (b < a.n_seq) a.chunk_start[b] = before + v - n;
    carry = all;
  }
  // the chunks' sequences and tokens, so that a block has its next item in one load
  for (int b = tid; b < a.n_seq; b += nt) {
    const int32_t end = a.len(b), n = chunks_of(a.own(b), chunk);
    int4* o = a.chunk_of + a.chunk_start[b];   // this thread wrote it
    for (int32_t c = 0; c < n; ++c) {
      const int32_t t0 = a.prefix_len + c * chunk;
      if (a.dbg_chunk(o + c - a.chunk_of)) o[c] = make_int4(b, t0, range_end(t0, chunk, end), 0);
    }
  }
  if (tid == 0) {
    a.chunk_start[a.n_seq] = carry;
    a.plan->n_chunks = carry;
    a.plan->taken = 0;
  }
}

// e with 2^e amax in [2^13, 2^14); 0 for a zero or infinite query.
__device__ __forceinline__ int query_exponent(float amax) {
  const int ex = int((__float_as_uint(amax) >> 23) & 255u);
  return ex > 0 && ex < 255 ? min(max(140 - ex, -100), 100) : 0;
}

// Row r of head h in the fp16 tiles that the tcgen05 kernel copies to shared
// memory as they are: tiles of 128 rows, each (for fp16 outputs) followed by the
// rests; a tile is d / 64 pieces of rows of 128 bytes whose 16-byte chunks are
// XOR-swizzled by the row. The 8 coordinates of a chunk lie in the order that
// decoding the codes gives (prefix_mma.cuh: decoded_coord).
template <int D>
struct QueryRow {
  uint8_t* p;
  float* factor;
  int r;
  bool exact, four;
  __device__ __forceinline__ QueryRow(const PrefixArgs& a, int h, int row) {
    exact = !a.bf16;
    four = a.bits == 4;
    const int tiles = (a.n_seq * a.q_per_kv + 127) / 128;
    const int64_t tile = int64_t(h) * tiles + row / 128;
    r = row % 128;
    p = a.q_image + tile * (256 * D * (exact ? 2 : 1));
    factor = a.q_factor + tile * 128 + r;
  }
  __device__ __forceinline__ void put(int c, float x) const {
    const int at = four ? (c & 3) * 2 + ((c >> 2) & 1)
                        : (c & 4) + (c & 1) * 2 + ((c >> 1) & 1);
    uint8_t* q = p + (c >> 6) * 16384 + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + at * 2;
    const __half hi = __float2half_rn(x);
    *reinterpret_cast<__half*>(q) = hi;
    if (exact) *reinterpret_cast<__half*>(q + 256 * D) = __float2half_rn(x - __half2float(hi));
  }
};

template <int ROT, int D>
__global__ void __launch_bounds__(256) prefix_prepare_kernel(const PrefixArgs a) {
  constexpr int E = D / 64;
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int hq = a.heads * a.q_per_kv;
  const int64_t total = int64_t(a.n_seq) * hq;
  const float f = a.scale * kLog2e;
  for (int64_t v = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; v < total;
       v += (int64_t(gridDim.x) * blockDim.x) >> 5) {
    if (!a.dbg_query(v)) continue;
    const int h = int(v % hq) / a.q_per_kv;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + v * (D / 2) + lane * E;
    const int8_t* sg = a.k_signs + int64_t(h) * D + 2 * E * lane;
    float2 z[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t w = q[e];
      const float x0 = lo_f32(w, a.bf16), x1 = hi_f32(w, a.bf16);
      z[e] = make_float2(sg[2 * e] < 0 ? -x0 : x0, sg[2 * e + 1] < 0 ? -x1 : x1);
    }
    warp_rotate_forward<ROT, D>(z, lane);
    const float2* lam = reinterpret_cast<const float2*>(a.k_lambda + int64_t(h) * D);
    float2* o = reinterpret_cast<float2*>(a.qrot + v * D);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = warp_pair<ROT, D>(lane, e);
      const float2 l = lam[k];
      z[e] = make_float2(z[e].x * l.x * f, z[e].y * l.y * f);
      o[k] = z[e];
      amax = fmaxf(amax, fmaxf(fabsf(z[e].x), fabsf(z[e].y)));
    }
    if (a.pre_mma) {
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, i));
      const int e2 = query_exponent(amax);
      const float up = __uint_as_float(uint32_t(e2 + 127) << 23);
      const int b = int(v / hq), j = int(v % hq) % a.q_per_kv;
      const int r = b * a.q_per_kv + j;
      const QueryRow<D> row(a, h, r);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int k = warp_pair<ROT, D>(lane, e);
        row.put(2 * k, z[e].x * up);
        row.put(2 * k + 1, z[e].y * up);
      }
      if (lane == 0) *row.factor = __uint_as_float(uint32_t(127 - e2) << 23);
    }
  }
  if (a.pre_mma) {   // rows behind the last query: zeros
    const int M = a.n_seq * a.q_per_kv, pad = (M + 127) / 128 * 128 - M;
    for (int64_t v = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         v < int64_t(pad) * a.heads; v += (int64_t(gridDim.x) * blockDim.x) >> 5) {
      const QueryRow<D> row(a, int(v / pad), M + int(v % pad));
      for (int c = lane; c < D; c += 32) row.put(c, 0.0f);
      if (lane == 0) *row.factor = 1.0f;
    }
  }
  if (blockIdx.x == 0) plan_own_tokens(a);
}

// ---------------------------------------------------------------------------
// Parts on the warp-level tensor cores (mma.sync)
// ---------------------------------------------------------------------------
//
// An item is up to 8 query rows x a range of tokens of one head. A warp takes
// 32 tokens at a time through a ring of cp.async stages and keeps its own
// online softmax. Tokens are the rows of both products' left operands:
//
// Scores, S[token][query] = sum_G sigma_G D_G, D_G = sum_{j in G} c_j q_j, one
// m16n8k16 per 16 coordinates. The codes enter exactly: with u = c + 8 (int4)
// or c + 128 (int8), the 16-bit pattern u is the fp16 subnormal u 2^-24, so one
// AND-XOR makes two operands of a packed word. The offset leaves through one
// more product, of the scales (fp16, exact) with -8 2^-24 sum_{j in G} q_j. The
// query is scaled by a power of two to [2^13, 2^14) and held as fp16 hi (+ lo
// when the output is fp16). The scale multiplies D_G in float32, so a score's
// roundings to fewer bits are the query's, 2^-12 for bf16 outputs (whose own
// step is 2^-9), 2^-23 for fp16, and the offset's: its lo ends at fp16's last
// subnormal bit, half a step of which is half of c q at q = 1, where q is up to
// 2^14: 2^-17 of a score's standard deviation over 8 groups of 16 int4 codes.
//
// Values, O[coord][query] += sum_t (sigma c)[coord][t] p'[t][query], p' =
// 2^7 e^{x - m}, m a reference that follows the maximum when that grows by more
// than 2^8 (the factors keep small weights normal and large ones below 2^15).
// sigma c is rounded once to fp16 (kLargeScale). The 8-bit
// transposing ldmatrix gives lane (g, t) coordinate g of tokens 4t .. 4t + 3,
// and the score rows take their tokens in the order that hands the lane's p'
// over with one movmatrix. p' is fp16 hi (+ lo for fp16 outputs).
//
// What bounds it: latency. Codes and scales of a vector are read once per 8
// queries, one chunk of a warp is one chain (scores, maximum, exponentials,
// movmatrix, values), and 16 to 20 warps per SM fill about half the issue slots.
// 64 ragged sequences of up to 2048 tokens, 8 heads of d = 64, int4, 37.5 MB: 40
// us for the whole call; this kernel under ncu, from cold caches, 34 us at 14 % of
// the memory's rate, 16 % of the tensor pipe and 48 % of the issue slots.

constexpr int kTileWarps = 4;
constexpr int kTileChunk = 32;   // tokens a warp takes at a time

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void ldmatrix_bytes_trans(uint32_t& r0, uint32_t& r1, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x1.trans.shared.b8 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr));
}
// The products sigma c are held as fp16. A scale is a whole number of 2^-24 and c
// a whole number, so sigma c has no bits below the subnormals' last one: it is
// rounded to 11 significant bits and to nothing else, however small the scale.
// Scales below this one, 8192 with |c| <= 8 or 512 with |c| <= 128, keep it at
// 65504 at most. A row that attends to a token with a larger scale, or with one
// that is not finite, takes NaN for its sum, and the join does it anew in float32.
// Calibrated scales are of order one; only vectors next to fp16's own end reach it.
template <int BITS>
constexpr uint32_t kLargeScale = BITS == 4 ? 0x7000u : 0x6000u;
// 0x8000 in each half that is an infinite or NaN fp16.
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t s) {
  return ((s & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
// 0x8000 in each half whose magnitude is at least that, infinite or NaN.
template <int BITS>
__device__ __forceinline__ uint32_t large_halves(uint32_t s) {
  return ((s & 0x7FFF7FFFu) + (0x8000u - kLargeScale<BITS>) * 0x10001u) & 0x80008000u;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2_away(float lo, float hi) {
  const __half2 h = __halves2half2(lo < 0.0f ? __float2half_rd(lo) : __float2half_ru(lo),
                                   hi < 0.0f ? __float2half_rd(hi) : __float2half_ru(hi));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The part of (x, y) that their fp16 roundings h leave, rounded to fp16.
__device__ __forceinline__ uint32_t half2_rest(float x, float y, uint32_t h) {
  const float2 f = unpack_half2(h);
  return pack_half2(x - f.x, y - f.y);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A constant in a register (zero is a kernel argument that is 0, so that it
// cannot be folded): (w & mask) ^ magic is one instruction with one immediate and
// one register, two with two immediates.
__device__ __forceinline__ uint32_t in_register(uint32_t c, uint32_t zero) { return c ^ zero; }
// 16 bytes of global memory to shared memory, zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
               "r"(on ? BYTES : 0)
               : "memory");
}

// Shared memory of one warp: kStages stages of 32 tokens. Rows are padded by 16
// bytes, which puts the 8 rows that a load of any kind here touches together on
// distinct banks. Scale rows are 16 bytes at least, their unused part zero.
template <int D, int BITS, int G>
struct TileLayout {
  static constexpr int CB = D * BITS / 8, NG = D / G, NS16 = D / 16;
  static constexpr int RS = CB + 16;
  static constexpr int SB = 2 * NG, SBS = SB < 16 ? 16 : SB;
  static constexpr int kK = 0, kV = 32 * RS, kKS = 64 * RS, kVS = kKS + 32 * SBS;
  static constexpr int kStage = kVS + 32 * SBS;
  static constexpr int kStages = 2;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kMl = kTileWarps * kWarp;             // the warps' (m, l) of 8 rows
  // the item's queries, the same for its warps: right operands by coordinate
  // group of 16 and lane, hi then lo; float sums [NS16][8 rows]
  static constexpr int kQf = kMl + kTileWarps * 8 * 8;
  static constexpr int kQs = kQf + 2 * NS16 * 32 * 8;
  static constexpr int kBytes = kQs + NS16 * 8 * 4;
  static_assert(kWarp >= 8 * D * 4, "a warp's partial sums fit over its stages");
};

// The item's rows and tokens (shared by the kernels below).
struct PartItem {
  int h, b, r0, nr, t0, t1;
  bool pre;
  int64_t part;
  const int32_t* table;
};

// Own-token item i: a chunk of a sequence (rec, of chunk own_chunk()), head h,
// row tile rt.
__device__ __forceinline__ int64_t own_chunk(const PrefixArgs& a, int64_t i, int tiles) {
  return i / (int64_t(tiles) * a.heads);
}
__device__ __forceinline__ PartItem own_item(const PrefixArgs& a, int64_t i, int tiles, int4 rec) {
  PartItem p;
  p.pre = false;
  const int rt = int(i % tiles);
  const int64_t q = i / tiles;
  p.h = int(q % a.heads);
  p.b = rec.x;
  p.r0 = rt * kPrefixRows;
  p.nr = min(kPrefixRows, a.q_per_kv - p.r0);
  p.t0 = rec.y;
  p.t1 = rec.z;
  p.part = q * a.q_per_kv + p.r0;
  p.table = a.block_table + int64_t(rec.x) * a.max_pages;
  return p;
}
// Prefix item i: part s of the prefix, head h, row tile rt.
__device__ __forceinline__ PartItem pre_item(const PrefixArgs& a, int64_t i, int tiles) {
  PartItem p;
  p.pre = true;
  const int M = a.n_seq * a.q_per_kv;
  const int rt = int(i % tiles);
  const int64_t q = i / tiles;
  p.h = int(q % a.heads);
  const int s = int(q / a.heads);
  p.b = 0;
  p.r0 = rt * kPrefixRows;
  p.nr = min(kPrefixRows, M - p.r0);
  p.t0 = s * a.prefix_per;
  p.t1 = range_end(p.t0, a.prefix_per, a.prefix_len);
  p.part = (int64_t(s) * a.heads + p.h) * M + p.r0;
  p.table = a.prefix_table;
  return p;
}

template <int D, int BITS, int G, bool EXACT>
__global__ void __launch_bounds__(kTileWarps * 32, D == 256 ? 2 : D == 128 ? 4 : 5)
    prefix_tile_kernel(const PrefixArgs a) {
  using L = TileLayout<D, BITS, G>;
  constexpr int CB = L::CB, NG = L::NG, NS = L::kStages, S16 = L::NS16, NW = kTileWarps;
  constexpr int PPT = CB / 16;          // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  grid_launch_dependents();
  grid_dependency_wait();
  float2(*ml_sh)[8] = reinterpret_cast<float2(*)[8]>(smem + L::kMl);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ws = smem + warp * L::kWarp;
  const uint32_t ws_a = smem_addr(ws);
  const int qpk = a.q_per_kv, hq = a.heads * qpk;
  const int M = a.n_seq * qpk;
  const int pre_tiles =
      a.prefix_len > 0 && !a.pre_mma ? (M + kPrefixRows - 1) / kPrefixRows : 0;
  const int64_t n_pre = int64_t(a.prefix_splits) * a.heads * pre_tiles;
  const int own_tiles = (qpk + kPrefixRows - 1) / kPrefixRows;
  const int64_t n_items = n_pre + int64_t(a.plan->n_chunks) * a.heads * own_tiles;

  // A block takes the next item when it is done with one: sequences differ in
  // length, and which block does an item changes nothing in it.
  __shared__ int32_t next_sh;
  __shared__ int4 rec_sh;
  auto record = [&](int64_t i) {
    if (i < n_pre || i >= n_items) return make_int4(0, 0, 0, 0);
    const int64_t c = own_chunk(a, i - n_pre, own_tiles);
    return a.dbg_chunk(c) ? a.chunk_of[c] : make_int4(0, 0, 0, 0);
  };
  int4 rec = record(blockIdx.x);
  for (int64_t it = blockIdx.x; it < n_items;) {
    const PartItem p =
        it < n_pre ? pre_item(a, it, pre_tiles) : own_item(a, it - n_pre, own_tiles, rec);
    // the next item and its record are on their way while this one is done
    int32_t next = 0;
    int4 next_rec;
    if (threadIdx.x == 0) {
      next = atomicAdd(&a.plan->taken, 1);
      next_rec = record(int64_t(gridDim.x) + next);
    }
    const int n_chunks = max(0, (p.t1 - p.t0 - kTileChunk * warp + kTileChunk * NW - 1) /
                                    (kTileChunk * NW));
    // zero the unused part of the scale rows (partial sums lay there before)
    if constexpr (L::SB < 16) {
      for (int st = 0; st < NS; ++st) {
        *reinterpret_cast<uint4*>(ws + st * L::kStage + L::kKS + lane * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(ws + st * L::kStage + L::kVS + lane * 16) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }

    // pool row of this lane's token of chunk c, -1 for none
    auto row_of = [&](int c) {
      const int tok = p.t0 + kTileChunk * (warp + NW * c) + lane;
      return c < n_chunks && tok < p.t1 ? int32_t(a.pool_row(p.pre, p.table, uint32_t(tok))) : -1;
    };
    // copies chunk c, this lane's token in pool row `row`, into stage c % NS
    auto issue = [&](int c, int32_t row) {
      if (c < n_chunks) {
        const uint32_t st = ws_a + uint32_t(c % NS) * L::kStage;
#pragma unroll
        for (int k = 0; k < PPT; ++k) {
          const int i = lane + 32 * k, tok = i / PPT, pc = i % PPT;
          const int32_t r = __shfl_sync(0xffffffffu, row, tok);
          const int64_t vec = int64_t(r < 0 ? 0 : r) * a.heads + p.h;
          // score rows: token 2i in row i, token 2i + 1 in row i + 8 of each 16
          const int kr = (tok & 16) | ((tok & 1) << 3) | ((tok & 15) >> 1);
          copy16(st + L::kK + kr * L::RS + pc * 16, a.k_codes + vec * CB + pc * 16, r >= 0);
          copy16(st + L::kV + tok * L::RS + pc * 16, a.v_codes + vec * CB + pc * 16, r >= 0);
        }
        const int64_t vec = int64_t(row < 0 ? 0 : row) * a.heads + p.h;
        const int kr = (lane & 16) | ((lane & 1) << 3) | ((lane & 15) >> 1);
        const uint32_t dk = st + L::kKS + kr * L::SBS, dv = st + L::kVS + lane * L::SBS;
        const uint16_t *ks = a.k_scales + vec * NG, *vs = a.v_scales + vec * NG;
        if constexpr (L::SB >= 16) {
#pragma unroll
          for (int i = 0; i < L::SB / 16; ++i) {
            copy16(dk + 16 * i, ks + 8 * i, row >= 0);
            copy16(dv + 16 * i, vs + 8 * i, row >= 0);
          }
        } else if constexpr (L::SB >= 4) {
          copy_small<L::SB>(dk, ks, row >= 0);
          copy_small<L::SB>(dv, vs, row >= 0);
        } else {   // one scale: 2 bytes, below the smallest asynchronous copy
          uint8_t* sp = ws + (c % NS) * L::kStage;
          *reinterpret_cast<uint16_t*>(sp + L::kKS + kr * L::SBS) = row >= 0 ? ks[0] : uint16_t(0);
          *reinterpret_cast<uint16_t*>(sp + L::kVS + lane * L::SBS) = row >= 0 ? vs[0] : uint16_t(0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int32_t row_at[NS];   // rows of the chunks in flight, then of the next one
#pragma unroll
    for (int c = 0; c < NS; ++c) row_at[c] = row_of(c);
#pragma unroll
    for (int c = 0; c < NS - 1; ++c) issue(c, row_at[c]);

    // query g, this lane's coordinates 16 s + 4 t .. + 3: every warp finds the
    // row's scale, each makes the operands of every fourth s
    const int rq = p.r0 + min(g, p.nr - 1);
    const int bq = p.pre ? rq / qpk : p.b;
    const float* qv = a.qrot + (int64_t(bq) * hq + p.h * qpk + (p.pre ? rq % qpk : rq)) * D;
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < S16; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(qv + 16 * s + 4 * t);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = query_exponent(amax);
    const float up = __uint_as_float(uint32_t(e + 127) << 23);
    const uint32_t qf = smem_addr(smem + L::kQf) + lane * 8;
    float* qsum = reinterpret_cast<float*>(smem + L::kQs);
#pragma unroll
    for (int i = 0; i < S16 / NW; ++i) {
      const int s = warp + NW * i;
      const float4 x = *reinterpret_cast<const float4*>(qv + 16 * s + 4 * t);
      constexpr float odd = BITS == 4 ? 0.0625f : 1.0f;   // int4: odd coordinates' codes are 16 u
      const float x0 = x.x * up, x1 = x.y * up * odd, x2 = x.z * up, x3 = x.w * up * odd;
      const uint2 hi = make_uint2(pack_half2(x0, x2), pack_half2(x1, x3));
      sts64(qf + s * 256, hi);
      float2 f0 = unpack_half2(hi.x), f1 = unpack_half2(hi.y);
      if constexpr (EXACT) {
        const uint2 lo = make_uint2(half2_rest(x0, x2, hi.x), half2_rest(x1, x3, hi.y));
        sts64(qf + (S16 + s) * 256, lo);
        const float2 l0 = unpack_half2(lo.x), l1 = unpack_half2(lo.y);
        f0 = make_float2(f0.x + l0.x, f0.y + l0.y);
        f1 = make_float2(f1.x + l1.x, f1.y + l1.y);
      }
      float sum = (f0.x + f0.y) + (f1.x + f1.y) * (1.0f / odd);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (t == 0) qsum[8 * s + g] = sum;
    }
    __syncthreads();
    // offsets of groups 2t, 2t + 1 (+ 8 o) as fp16 hi and lo: -(8 or 128) 2^-24 sum q.
    // hi is rounded away from zero, so lo has the other sign or is zero: an infinite
    // scale of keys then makes the score NaN, never the -inf of a token not attended to
    constexpr int NO = NG > 8 ? NG / 8 : 1;
    uint32_t off[NO][2];
#pragma unroll
    for (int o = 0; o < NO; ++o) {
      float x[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int gi = 8 * o + 2 * t + k;
        if (gi < NG) {
#pragma unroll
          for (int i = 0; i < G / 16; ++i) x[k] += qsum[8 * (gi * (G / 16) + i) + g];
        }
        x[k] *= BITS == 4 ? -0x1p-21f : -0x1p-17f;
      }
      off[o][0] = pack_half2_away(x[0], x[1]);
      off[o][1] = half2_rest(x[0], x[1], off[o][0]);
    }
    // columns 2t and 2t + 1 of the score tile: their factor, token limit
    const float down = __uint_as_float(uint32_t(127 - e) << 23) * 0x1p24f;
    const int lim_g = p.pre ? a.len(bq) : p.t1;
    float fs[2];
    int lim[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      fs[c] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * c);
      lim[c] = __shfl_sync(0xffffffffu, lim_g, 8 * t + 4 * c);
    }

    // u of even and odd coordinates as fp16 subnormals; 1024 + u, 1024 + 16 u
    const uint32_t u_lo = in_register(BITS == 4 ? 0x00080008u : 0x00800080u, a.zero);
    const uint32_t u_hi = in_register(0x00800080u, a.zero);
    const uint32_t h_lo = in_register(BITS == 4 ? 0x64086408u : 0x64806480u, a.zero);
    const uint32_t h_hi = in_register(0x64806480u, a.zero);
    float O[S16][4];
    // per column the reference of the weights (within 2^8 of the maximum), their sum
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int bad = INT_MAX;   // the first prefix token with a large scale of values
#pragma unroll
    for (int s = 0; s < S16; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[s][i] = 0.0f;

    for (int c = 0; c < n_chunks; ++c) {
      const uint32_t here = __ballot_sync(0xffffffffu, row_at[0] >= 0);
#pragma unroll
      for (int i = 0; i + 1 < NS; ++i) row_at[i] = row_at[i + 1];
      issue(c + NS - 1, row_at[NS - 2]);
      row_at[NS - 1] = row_of(c + NS);
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
      __syncwarp();
      const uint32_t st = ws_a + uint32_t(c % NS) * L::kStage;
      const int tk = p.t0 + kTileChunk * (warp + NW * c);

      // A row that ends before a token has weight 0 there, which a value past fp16
      // would still make NaN: large scales enter as 0, and the rows that reach the
      // first of them take NaN for their sum at the end. (A sequence's own tokens
      // end for all rows together, behind them are zeros; a value past fp16 makes the
      // sums infinite or NaN.)
      if (p.pre) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < (NG + 7) / 8; ++i) {
          const uint4 u = lds128(st + L::kVS + lane * L::SBS + 16 * i);
          any |= large_halves<BITS>(u.x) | large_halves<BITS>(u.y) | large_halves<BITS>(u.z) |
                 large_halves<BITS>(u.w);
        }
        if (__any_sync(0xffffffffu, any != 0)) {
          if (any) {
            bad = min(bad, tk + lane);
            uint16_t* sv = reinterpret_cast<uint16_t*>(ws + (c % NS) * L::kStage + L::kVS +
                                                       lane * L::SBS);
            for (int i = 0; i < NG; ++i) sv[i] = 0;
          }
          __syncwarp();
        }
      }

      // scores of the chunk's two tiles: rows g, g + 8 = tokens 2g, 2g + 1
      float S[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint32_t k0 = st + L::kK + (16 * mt + g) * L::RS, k1 = k0 + 8 * L::RS;
        const uint32_t s0 = st + L::kKS + (16 * mt + g) * L::SBS, s1 = s0 + 8 * L::SBS;
#pragma unroll
        for (int i = 0; i < 4; ++i) S[mt][i] = 0.0f;
#pragma unroll
        for (int o = 0; o < NO; ++o) {
          const uint32_t w0 = lds32(s0 + 16 * o + 4 * t), w1 = lds32(s1 + 16 * o + 4 * t);
          mma_f16(S[mt], w0, w1, w0, w1, off[o][0], off[o][1]);
        }
        float sg0[NG], sg1[NG];
#pragma unroll
        for (int i = 0; i < (NG + 7) / 8; ++i) {
          const uint4 u0 = lds128(s0 + 16 * i), u1 = lds128(s1 + 16 * i);
          const uint32_t x0[4] = {u0.x, u0.y, u0.z, u0.w}, x1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int k = 0; k < 8 && 8 * i + k < NG; ++k) {
            const float2 f0 = unpack_half2(x0[k / 2]), f1 = unpack_half2(x1[k / 2]);
            sg0[8 * i + k] = k % 2 ? f0.y : f0.x;
            sg1[8 * i + k] = k % 2 ? f1.y : f1.x;
          }
        }
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < G / 16; ++i) {
            const int s = gi * (G / 16) + i;
            uint32_t a0, a1, a2, a3;
            if constexpr (BITS == 4) {
              const uint32_t sel = t & 1 ? 0x4342u : 0x4140u;
              const uint32_t y0 = __byte_perm(lds32(k0 + 8 * s + 4 * (t >> 1)), 0u, sel);
              const uint32_t y1 = __byte_perm(lds32(k1 + 8 * s + 4 * (t >> 1)), 0u, sel);
              a0 = (y0 & 0x000F000Fu) ^ u_lo;
              a1 = (y1 & 0x000F000Fu) ^ u_lo;
              a2 = (y0 & 0x00F000F0u) ^ u_hi;
              a3 = (y1 & 0x00F000F0u) ^ u_hi;
            } else {
              const uint32_t y0 = lds32(k0 + 16 * s + 4 * t), y1 = lds32(k1 + 16 * s + 4 * t);
              a0 = (y0 & 0x00FF00FFu) ^ u_lo;
              a1 = (y1 & 0x00FF00FFu) ^ u_lo;
              a2 = ((y0 >> 8) & 0x00FF00FFu) ^ u_lo;
              a3 = ((y1 >> 8) & 0x00FF00FFu) ^ u_lo;
            }
            const uint2 qh = lds64(qf + s * 256);
            mma_f16(acc, a0, a1, a2, a3, qh.x, qh.y);
            if constexpr (EXACT) {
              const uint2 ql = lds64(qf + (S16 + s) * 256);
              mma_f16(acc, a0, a1, a2, a3, ql.x, ql.y);
            }
          }
          S[mt][0] = fmaf(sg0[gi], acc[0], S[mt][0]);
          S[mt][1] = fmaf(sg0[gi], acc[1], S[mt][1]);
          S[mt][2] = fmaf(sg1[gi], acc[2], S[mt][2]);
          S[mt][3] = fmaf(sg1[gi], acc[3], S[mt][3]);
        }
      }
      // scale, mask, running maximum (equal in the 8 lanes of a column)
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[mt][i] *= fs[i & 1];
      if (here != 0xffffffffu || __any_sync(0xffffffffu, tk + kTileChunk > min(lim[0], lim[1]))) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 16 * mt + 2 * g + (i >> 1);
            if (!((here >> tok) & 1u) || tk + tok >= lim[i & 1]) S[mt][i] = -INFINITY;
          }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i & 1] = fmaxf(mx[i & 1], S[mt][i]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
      }
      const bool g0 = mx[0] > m[0] + 8.0f || (m[0] == -INFINITY && mx[0] > -INFINITY);
      const bool g1 = mx[1] > m[1] + 8.0f || (m[1] == -INFINITY && mx[1] > -INFINITY);
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float al0 = !g0 ? 1.0f : m[0] == -INFINITY ? 0.0f : ex2(m[0] - mx[0]);
        const float al1 = !g1 ? 1.0f : m[1] == -INFINITY ? 0.0f : ex2(m[1] - mx[1]);
        l[0] *= al0;
        l[1] *= al1;
#pragma unroll
        for (int s = 0; s < S16; ++s) {
          O[s][0] *= al0;
          O[s][1] *= al1;
          O[s][2] *= al0;
          O[s][3] *= al1;
        }
        if (g0) m[0] = mx[0];
        if (g1) m[1] = mx[1];
      }
      // p' = 2^7 e^{x - m}; without any token yet the reference is 0 and p' = 0
      const float b0 = (m[0] == -INFINITY ? 0.0f : m[0]) - 7.0f;
      const float b1 = (m[1] == -INFINITY ? 0.0f : m[1]) - 7.0f;
      uint32_t ph[2][2], pl[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = ex2(S[mt][2 * r] - b0), p1 = ex2(S[mt][2 * r + 1] - b1);
          const uint32_t h = pack_half2(p0, p1);
          ph[mt][r] = movmatrix_trans(h);
          l[0] += p0;
          l[1] += p1;
          if constexpr (EXACT) pl[mt][r] = movmatrix_trans(half2_rest(p0, p1, h));
        }
      // values
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // scales of tokens 4t .. 4t + 3 of the tile as (4t, 4t + 2), (4t + 1, 4t + 3)
        uint32_t se[NG], so[NG];
        const uint32_t sv = st + L::kVS + (16 * mt + 4 * t) * L::SBS;
#pragma unroll
        for (int i = 0; i < (NG + 7) / 8; ++i) {
          const uint4 u0 = lds128(sv + 16 * i), u1 = lds128(sv + L::SBS + 16 * i);
          const uint4 u2 = lds128(sv + 2 * L::SBS + 16 * i), u3 = lds128(sv + 3 * L::SBS + 16 * i);
          const uint32_t x0[4] = {u0.x, u0.y, u0.z, u0.w}, x1[4] = {u1.x, u1.y, u1.z, u1.w};
          const uint32_t x2[4] = {u2.x, u2.y, u2.z, u2.w}, x3[4] = {u3.x, u3.y, u3.z, u3.w};
#pragma unroll
          for (int k = 0; k < 8 && 8 * i + k < NG; ++k) {
            se[8 * i + k] = __byte_perm(x0[k / 2], x2[k / 2], k % 2 ? 0x7632 : 0x5410);
            so[8 * i + k] = __byte_perm(x1[k / 2], x3[k / 2], k % 2 ? 0x7632 : 0x5410);
          }
        }
        const uint32_t vr = st + L::kV + (16 * mt + (lane & 15)) * L::RS;
        auto weigh = [&](int s, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          const uint32_t e0 = se[16 * s / G], o0 = so[16 * s / G];
          a0 = hmul2(a0, e0);
          a1 = hmul2(a1, e0);
          a2 = hmul2(a2, o0);
          a3 = hmul2(a3, o0);
          mma_f16(O[s], a0, a1, a2, a3, ph[mt][0], ph[mt][1]);
          if constexpr (EXACT) mma_f16(O[s], a0, a1, a2, a3, pl[mt][0], pl[mt][1]);
        };
        // fp16 1024 + u, or 1024 + 16 u, to c (exact)
        constexpr uint32_t k1 = 0x3C003C00u, k16 = 0x2C002C00u;   // 1, 2^-4
        // -1032, -72, -1152
        constexpr uint32_t o8 = 0xE408E408u, o72 = 0xD480D480u, o128 = 0xE480E480u;
        if constexpr (BITS == 4) {
#pragma unroll
          for (int s = 0; s < S16; s += 2) {
            uint32_t r[2];
            ldmatrix_bytes_trans(r[0], r[1], vr + 8 * s);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t y = r[i] >> 8;
              weigh(s + i, hfma2((r[i] & 0x000F000Fu) ^ h_lo, k1, o8),
                    hfma2((r[i] & 0x00F000F0u) ^ h_hi, k16, o72),
                    hfma2((y & 0x000F000Fu) ^ h_lo, k1, o8),
                    hfma2((y & 0x00F000F0u) ^ h_hi, k16, o72));
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < S16; ++s) {
            uint32_t r0, r1;
            ldmatrix_bytes_trans(r0, r1, vr + 16 * s);
            weigh(s, hfma2((r0 & 0x00FF00FFu) ^ h_lo, k1, o128),
                  hfma2((r1 & 0x00FF00FFu) ^ h_lo, k1, o128),
                  hfma2(((r0 >> 8) & 0x00FF00FFu) ^ h_lo, k1, o128),
                  hfma2(((r1 >> 8) & 0x00FF00FFu) ^ h_lo, k1, o128));
          }
        }
      }
      __syncwarp();   // every lane is done with the stage before it is refilled
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    // the warp's state over its stages: (m, l) and O[query][coord]
    float* wo = reinterpret_cast<float*>(ws);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    if (p.pre) {
      bad = __reduce_min_sync(0xffffffffu, bad);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (lim[c] > bad) l[c] = NAN;
    }
    if (g == 0) {
      ml_sh[warp][2 * t] = make_float2(m[0], l[0] * 0x1p-7f);
      ml_sh[warp][2 * t + 1] = make_float2(m[1], l[1] * 0x1p-7f);
    }
#pragma unroll
    for (int s = 0; s < S16; ++s) {
      constexpr float f = 0x1p-7f;
      if constexpr (BITS == 4) {   // rows g, g + 8: coordinates 2g, 2g + 1
        float* o = wo + 2 * t * D + 16 * s + 2 * g;
        *reinterpret_cast<float2*>(o) = make_float2(O[s][0] * f, O[s][2] * f);
        *reinterpret_cast<float2*>(o + D) = make_float2(O[s][1] * f, O[s][3] * f);
      } else {                     // coordinates g, g + 8
        float* o = wo + 2 * t * D + 16 * s + g;
        o[0] = O[s][0] * f;
        o[8] = O[s][2] * f;
        o[D] = O[s][1] * f;
        o[D + 8] = O[s][3] * f;
      }
    }
    if (threadIdx.x == 0) {
      next_sh = next;
      rec_sh = next_rec;
    }
    __syncthreads();
    it = int64_t(gridDim.x) + next_sh;
    rec = rec_sh;
    float* to_acc = p.pre ? a.pre_acc : a.own_acc;
    float2* to_ml = p.pre ? a.pre_ml : a.own_ml;
    for (int i = threadIdx.x; i < p.nr * (D / 4); i += NW * 32) {
      const int r = i / (D / 4), j = i % (D / 4);
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) mt = fmaxf(mt, ml_sh[w][r].x);
      float lt = 0.0f;
      float4 at = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 x = ml_sh[w][r];
        const float f = x.x == -INFINITY ? 0.0f : ex2(x.x - mt);
        const float4 v = reinterpret_cast<const float4*>(smem + w * L::kWarp)[r * (D / 4) + j];
        lt = fmaf(f, x.y, lt);
        at = make_float4(fmaf(f, v.x, at.x), fmaf(f, v.y, at.y), fmaf(f, v.z, at.z),
                         fmaf(f, v.w, at.w));
      }
      if (!a.dbg_part(p.pre, p.part + r)) continue;
      reinterpret_cast<float4*>(to_acc + (p.part + r) * D)[j] = at;
      if (j == 0) to_ml[p.part + r] = make_float2(mt, lt);
    }
    __syncthreads();   // the partial sums are read before the next item's copies land there
  }
}

// A query head whose sums are not finite, by a warp: either its query or a scale is
// not, and NaN is the answer; or a scale is larger than the parts' fp16 holds
// (kLargeScale), and the head is done anew, in float32. (Neither function is inlined,
// the arguments stay in the constant bank and the join's blocks per SM are stated, so
// that its own path keeps its registers: with a stack frame, or with all warps of the
// join in here, a call of the attention took 1 to 5 us more.)
template <int NW>
__device__ __forceinline__ int64_t merged_row() {
  return NW == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5) : int64_t(blockIdx.x);
}
template <int D, int NW>
__device__ __noinline__ bool row_is_finite(const PrefixArgs& a) {
  const int64_t v = merged_row<NW>();
  const int hq = a.heads * a.q_per_kv, b = int(v / hq), h = int(v % hq) / a.q_per_kv;
  const int lane = threadIdx.x & 31, ng = D >> a.lg_group, len = a.len(b);
  bool ok = true;
  for (int k = lane; k < D; k += 32) ok = ok && fabsf(a.qrot[v * D + k]) < INFINITY;
  // the scales, a token to a lane (positions below 2^31 - 65536)
  for (int t = lane; __all_sync(0xffffffffu, ok) && t - lane < len; t += 32) {
    const int32_t* table = t < a.prefix_len ? a.prefix_table : a.block_table + int64_t(b) * a.max_pages;
    const int64_t row = t < len ? a.pool_row(t < a.prefix_len, table, uint32_t(t)) : -1;
    if (row < 0) continue;
    const int64_t at = (row * a.heads + h) * ng;
    if (ng >= 8) {
      for (int i = 0; i < ng; i += 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(a.k_scales + at + i);
        const uint4 y = *reinterpret_cast<const uint4*>(a.v_scales + at + i);
        ok = ok && !(nonfinite_halves(x.x) | nonfinite_halves(x.y) | nonfinite_halves(x.z) |
                     nonfinite_halves(x.w) | nonfinite_halves(y.x) | nonfinite_halves(y.y) |
                     nonfinite_halves(y.z) | nonfinite_halves(y.w));
      }
    } else {
      for (int i = 0; i < ng; ++i)
        ok = ok && !nonfinite_halves(a.k_scales[at + i] | uint32_t(a.v_scales[at + i]) << 16);
    }
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

// Codes of coordinates 2k and 2k + 1 of vector vec, times their scale.
template <int D>
__device__ __forceinline__ float2 decoded_pair(const PrefixArgs& a, const uint8_t* codes,
                                               const uint16_t* scales, int64_t vec, int k) {
  const float f = __half2float(
      __ushort_as_half(scales[vec * (D >> a.lg_group) + ((2 * k) >> a.lg_group)]));
  int c0, c1;
  if (a.bits == 4) {
    const int w = codes[vec * (D / 2) + k];
    c0 = (w & 15) - ((w & 8) << 1);
    c1 = (w >> 4) - ((w & 128) >> 3);
  } else {
    const int8_t* p = reinterpret_cast<const int8_t*>(codes) + vec * D + 2 * k;
    c0 = p[0];
    c1 = p[1];
  }
  return make_float2(f * float(c0), f * float(c1));
}

template <int E>
struct RowState {
  float m, l;
  float2 acc[E];   // the pairs warp_pair(lane, e)
};
template <int ROT, int D, int NW>
__device__ __noinline__ RowState<D / 64> attend_float32(const PrefixArgs& a) {
  constexpr int E = D / 64;
  const int64_t v = merged_row<NW>();
  const int hq = a.heads * a.q_per_kv, b = int(v / hq), h = int(v % hq) / a.q_per_kv;
  const int lane = threadIdx.x & 31, len = a.len(b);
  RowState<E> s;
  s.m = -INFINITY;
  s.l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) s.acc[e] = make_float2(0.0f, 0.0f);
#pragma unroll 1
  for (int t = 0; t < len; ++t) {
    const int32_t* table = t < a.prefix_len ? a.prefix_table : a.block_table + int64_t(b) * a.max_pages;
    const int64_t row = a.pool_row(t < a.prefix_len, table, uint32_t(t));
    if (row < 0) continue;
    const int64_t vec = row * a.heads + h;
    float x = 0.0f;
    float2 y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = warp_pair<ROT, D>(lane, e);
      const float2 z = reinterpret_cast<const float2*>(a.qrot + v * D)[k];
      const float2 c = decoded_pair<D>(a, a.k_codes, a.k_scales, vec, k);
      x = fmaf(z.x, c.x, fmaf(z.y, c.y, x));
      y[e] = decoded_pair<D>(a, a.v_codes, a.v_scales, vec, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const float top = fmaxf(s.m, x), f = exp2f(s.m - top), p = exp2f(x - top);
    s.m = top;
    s.l = fmaf(s.l, f, p);
#pragma unroll
    for (int e = 0; e < E; ++e)
      s.acc[e] = make_float2(fmaf(s.acc[e].x, f, p * y[e].x), fmaf(s.acc[e].y, f, p * y[e].y));
  }
  return s;
}

// NW warps per query head, four heads to a block of the one-warp form. The parts'
// (m, l) by all lanes, then their weighted sums, a warp a part in turn, added over
// the warps in order; the rotation by the first warp.
template <int ROT, int D, int NW>
__global__ void __launch_bounds__(NW == 1 ? 128 : NW * 32,
                                  NW == 1 && D == 256 ? 5 : NW == 16 ? 2 : 8)
    prefix_merge_kernel(const __grid_constant__ PrefixArgs a) {
  constexpr int E = D / 64;
  __shared__ float acc_sh[NW][D];
  __shared__ float2 ml_sh[NW];
  __shared__ __align__(16) float end_sh[NW == 1 ? 4 : D + D / 4];   // lambda, signs
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : int(threadIdx.x >> 5);
  const int g = a.q_per_kv, hq = a.heads * g;
  const int64_t v = merged_row<NW>();
  if (NW == 1 && v >= int64_t(a.n_seq) * hq) return;
  if (!a.dbg_query(v)) return;   // the same in a block
  const int b = int(v / hq), h = int(v % hq) / g, j = int(v % hq) % g;
  const int64_t M = int64_t(a.n_seq) * g;
  if constexpr (NW > 1) {
    const int i = int(threadIdx.x);
    if (i < D / 4) copy16(smem_addr(end_sh + 4 * i), a.v_lambda + int64_t(h) * D + 4 * i, true);
    else if (i < D / 4 + D / 16)
      copy16(smem_addr(end_sh + D + 4 * (i - D / 4)),
             a.v_signs + int64_t(h) * D + 16 * (i - D / 4), true);
  }
  const int n_pre = a.prefix_len > 0 && a.len(b) > 0 ? a.prefix_splits : 0;
  const int c0 = a.chunk_start[b], n = n_pre + a.chunk_start[b + 1] - c0;
  // parts 0 .. n_pre - 1 of the prefix, then the sequence's own
  auto row_of = [&](int i) {
    return i < n_pre ? (int64_t(i) * a.heads + h) * M + int64_t(b) * g + j
                     : (int64_t(c0 + i - n_pre) * a.heads + h) * g + j;
  };
  auto ml_of = [&](int i) {
    return a.dbg_part(i < n_pre, row_of(i)) ? (i < n_pre ? a.pre_ml : a.own_ml)[row_of(i)]
                                            : make_float2(-INFINITY, 0.0f);
  };
  // a part without tokens has l = 0 (a NaN goes on)
  float m = -INFINITY;
  for (int i = NW == 1 ? lane : int(threadIdx.x); i < n; i += NW * 32) m = fmaxf(m, ml_of(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (NW > 1) {
    if (lane == 0) ml_sh[warp].x = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, ml_sh[w].x);
  }
  const float ref = m == -INFINITY ? 0.0f : m;

  float l = 0.0f;
  float2 acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float2(0.0f, 0.0f);
  // the one-warp form loads the pairs that its lanes rotate, the others pass
  // them through shared memory
  int at[E];
#pragma unroll
  for (int e = 0; e < E; ++e) at[e] = NW == 1 ? warp_pair<ROT, D>(lane, e) : lane + 32 * e;
#pragma unroll 4
  for (int i = warp; i < n; i += NW) {
    const int64_t r = row_of(i);
    if (!a.dbg_part(i < n_pre, r)) continue;
    const float2 ml = (i < n_pre ? a.pre_ml : a.own_ml)[r];
    const float2* src = reinterpret_cast<const float2*>((i < n_pre ? a.pre_acc : a.own_acc) + r * D);
    float2 x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = src[at[e]];
    if (ml.y > 0.0f || ml.y != ml.y) {
      const float c = exp2f(ml.x - ref);
      l = fmaf(ml.y, c, l);
#pragma unroll
      for (int e = 0; e < E; ++e)
        acc[e] = make_float2(fmaf(x[e].x, c, acc[e].x), fmaf(x[e].y, c, acc[e].y));
    }
  }
  if constexpr (NW > 1) {
    if (lane == 0) ml_sh[warp].y = l;
#pragma unroll
    for (int e = 0; e < E; ++e) reinterpret_cast<float2*>(acc_sh[warp])[lane + 32 * e] = acc[e];
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (warp > 0) return;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) l += ml_sh[w].y;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc[e] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 x = reinterpret_cast<const float2*>(acc_sh[w])[warp_pair<ROT, D>(lane, e)];
        acc[e] = make_float2(acc[e].x + x.x, acc[e].y + x.y);
      }
    }
  }
  // lambda and signs: on their way before the calls below, which nothing is moved
  // across; from shared memory they need no registers over them
  float2 lam[E];
  int8_t sg[2 * E];
  if constexpr (NW == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      lam[e] = reinterpret_cast<const float2*>(a.v_lambda + int64_t(h) * D)[warp_pair<ROT, D>(lane, e)];
      sg[2 * e] = a.v_signs[int64_t(h) * D + 2 * (E * lane + e)];
      sg[2 * e + 1] = a.v_signs[int64_t(h) * D + 2 * (E * lane + e) + 1];
    }
  }
  bool finite = fabsf(l) < INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e)
    finite = finite && fabsf(acc[e].x) < INFINITY && fabsf(acc[e].y) < INFINITY;
  if (!__all_sync(0xffffffffu, finite)) {
    l = NAN;
    if (row_is_finite<D, NW>(a)) {
      const RowState<E> s = attend_float32<ROT, D, NW>(a);
      m = s.m;
      l = s.l;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = s.acc[e];
    }
  }
  if constexpr (NW > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      lam[e] = reinterpret_cast<const float2*>(end_sh)[warp_pair<ROT, D>(lane, e)];
      sg[2 * e] = reinterpret_cast<const int8_t*>(end_sh + D)[2 * (E * lane + e)];
      sg[2 * e + 1] = reinterpret_cast<const int8_t*>(end_sh + D)[2 * (E * lane + e) + 1];
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : l;   // no token: 0 (a NaN stays)
#pragma unroll
  for (int e = 0; e < E; ++e)
    acc[e] = make_float2(acc[e].x * inv * lam[e].x, acc[e].y * inv * lam[e].y);
  warp_rotate_inverse<ROT, D>(acc, lane);
  uint32_t* o = reinterpret_cast<uint32_t*>(a.out) + v * (D / 2) + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float x0 = sg[2 * e] < 0 ? -acc[e].x : acc[e].x;
    const float x1 = sg[2 * e + 1] < 0 ? -acc[e].y : acc[e].y;
    if (a.bf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x0, x1);
      o[e] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(x0, x1);
      o[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  if (a.lse && lane == 0) a.lse[v] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace srftq
