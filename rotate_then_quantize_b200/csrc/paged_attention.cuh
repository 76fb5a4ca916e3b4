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
// Three launches on the caller's stream:
//   prefix_prepare_kernel   a warp per query: lambda_K * R_K (s_K q) * scale *
//                           log2 e into the workspace; block 0 also plans the
//                           split of the sequences' own tokens;
//   prefix_partial_kernel   the parts, each (m, l, a) into the workspace;
//   prefix_merge_kernel     a warp per query head: joins its parts, applies
//                           lambda_V / l, R_V^T and s_V, rounds once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pages.cuh"
#include "ptx.cuh"
#include "warp_rotate.cuh"

namespace srftq {

constexpr int kPrefixRows = 8;        // query rows of one item
constexpr int kPrefixWarps = 4;       // warps of a block, each with its own online softmax
constexpr int kPrefixMaxG = 16;       // query heads per KV head
constexpr float kLog2e = 1.4426950408889634f;

// Plan of the own tokens, in the workspace: header, then start[n_seq + 1], the
// first chunk of every sequence (chunk c of sequence b covers the own tokens
// [c chunk, (c + 1) chunk)).
struct PrefixPlan {
  int32_t chunk;      // tokens per chunk, a multiple of 64
  int32_t n_chunks;   // chunks of all sequences
  int32_t pad[2];
};

struct PrefixArgs {
  int32_t n_seq, heads, q_per_kv, lg_group;
  int32_t prefix_len, max_pages, max_chunks;
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
  float* qrot;                         // workspace: rotated queries
  PrefixPlan* plan;
  int32_t* chunk_start;
  float2* pre_ml;                      // [splits][heads][n_seq q_per_kv]
  float* pre_acc;                      // the same rows of d
  float2* own_ml;                      // [chunks][heads][q_per_kv]
  float* own_acc;

  // tokens of sequence b: all, those of its own
  __device__ __forceinline__ int32_t len(int b) const {
    const int64_t cap = int64_t(max_pages) * map.page.d;
    const int64_t most = cap > prefix_len ? cap : prefix_len;
    const int32_t n = seq_lens[b];
    return n < 0 ? 0 : n > most ? int32_t(most) : n;
  }
  __device__ __forceinline__ int32_t own(int b) const { return max(len(b) - prefix_len, 0); }
};

__device__ __forceinline__ float lo_f32(uint32_t w, bool bf16) {
  return bf16 ? __uint_as_float(w << 16) : __half2float(__ushort_as_half(uint16_t(w)));
}
__device__ __forceinline__ float hi_f32(uint32_t w, bool bf16) {
  return bf16 ? __uint_as_float(w & 0xFFFF0000u) : __half2float(__ushort_as_half(uint16_t(w >> 16)));
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
  // chunks of at least 64 tokens, few enough that sum ceil(own / chunk) <= goal + n_seq
  const int64_t per = (total + a.chunk_goal - 1) / a.chunk_goal;
  const int32_t chunk = int32_t(per <= 64 ? 64 : (per + 63) / 64 * 64);
  int32_t carry = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += nt) {
    const int b = b0 + tid;
    const int32_t n = b < a.n_seq ? (a.own(b) + chunk - 1) / chunk : 0;
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
  if (tid == 0) {
    a.chunk_start[a.n_seq] = carry;
    a.plan->chunk = chunk;
    a.plan->n_chunks = carry;
  }
}

template <int ROT, int D>
__global__ void __launch_bounds__(256) prefix_prepare_kernel(const PrefixArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 31;
  const int hq = a.heads * a.q_per_kv;
  const int64_t total = int64_t(a.n_seq) * hq;
  const float f = a.scale * kLog2e;
  for (int64_t v = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; v < total;
       v += (int64_t(gridDim.x) * blockDim.x) >> 5) {
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
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = warp_pair<ROT, D>(lane, e);
      const float2 l = lam[k];
      o[k] = make_float2(z[e].x * l.x * f, z[e].y * l.y * f);
    }
  }
  if (blockIdx.x == 0) plan_own_tokens(a);
}

// sigma * code of this lane's EP consecutive coordinates of a pool row.
template <int D, int BITS>
__device__ __forceinline__ void lane_values(const uint8_t* codes, float sigma, int lane,
                                            float (&v)[D / 32]) {
  constexpr int EP = D / 32, NB = EP * BITS / 8;
  const int8_t* p = reinterpret_cast<const int8_t*>(codes) + lane * NB;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int c = p[i];
    if constexpr (BITS == 8) {
      v[i] = sigma * float(c);
    } else {
      v[2 * i] = sigma * float((c << 28) >> 28);
      v[2 * i + 1] = sigma * float(c >> 4);
    }
  }
}

// One item: rows (query rows) x tokens [t0, t1) of one head, by a block.
template <int D, int BITS>
__global__ void __launch_bounds__(kPrefixWarps * 32) prefix_partial_kernel(const PrefixArgs a) {
  constexpr int EP = D / 32, CB = D * BITS / 8, R = kPrefixRows, NW = kPrefixWarps;
  __shared__ float acc_sh[NW][R][D];
  __shared__ float2 ml_sh[NW][R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = a.q_per_kv, hq = a.heads * g;
  const int M = a.n_seq * g;                             // query rows of a head
  const int pre_tiles = a.prefix_len > 0 ? (M + R - 1) / R : 0;
  const int64_t n_pre = int64_t(a.prefix_splits) * a.heads * pre_tiles;
  const int own_tiles = (g + R - 1) / R;
  const int64_t n_own = int64_t(a.plan->n_chunks) * a.heads * own_tiles;
  const int NG = D >> a.lg_group;
  for (int64_t it = blockIdx.x; it < n_pre + n_own; it += gridDim.x) {
    const bool pre = it < n_pre;
    int h, r0, nr, t0, t1, b = 0;
    int64_t part;                // index of the part's first row
    const int32_t* table;
    if (pre) {
      const int rt = int(it % pre_tiles);
      const int64_t q = it / pre_tiles;
      h = int(q % a.heads);
      const int s = int(q / a.heads);
      r0 = rt * R;
      nr = min(R, M - r0);
      t0 = s * a.prefix_per;
      t1 = min(t0 + a.prefix_per, a.prefix_len);
      part = (int64_t(s) * a.heads + h) * M + r0;
      table = a.prefix_table;
    } else {
      const int64_t i = it - n_pre;
      const int rt = int(i % own_tiles);
      const int64_t q = i / own_tiles;
      h = int(q % a.heads);
      const int c = int(q / a.heads);
      int lo = 0, hi = a.n_seq;   // the sequence of chunk c: last start <= c
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.chunk_start[mid] <= c) lo = mid; else hi = mid;
      }
      b = lo;
      r0 = rt * R;
      nr = min(R, g - r0);
      t0 = a.prefix_len + (c - a.chunk_start[b]) * a.plan->chunk;
      t1 = min(t0 + a.plan->chunk, a.len(b));
      part = (int64_t(c) * a.heads + h) * g + r0;
      table = a.block_table + int64_t(b) * a.max_pages;
    }
    float q[R][EP], acc[R][EP], m[R], l[R];
    int lim[R];                  // tokens that the row sees
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int rr = r0 + min(r, nr - 1);
      const int bb = pre ? rr / g : b;
      const int64_t v = int64_t(bb) * hq + h * g + (pre ? rr % g : rr);
      lim[r] = a.len(bb);
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        q[r][e] = a.qrot[v * D + lane * EP + e];
        acc[r][e] = 0.0f;
      }
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
    for (int t = t0 + warp; t < t1; t += NW) {
      const int64_t row = a.map.row(table, uint32_t(t));
      if (row < 0) continue;     // no page: the token is not there
      const int64_t vec = row * a.heads + h;
      const int gi = (lane * EP) >> a.lg_group;
      float kv[EP], vv[EP];
      lane_values<D, BITS>(a.k_codes + vec * CB, __half2float(__ushort_as_half(a.k_scales[vec * NG + gi])),
                           lane, kv);
      lane_values<D, BITS>(a.v_codes + vec * CB, __half2float(__ushort_as_half(a.v_scales[vec * NG + gi])),
                           lane, vv);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < EP; ++e) s = fmaf(q[r][e], kv[e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (t < lim[r]) {
          const float mn = fmaxf(m[r], s);
          const float al = exp2f(m[r] - mn), p = exp2f(s - mn);
          m[r] = mn;
          l[r] = fmaf(l[r], al, p);
#pragma unroll
          for (int e = 0; e < EP; ++e) acc[r][e] = fmaf(acc[r][e], al, p * vv[e]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < EP; ++e) acc_sh[warp][r][lane * EP + e] = acc[r][e];
      if (lane == 0) ml_sh[warp][r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nr * D; i += NW * 32) {
      const int r = i / D, j = i % D;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) mt = fmaxf(mt, ml_sh[w][r].x);
      float lt = 0.0f, at = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float mw = ml_sh[w][r].x;
        const float c = mw == -INFINITY ? 0.0f : exp2f(mw - mt);
        lt = fmaf(c, ml_sh[w][r].y, lt);
        at = fmaf(c, acc_sh[w][r][j], at);
      }
      (pre ? a.pre_acc : a.own_acc)[(part + r) * D + j] = at;
      if (j == 0) (pre ? a.pre_ml : a.own_ml)[part + r] = make_float2(mt, lt);
    }
    __syncthreads();
  }
}

template <int ROT, int D>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const PrefixArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 31;
  const int g = a.q_per_kv, hq = a.heads * g;
  const int64_t total = int64_t(a.n_seq) * hq;
  const int64_t v = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (v >= total) return;
  const int b = int(v / hq), h = int(v % hq) / g, j = int(v % hq) % g;
  const int64_t M = int64_t(a.n_seq) * g;
  float m = -INFINITY, l = 0.0f;
  float2 acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float2(0.0f, 0.0f);
  auto join = [&](float2 ml, const float* src) {
    if (!(ml.y > 0.0f || ml.y != ml.y)) return;   // a part without tokens (a NaN goes on)
    const float mn = fmaxf(m, ml.x);
    const float c0 = m == -INFINITY ? 0.0f : exp2f(m - mn), c1 = exp2f(ml.x - mn);
    m = mn;
    l = l * c0 + ml.y * c1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 x = reinterpret_cast<const float2*>(src)[warp_pair<ROT, D>(lane, e)];
      acc[e] = make_float2(acc[e].x * c0 + x.x * c1, acc[e].y * c0 + x.y * c1);
    }
  };
  if (a.len(b) > 0 && a.prefix_len > 0) {
    for (int s = 0; s < a.prefix_splits; ++s) {
      const int64_t i = (int64_t(s) * a.heads + h) * M + int64_t(b) * g + j;
      join(a.pre_ml[i], a.pre_acc + i * D);
    }
  }
  for (int c = a.chunk_start[b]; c < a.chunk_start[b + 1]; ++c) {
    const int64_t i = (int64_t(c) * a.heads + h) * g + j;
    join(a.own_ml[i], a.own_acc + i * D);
  }
  const float inv = l > 0.0f ? 1.0f / l : l;   // no token: 0 (a NaN stays)
  const float2* lam = reinterpret_cast<const float2*>(a.v_lambda + int64_t(h) * D);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float2 f = lam[warp_pair<ROT, D>(lane, e)];
    acc[e] = make_float2(acc[e].x * inv * f.x, acc[e].y * inv * f.y);
  }
  warp_rotate_inverse<ROT, D>(acc, lane);
  const int8_t* sg = a.v_signs + int64_t(h) * D + 2 * E * lane;
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
