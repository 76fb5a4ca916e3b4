// Launcher of the shared-prefix attention over a paged cache (paged_attention.cuh).
#include <climits>

#include "launch_impl.cuh"
#include "launch_prefix_tiles.cuh"

namespace srftq {

// Which kernel takes the prefix. The tcgen05 kernels compute 128 query rows per
// KV head whatever their number, the warp-level one 8 at a time, so its time per
// token grows with the rows and breaks even at kEvenRows of each 128; a launch
// more, the query tiles and a block's start cost the others 5 us, which the rows
// beyond must win back over all tokens and heads. Both fit int4 with 8 heads of d =
// 128 and 4 of 256; elsewhere the rule is off by up to a fifth next to its border,
// for int8 at d = 256 by a third. One B200, fp16 / bf16, us a call, warp-level
// against tcgen05 (* where the rule takes the slower one). int4:
//   28672 tokens, 8 heads of d = 128: 16 rows 49 : 55 / 44 : 46, 24 rows 63 : 55 /
//     53 : 46, 32 rows 75 : 55 / 65 : 45, 64 rows 126 : 59 / 110 : 49;
//   28672 tokens, 4 heads of d = 256: 24 rows 69 : 104 / 61 : 69, 32 rows 83 : 103 /
//     73 : 68, 48 rows 108 : 104 / 92 : 69;
//   6000 tokens, d = 128: 24 rows 32 : 36 / 29 : 32, 32 rows 36 : 36 / 33 : 31;
//   1024 tokens, d = 128: 32 rows 25 : 30 / 25 : 28, 48 rows 27 : 31 / 26 : 29;
//   28672 tokens, 8 heads of d = 64: 16 rows 35 : 45 / 33 : 38, 24 rows 45 : 45 /
//     41 : 38, 32 rows 54 : 45 / 49 : 37; 6000 tokens: 32 rows 25 : 29 / 23 : 25,
//     48 rows 29 : 31* / 27 : 29*, 64 rows 33 : 31 / 31 : 29;
//   28672 tokens, 2 heads of d = 128: 24 rows 31 : 38 / 29 : 33, 32 rows 33 : 38* /
//     31 : 33*, 48 rows 39 : 39 / 35 : 35, 64 rows 45 : 39 / 40 : 35; 1 head: 48 rows
//     31 : 37* / 29 : 33*, 64 rows 33 : 38* / 29 : 34*, 96 rows 38 : 39 / 35 : 35;
//   120000 tokens, 2 heads of d = 128: 16 rows 47 : 58 / 43 : 48, 24 rows 62 : 60 /
//     54 : 50, 32 rows 72 : 59 / 64 : 49;
//   28672 tokens, 1 head of d = 256: 64 rows 57 : 66 / 51 : 50, 96 rows 65 : 68* /
//     58 : 51.
// int8:
//   28672 tokens, 8 heads of d = 128: 16 rows 58 : 60 / 50 : 47*, 24 rows 74 : 62 /
//     63 : 48; 4096 tokens: 32 rows 30 : 33 / 28 : 29, 48 rows 38 : 35 / 35 : 33;
//   28672 tokens, 2 heads of d = 128: 24 rows 37 : 39 / 33 : 33, 32 rows 41 : 39 /
//     37 : 33;
//   28672 tokens, 4 heads of d = 256: 24 rows 96 : 108 / 85 : 78*, 32 rows 119 : 110* /
//     102 : 78*, 48 rows 160 : 118* / 134 : 83, 64 rows 197 : 116 / 165 : 85.
constexpr int64_t kMmaGain = 3 << 18;   // (rows beyond) x tokens x heads
constexpr int64_t even_rows(int32_t d, bool exact) { return d <= 128 ? 16 : exact ? 46 : 30; }

extern template int launch_prefix_tiles<64>(const PrefixArgs&, int, int, cudaStream_t);
extern template int launch_prefix_tiles<128>(const PrefixArgs&, int, int, cudaStream_t);
extern template int launch_prefix_tiles<256>(const PrefixArgs&, int, int, cudaStream_t);

namespace {

// Sizes of a call that the caller's workspace and the launches follow from:
// host values only, none of them dependent on the sequences' lengths.
struct PrefixShape {
  bool mma, shared;   // parts by tcgen05; its two units different rows, not alternate tokens
  int32_t splits, per, chunk_goal;
  int64_t q_off, image_off, factor_off, plan_off, start_off, chunk_off;
  int64_t pre_ml_off, pre_acc_off, own_ml_off, own_acc_off, bytes;
};

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

PrefixShape prefix_shape(int32_t d, int32_t heads, int64_t n_seq, int32_t g, int64_t prefix_len,
                         bool exact, int sms) {
  PrefixShape s{};
  const int64_t rows = n_seq * g;
  const int64_t even = (rows + kMmaRows - 1) / kMmaRows * even_rows(d, exact);
  s.mma = rows > even && prefix_len > kMmaGain / (rows - even) / heads;
  if (prefix_len > 0) {
    // blocks of one wave, their row tiles, and what a block's start and end and
    // a part's join cost in tokens; the number of parts with the least time on
    // those terms
    s.shared = s.mma && d <= 128 && !exact && rows > kMmaRows;
    const bool pair = s.mma && d <= 128 && !s.shared;   // a block makes two parts
    const int64_t slots = s.mma ? sms : 4 * int64_t(sms);
    const int64_t tile = s.shared ? 2 * kMmaRows : s.mma ? kMmaRows : kPrefixRows;
    const int64_t units = (rows + tile - 1) / tile * heads;
    const int64_t over = s.mma ? 512 : 128;
    const int64_t join = (4 + rows * heads * d / 10000) * (pair ? 2 : 1);
    int64_t best = 0, best_n = 1;
    const int64_t most = (prefix_len + 63) / 64;
    for (int64_t n = 1; n <= most && units * n <= 4 * slots + units; n += n / 16 + 1) {
      const int64_t per = ((prefix_len + n - 1) / n + 63) / 64 * 64;
      const int64_t cost = (units * n + slots - 1) / slots * (per + over) + n * join;
      if (best == 0 || cost < best) {
        best = cost;
        best_n = n;
      }
    }
    const int64_t per = ((prefix_len + best_n - 1) / best_n + 63) / 64 * 64;
    s.per = int32_t(per);
    s.splits = int32_t((prefix_len + per - 1) / per) * (pair ? 2 : 1);
  }
  s.chunk_goal = int32_t((8 * int64_t(sms) + heads - 1) / heads);
  const int64_t chunks = s.chunk_goal + n_seq;
  int64_t o = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = o;
    o += up16(bytes);
    return at;
  };
  s.q_off = take(n_seq * heads * g * d * 4);
  const int64_t padded = s.mma ? (rows + kMmaRows - 1) / kMmaRows * kMmaRows * heads : 0;
  s.image_off = take(padded * d * 2 * (exact ? 2 : 1));
  s.factor_off = take(padded * 4);
  s.plan_off = take(sizeof(PrefixPlan));
  s.start_off = take((n_seq + 1) * 4);
  s.chunk_off = take(chunks * 16);
  s.pre_ml_off = take(s.splits * heads * rows * 8);
  s.pre_acc_off = take(s.splits * heads * rows * d * 4);
  s.own_ml_off = take(chunks * heads * g * 8);
  s.own_acc_off = take(chunks * heads * g * d * 4);
  s.bytes = o;
  return s;
}

}  // namespace

int64_t prefix_attention_workspace(int32_t d, int32_t heads, int64_t n_seq, int32_t q_per_kv,
                                   int64_t prefix_len) {
  const int sms = Runtime::num_sms();
  const int64_t x = prefix_shape(d, heads, n_seq, q_per_kv, prefix_len, false, sms).bytes;
  const int64_t y = prefix_shape(d, heads, n_seq, q_per_kv, prefix_len, true, sms).bytes;
  return x > y ? x : y;
}

int launch_prefix_attention(const PrefixAttnCall& c) {
  const int sms = Runtime::num_sms();
  const PrefixShape s =
      prefix_shape(c.d, c.heads, c.n_seq, c.q_per_kv, c.prefix_len, !c.bf16, sms);
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  PrefixArgs a{};
  a.n_seq = int32_t(c.n_seq);
  a.heads = c.heads;
  a.q_per_kv = c.q_per_kv;
  a.lg_group = ilog2(c.group);
  a.prefix_len = int32_t(c.prefix_len);
  a.max_pages = int32_t(c.max_pages);
  a.pre_mma = s.mma;
  a.pre_shared = s.shared;
  a.prefix_splits = s.splits;
  a.prefix_per = s.per;
  a.chunk_goal = s.chunk_goal;
  a.map = PageMap{FastDiv::make(uint32_t(c.page_size)), int32_t(c.n_pages)};
  a.q = c.q;
  a.bf16 = c.bf16;
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.k_signs = c.k_signs;
  a.k_lambda = c.k_lambda;
  a.v_codes = c.v_codes;
  a.v_scales = c.v_scales;
  a.v_signs = c.v_signs;
  a.v_lambda = c.v_lambda;
  a.prefix_table = c.prefix_table;
  a.block_table = c.block_table;
  a.seq_lens = c.seq_lens;
  a.scale = c.scale;
  a.out = c.out;
  a.lse = c.lse;
  a.bits = c.bits;
  a.qrot = reinterpret_cast<float*>(ws + s.q_off);
  a.q_image = ws + s.image_off;
  a.q_factor = reinterpret_cast<float*>(ws + s.factor_off);
  a.plan = reinterpret_cast<PrefixPlan*>(ws + s.plan_off);
  a.chunk_start = reinterpret_cast<int32_t*>(ws + s.start_off);
  a.chunk_of = reinterpret_cast<int4*>(ws + s.chunk_off);
  a.pre_ml = reinterpret_cast<float2*>(ws + s.pre_ml_off);
  a.pre_acc = reinterpret_cast<float*>(ws + s.pre_acc_off);
  a.own_ml = reinterpret_cast<float2*>(ws + s.own_ml_off);
  a.own_acc = reinterpret_cast<float*>(ws + s.own_acc_off);
  a.guard = Runtime::guard_word();
  if (!a.guard) return SRFTQ_ERR_CUDA;
  const int64_t queries = c.n_seq * c.heads * c.q_per_kv;   // below 2^31 (check_prefix_sizes)
  const int64_t blocks = (queries + 7) / 8;                 // a warp per query
  int rc = SRFTQ_ERR_UNSUPPORTED;
  static_for<6, 9>([&](auto lg_) {
    constexpr int D = 1 << decltype(lg_)::value;
    if (c.d != D) return;
    const int g1 = int(blocks < 8 * sms ? blocks : 8 * sms);
    if (c.rotation == kSRFT) prefix_prepare_kernel<kSRFT, D><<<g1, 256, 0, c.stream>>>(a);
    else prefix_prepare_kernel<kSRHT, D><<<g1, 256, 0, c.stream>>>(a);
    rc = launch_prefix_tiles<D>(a, c.bits, c.group, c.stream);
    if (rc != SRFTQ_OK) return;
    // few query heads: more warps each, since then a block's own time counts;
    // very many: a warp each, for the blocks' barriers cost more than they save
    static_for<0, 3>([&](auto w_) {
      constexpr int NW = decltype(w_)::value == 0 ? 1 : decltype(w_)::value == 1 ? 4 : 16;
      if ((queries <= 2 * sms ? 16 : queries <= 16 * sms ? 4 : 1) != NW) return;
      const int grid = int(NW == 1 ? (queries + 3) / 4 : queries), threads = NW == 1 ? 128 : 32 * NW;
      rc = c.rotation == kSRFT
               ? launch_after<prefix_merge_kernel<kSRFT, D, NW>>(grid, threads, 0, c.stream, a)
               : launch_after<prefix_merge_kernel<kSRHT, D, NW>>(grid, threads, 0, c.stream, a);
    });
    if (rc != SRFTQ_OK) return;
    rc = finish_launch();
  });
  return rc;
}

}  // namespace srftq
