// Launchers of the paged codec: the kernels of codec.cuh (d <= 128) and
// codec_split.cuh (d = 256) with their pool side addressed by slots. Each head
// dimension is compiled in its own unit (launch_paged_d*.cu).
#pragma once

#include "launch_split.cuh"

namespace srftq {

// Tensor map of the contiguous fp16 side: boxes of HPT heads x RPT rows.
template <int D>
int encode_rows(CUtensorMap* tm, const uint16_t* base, int64_t H, int64_t N, int64_t Sl,
                int64_t slice_stride_rows, const TileGeom& g) {
  constexpr int XB = 2 * D, span = XB < 128 ? XB : 128;
  const uint64_t dims[4] = {uint64_t(D), uint64_t(H), uint64_t(N), uint64_t(Sl)};
  const uint64_t str[3] = {uint64_t(XB), uint64_t(H) * XB, uint64_t(slice_stride_rows) * H * XB};
  const uint32_t box[4] = {uint32_t(span / 2), 1u << g.hpt_log2,
                           uint32_t(kTileRows) >> g.hpt_log2, 1u};
  return Runtime::encode_4d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, const_cast<uint16_t*>(base), dims,
                            str, box, swizzle_mode(span));
}

// Calls f(Int<BITS>, Int<G>, Int<ROT>) for groups of 16 .. D coordinates.
template <int D, typename F>
int dispatch_paged(int bits, int group, int rot, F&& f) {
  int rc = SRFTQ_ERR_UNSUPPORTED;
  static_for<0, 2>([&](auto b_) {
    constexpr int BITS = decltype(b_)::value == 0 ? 4 : 8;
    static_for<4, ilog2(D) + 1>([&](auto lg_) {
      constexpr int G = 1 << decltype(lg_)::value;
      static_for<0, 2>([&](auto r_) {
        constexpr int ROT = decltype(r_)::value;
        if (bits == BITS && group == G && rot == ROT) rc = f(Int<BITS>{}, Int<G>{}, Int<ROT>{});
      });
    });
  });
  return rc;
}

template <int D>
int launch_quantize_paged(const PagedCall& c) {
  int64_t total = 0;
  const TileGeom g = make_geom(c.n_slices, c.n_rows, c.heads, &total);
  if (total > INT_MAX) return SRFTQ_ERR_UNSUPPORTED;
  CUtensorMap tm_x, tm_none;
  std::memset(&tm_none, 0, sizeof(tm_none));
  if (encode_rows<D>(&tm_x, c.x, c.heads, c.n_rows, c.n_slices, c.x_stride_rows, g) != 0)
    return SRFTQ_ERR_CUDA;
  unsigned* guard = Runtime::guard_word();
  if (!guard) return SRFTQ_ERR_CUDA;
  const QuantArgs a{g, c.signs, c.lambda, c.codes, c.scales, c.pool_rows, guard, c.slots};
  return dispatch_paged<D>(c.bits, c.group, c.rotation, [&](auto b_, auto g_, auto r_) {
    constexpr int BITS = decltype(b_)::value, G = decltype(g_)::value, ROT = decltype(r_)::value;
    int bps = 0, smem, rc;
    if constexpr (D == 256) {
      constexpr auto K = quantize_split_kernel<D, BITS, G, ROT, kSplitMinBlocks, true>;
      smem = SplitLayout<D, BITS, G, true>::kBytes + kSmemSlack;
      if ((rc = prepare_kernel<K>(smem, 64, &bps)) != SRFTQ_OK) return rc;
      const int64_t cap = int64_t(Runtime::num_sms()) * bps;
      K<<<int(total < cap ? total : cap), 64, smem, c.stream>>>(tm_x, tm_none, a);
    } else {
      constexpr auto K = quantize_kernel<D, BITS, G, ROT, 1, 1, min_blocks<D, 0>(), true>;
      smem = WarpLayout<D, BITS, G, 1, true>::kWarpBytes + kSmemSlack;
      if ((rc = prepare_kernel<K>(smem, 32, &bps)) != SRFTQ_OK) return rc;
      const int64_t cap = int64_t(Runtime::num_sms()) * bps;
      K<<<int(total < cap ? total : cap), 32, smem, c.stream>>>(tm_x, tm_none, a);
    }
    return finish_launch();
  });
}

template <int D>
int launch_dequantize_paged(const PagedCall& c) {
  int64_t total = 0;
  const TileGeom g = make_geom(c.n_slices, c.n_rows, c.heads, &total);
  if (total > INT_MAX) return SRFTQ_ERR_UNSUPPORTED;
  CUtensorMap tm_x, tm_none;
  std::memset(&tm_none, 0, sizeof(tm_none));
  if (encode_rows<D>(&tm_x, c.xhat, c.heads, c.n_rows, c.n_slices, c.x_stride_rows, g) != 0)
    return SRFTQ_ERR_CUDA;
  unsigned* guard = Runtime::guard_word();
  if (!guard) return SRFTQ_ERR_CUDA;
  const DequantArgs a{g,           c.signs, c.lambda,        c.codes, c.scales,
                      c.pool_rows, c.xhat,  c.x_stride_rows, guard,   c.slots};
  return dispatch_paged<D>(c.bits, c.group, c.rotation, [&](auto b_, auto g_, auto r_) {
    constexpr int BITS = decltype(b_)::value, G = decltype(g_)::value, ROT = decltype(r_)::value;
    int bps = 0, smem, rc;
    if constexpr (D == 256) {
      constexpr auto K = dequantize_split_kernel<D, BITS, G, ROT, kSplitMinBlocks, true>;
      smem = SplitLayout<D, BITS, G, false>::kBytes + kSmemSlack;
      if ((rc = prepare_kernel<K>(smem, 64, &bps)) != SRFTQ_OK) return rc;
      const int64_t cap = int64_t(Runtime::num_sms()) * bps;
      K<<<int(total < cap ? total : cap), 64, smem, c.stream>>>(tm_none, tm_x, a);
    } else {
      constexpr auto K = dequantize_kernel<D, BITS, G, ROT, 1, 1, min_blocks<D, 0>(), true>;
      smem = WarpLayout<D, BITS, G, 1, false>::kWarpBytes + kSmemSlack;
      if ((rc = prepare_kernel<K>(smem, 32, &bps)) != SRFTQ_OK) return rc;
      const int64_t cap = int64_t(Runtime::num_sms()) * bps;
      K<<<int(total < cap ? total : cap), 32, smem, c.stream>>>(tm_none, tm_x, a);
    }
    return finish_launch();
  });
}

}  // namespace srftq
