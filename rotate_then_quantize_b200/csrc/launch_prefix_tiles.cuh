// Launcher of the parts kernel of the shared-prefix attention; each head
// dimension is compiled in its own unit (launch_prefix_d*.cu).
#pragma once

#include "launch_impl.cuh"
#include "paged_attention.cuh"
#include "prefix_mma.cuh"
#include "prefix_pair.cuh"

namespace srftq {

// A programmatic launch: the grid may start while the one before it on the
// stream finishes, and waits for its results with griddepcontrol.wait.
template <auto K>
int launch_after(int grid, int threads, int smem, cudaStream_t stream, const PrefixArgs& a) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, K, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return SRFTQ_ERR_CUDA;
  }
  return SRFTQ_OK;
}

// The prefix's parts on tcgen05: d = 256, whose accumulators fill the tensor
// memory, by one unit per SM; else two units (a.pre_shared: of different rows).
template <int D, int BITS, int G, bool EXACT>
int launch_prefix_mma(const PrefixArgs& a, cudaStream_t stream) {
  const int64_t M = int64_t(a.n_seq) * a.q_per_kv;
  if constexpr (D == 256) {
    using L = PrefixMma<BITS, G, EXACT>;
    constexpr auto K = prefix_mma_kernel<BITS, G, EXACT>;
    const int rc = prepare_smem<K>(L::kSmem);
    if (rc != SRFTQ_OK) return rc;
    const int64_t tiles = (M + kMmaRows - 1) / kMmaRows;
    return launch_after<K>(int(tiles * a.heads * a.prefix_splits), L::kThreads, L::kSmem, stream, a);
  } else {
    int rc = SRFTQ_ERR_UNSUPPORTED;
    static_for<0, EXACT ? 1 : 2>([&](auto s_) {
      constexpr bool SHARED = decltype(s_)::value != 0;
      if (a.pre_shared != SHARED) return;
      using L = PrefixPair<D, BITS, G, EXACT, SHARED>;
      constexpr auto K = prefix_pair_kernel<D, BITS, G, EXACT, SHARED>;
      rc = prepare_smem<K>(L::kSmem);
      if (rc != SRFTQ_OK) return;
      const int64_t rows = SHARED ? 2 * kMmaRows : kMmaRows, blocks = (M + rows - 1) / rows;
      const int parts = SHARED ? a.prefix_splits : a.prefix_splits / 2;
      rc = launch_after<K>(int(blocks * a.heads * parts), L::kThreads, L::kSmem, stream, a);
    });
    return rc;
  }
}

// The own tokens' parts, and the prefix's: those either by the same kernel or,
// before it, by the tcgen05 kernel (a.pre_mma).
template <int D>
int launch_prefix_tiles(const PrefixArgs& a, int bits, int group, cudaStream_t stream) {
  int rc = SRFTQ_ERR_UNSUPPORTED;
  static_for<0, 2>([&](auto b_) {
    constexpr int BITS = decltype(b_)::value == 0 ? 4 : 8;
    static_for<4, ilog2(D) + 1>([&](auto lg_) {
      constexpr int G = 1 << decltype(lg_)::value;
      static_for<0, 2>([&](auto e_) {
        constexpr bool EXACT = decltype(e_)::value != 0;
        if (bits != BITS || group != G || EXACT == a.bf16) return;
        constexpr auto K = prefix_tile_kernel<D, BITS, G, EXACT>;
        constexpr int smem = TileLayout<D, BITS, G>::kBytes;
        int bps = 0;
        if (a.pre_mma) {
          rc = launch_prefix_mma<D, BITS, G, EXACT>(a, stream);
          if (rc != SRFTQ_OK) return;
        }
        rc = prepare_kernel<K>(smem, kTileWarps * 32, &bps);
        if (rc != SRFTQ_OK) return;
        rc = launch_after<K>(Runtime::num_sms() * bps, kTileWarps * 32, smem, stream, a);
      });
    });
  });
  return rc;
}

}  // namespace srftq
