// Rotations of one head-dim vector by a whole warp.
//
// The thread-per-vector transforms of transform.cuh move the most vectors per
// second, but one of them is about 2000 dependent-ish instructions: with only
// a few hundred vectors in a call (the queries and outputs of a decode step,
// the token a step appends) the call waits for that one chain. Here a warp
// holds one vector, d/32 reals to a lane, and each butterfly pass that spans
// lanes is a pair of shuffles, so a rotation is about 150 instructions long.
//
// SRFT ("When Quantization Is Free", Methodology 1): lane l holds the complex
// points z_m = u_{2m} + i u_{2m+1}, m = l E .. l E + E - 1 (E = d/64, L = d/2).
// A decimation-in-frequency FFT leaves Z_k at position p = bitrev(k). The
// Hermitian step needs Z_{L-k}: negation keeps the lowest set bit of k and
// flips the bits above it, so in bit-reversed positions the partner of p is
// p ^ (2^msb(p) - 1), one shuffle away. The lane ends with the packed pairs
// (y_{2k}, y_{2k+1}), k = bitrev(p). A group of 2^g coordinates is the 2^(g-1)
// bins that share the high bits of k, the low bits of p, so its lanes differ
// in the top bits of p. The inverse runs the steps backwards.
//
// SRHT: log2 d butterflies (a + b, a - b), natural order; lane l ends with the
// pairs l E .. l E + E - 1.
#pragma once

#include "common.cuh"
#include "transform.cuh"

namespace srftq {

// exp(-2 pi i k / D) for k < D / 2, rounded once from double.
template <int D>
struct TwiddleTable {
  float2 w[D / 2];
};
template <int D>
constexpr TwiddleTable<D> make_twiddles() {
  TwiddleTable<D> t{};
  for (int k = 0; k < D / 2; ++k) {
    t.w[k].x = float(ct::cos2pi(k, D));
    t.w[k].y = float(-ct::sin2pi(k, D));
  }
  return t;
}
static __device__ const TwiddleTable<64> g_twiddles_64 = make_twiddles<64>();
static __device__ const TwiddleTable<128> g_twiddles_128 = make_twiddles<128>();
static __device__ const TwiddleTable<256> g_twiddles_256 = make_twiddles<256>();
template <int D>
__device__ __forceinline__ const float2* twiddles() {
  if constexpr (D == 64) return g_twiddles_64.w;
  else if constexpr (D == 128) return g_twiddles_128.w;
  else return g_twiddles_256.w;
}

// Pair (coordinates 2k and 2k + 1) that element e of this lane holds in the
// rotated domain.
template <int ROT, int D>
__device__ __forceinline__ int warp_pair(int lane, int e) {
  constexpr int E = D / 64;
  const int p = lane * E + e;
  if constexpr (ROT == kSRHT) return p;
  return int(__brev(unsigned(p)) >> (32 - ilog2(D / 2)));
}

__device__ __forceinline__ float2 warp_xor(float2 v, int mask) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, mask),
                     __shfl_xor_sync(0xffffffffu, v.y, mask));
}
__device__ __forceinline__ float2 mul_cx(float2 a, float2 b) {
  return make_float2(fmaf(a.x, b.x, -a.y * b.y), fmaf(a.x, b.y, a.y * b.x));
}

// The elements of this lane's Hermitian partners (see the file comment).
template <int E>
__device__ __forceinline__ void warp_partners(const float2 (&z)[E], float2 (&q)[E], int lane) {
  const int src = lane ? lane ^ ((1 << (31 - __clz(lane))) - 1) : 0;
  static_for<0, E>([&](auto e_) {
    constexpr int e = decltype(e_)::value;
    const float2 v = z[e ^ (E - 1)];
    q[e] = make_float2(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src));
  });
  if (lane == 0) {   // positions 0 .. E - 1: 0 and 1 are their own partners, 2 and 3 each other's
    q[0] = z[0];
    if constexpr (E >= 2) q[1] = z[1];
    if constexpr (E == 4) {
      q[2] = z[3];
      q[3] = z[2];
    }
  }
}

// Walsh-Hadamard of the warp's D reals (unnormalised), natural order.
template <int E>
__device__ __forceinline__ void warp_walsh(float2 (&z)[E], int lane) {
  static_for<0, E>([&](auto e_) {
    constexpr int e = decltype(e_)::value;
    z[e] = make_float2(z[e].x + z[e].y, z[e].x - z[e].y);
  });
  static_for<0, ilog2(E)>([&](auto s_) {
    constexpr int h = 1 << decltype(s_)::value;
    static_for<0, E>([&](auto e_) {
      constexpr int e = decltype(e_)::value;
      if constexpr ((e & h) == 0) {
        const float2 a = z[e], b = z[e + h];
        z[e] = make_float2(a.x + b.x, a.y + b.y);
        z[e + h] = make_float2(a.x - b.x, a.y - b.y);
      }
    });
  });
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const float s = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 o = warp_xor(z[e], x);
      z[e] = make_float2(fmaf(s, z[e].x, o.x), fmaf(s, z[e].y, o.y));
    }
  }
}

// y = R u: z in = (u_{2m}, u_{2m+1}), m = lane E + e (signs applied); z out =
// the packed pairs warp_pair(lane, e), normalised.
template <int ROT, int D>
__device__ __forceinline__ void warp_rotate_forward(float2 (&z)[D / 64], int lane) {
  constexpr int E = D / 64, L = D / 2;
  constexpr float inv = float(inv_sqrt_pow2(D));
  if constexpr (ROT == kSRHT) {
    warp_walsh<E>(z, lane);
    static_for<0, E>([&](auto e_) {
      constexpr int e = decltype(e_)::value;
      z[e] = make_float2(z[e].x * inv, z[e].y * inv);
    });
  } else {
    const float2* tw = twiddles<D>();
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) {   // span h = x E
      const bool up = lane & x;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 w = tw[((lane & (x - 1)) * E + e) * (D / (2 * x * E))];
        const float2 o = warp_xor(z[e], x);
        const float2 sum = make_float2(z[e].x + o.x, z[e].y + o.y);
        const float2 dif = mul_cx(make_float2(o.x - z[e].x, o.y - z[e].y), w);
        z[e] = up ? dif : sum;
      }
    }
    static_for<0, ilog2(E)>([&](auto s_) {
      constexpr int h = E >> (decltype(s_)::value + 1);
      static_for<0, E>([&](auto e_) {
        constexpr int e = decltype(e_)::value;
        if constexpr ((e & h) == 0) {
          constexpr int j = e & (h - 1);
          constexpr float wr = float(ct::cos2pi(j, 2 * h)), wi = float(-ct::sin2pi(j, 2 * h));
          const float2 a = z[e], b = z[e + h];
          z[e] = make_float2(a.x + b.x, a.y + b.y);
          const float2 d = make_float2(a.x - b.x, a.y - b.y);
          z[e + h] = j == 0 ? d : mul_cx(d, make_float2(wr, wi));
        }
      });
    });
    float2 q[E];
    warp_partners<E>(z, q, lane);
    constexpr float half_gain = float(0.70710678118654752440 * inv_sqrt_pow2(D));   // sqrt2 / 2 / sqrt d
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = warp_pair<kSRFT, D>(lane, e);
      const float2 ev = make_float2(z[e].x + q[e].x, z[e].y - q[e].y);
      const float2 od = make_float2(z[e].x - q[e].x, z[e].y + q[e].y);
      const float2 t = mul_cx(tw[k], od);
      const float2 y = make_float2((ev.x + t.y) * half_gain, (ev.y - t.x) * half_gain);
      z[e] = k == 0 ? make_float2((z[e].x + z[e].y) * inv, (z[e].x - z[e].y) * inv) : y;
    }
  }
  (void)L;
}

// u = R^T y: z in = the packed pairs warp_pair(lane, e); z out = (u_{2m},
// u_{2m+1}), m = lane E + e (before the signs).
template <int ROT, int D>
__device__ __forceinline__ void warp_rotate_inverse(float2 (&z)[D / 64], int lane) {
  constexpr int E = D / 64;
  constexpr float inv = float(inv_sqrt_pow2(D));
  if constexpr (ROT == kSRHT) {
    warp_walsh<E>(z, lane);
    static_for<0, E>([&](auto e_) {
      constexpr int e = decltype(e_)::value;
      z[e] = make_float2(z[e].x * inv, z[e].y * inv);
    });
  } else {
    const float2* tw = twiddles<D>();
    float2 q[E];
    warp_partners<E>(z, q, lane);
    constexpr float gain = float(0.70710678118654752440 * inv_sqrt_pow2(D));   // 1 / sqrt(2 d)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = warp_pair<kSRFT, D>(lane, e);
      // Z_k = E + i conj(W^k) (X_k - conj X_{L-k}), E = X_k + conj X_{L-k}
      const float2 ev = make_float2(z[e].x + q[e].x, z[e].y - q[e].y);
      const float2 df = make_float2(z[e].x - q[e].x, z[e].y + q[e].y);
      const float2 w = tw[k];
      const float2 t = mul_cx(make_float2(w.x, -w.y), df);
      const float2 y = make_float2((ev.x - t.y) * gain, (ev.y + t.x) * gain);
      z[e] = k == 0 ? make_float2((z[e].x + z[e].y) * inv, (z[e].x - z[e].y) * inv) : y;
    }
    static_for<0, ilog2(E)>([&](auto s_) {
      constexpr int h = 1 << decltype(s_)::value;
      static_for<0, E>([&](auto e_) {
        constexpr int e = decltype(e_)::value;
        if constexpr ((e & h) == 0) {
          constexpr int j = e & (h - 1);
          constexpr float wr = float(ct::cos2pi(j, 2 * h)), wi = float(ct::sin2pi(j, 2 * h));
          const float2 b = j == 0 ? z[e + h] : mul_cx(z[e + h], make_float2(wr, wi));
          const float2 a = z[e];
          z[e] = make_float2(a.x + b.x, a.y + b.y);
          z[e + h] = make_float2(a.x - b.x, a.y - b.y);
        }
      });
    });
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const bool up = lane & x;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 w = tw[((lane & (x - 1)) * E + e) * (D / (2 * x * E))];
        const float2 t = up ? mul_cx(z[e], make_float2(w.x, -w.y)) : z[e];
        const float2 o = warp_xor(t, x);
        z[e] = up ? make_float2(o.x - t.x, o.y - t.y) : make_float2(t.x + o.x, t.y + o.y);
      }
    }
  }
}

}  // namespace srftq
