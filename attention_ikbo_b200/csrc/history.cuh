// history.cuh -- device pieces shared by the history-cache kernels.
//
// A row is one head of one token: dh values.  dh/8 lanes hold it, 8 consecutive channels each, so a warp holds
// 256/dh rows (2 at dh = 128, 4 at dh = 64) and every lane moves 16 bytes of bf16 or one 32-bit word of 4-bit codes.
#pragma once

#include "history.h"

namespace rocs {

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Rotation of one row's channel pairs (a, b) -> (a c - b s, b c + a s).  A lane's part of the table row is the same for
// every head of the token, so it is loaded once.  Halves: channel i < rot/2 pairs with i + rot/2, held by the lane
// rot/16 further on; interleaved: 2i pairs with 2i + 1, in the same lane.  Products and sums are rounded one by one
// (no fused multiply-add), so that a rotated key has the same bits wherever it is rotated: the 4-bit codes taken from
// it then do not depend on how the expression was compiled.
template <int DH>
struct Rotation {
  float c[8], s[8];
  int partner;  // lane with the other half (halves), -1: this lane's channels are not rotated
  bool second;  // this lane holds the second channels of its pairs (halves)
  __device__ __forceinline__ void load(const float* row, int rot, bool interleaved, int lane) {
    constexpr int LPR = DH / 8;
    const int l = lane & (LPR - 1), half = rot >> 1;
    partner = -1;
    second = false;
    if (8 * l >= rot) return;
    if (interleaved) {
      partner = lane;
      const float4 a = *reinterpret_cast<const float4*>(row + 4 * l), b = *reinterpret_cast<const float4*>(row + half + 4 * l);
      c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
      s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
    } else {
      second = 8 * l >= half;
      partner = second ? lane - half / 8 : lane + half / 8;
      const int i = second ? 8 * l - half : 8 * l;
      load8(row + i, c);
      load8(row + half + i, s);
    }
  }
  __device__ __forceinline__ void apply(float (&v)[8], bool interleaved, int lane) const {
    if (interleaved) {
      if (partner >= 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = v[2 * k], b = v[2 * k + 1];
          v[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
          v[2 * k + 1] = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
        }
      }
      return;
    }
    const int src = partner >= 0 ? partner : lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float o = __shfl_sync(0xffffffffu, v[k], src);
      if (partner >= 0) {
        const float x = __fmul_rn(v[k], c[k]), y = __fmul_rn(o, s[k]);
        v[k] = second ? __fadd_rn(x, y) : __fsub_rn(x, y);
      }
    }
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Largest r with off[r] <= t, for a t below off[R]: the warp narrows [0, R) by a factor of 32 with each load.
__device__ __forceinline__ int request_of(const int32_t* off, int R, int t, int lane) {
  int lo = 0, n = R;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool below = lane * step < n && off[i] <= t;  // monotone over the lanes; lane 0 is true
    const unsigned b = __ballot_sync(0xffffffffu, below);
    const int k = 31 - __clz(b | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

}  // namespace rocs
