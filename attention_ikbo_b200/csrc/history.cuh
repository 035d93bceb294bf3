// history.cuh -- device pieces shared by the history-cache kernels.
//
// A row is one head of one token: dh values.  dh/16 lanes hold it, 16 channels each in two groups of 8, so a warp holds
// 512/dh rows (4 at dh = 128, 8 at dh = 64).  With channel i turned with channel i + rot/2 a lane's groups are rot/2
// apart, so both channels of a pair are in one lane and the rotation needs no shuffles; otherwise they are neighbours.
// Rows are numbered token * heads + head, and a warp takes U * 512/dh of them in a row, whatever the number of heads.
#pragma once

#include "history.h"

namespace rocs {

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// First channels of a lane's two groups: lane l of a row's dh/16.  turned: rot/16, with halves paired; 0 otherwise.
__device__ __forceinline__ void groups_of(int l, int turned, int& c0, int& c1) {
  c0 = l < turned ? 8 * l : 16 * l;
  c1 = l < turned ? 8 * (l + turned) : 16 * l + 8;
}

// Rotation of one row's channel pairs (a, b) -> (a c - b s, b c + a s).  Halves: channel i < rot/2 pairs with i + rot/2;
// interleaved: 2i pairs with 2i + 1.  Products and sums are rounded one by one (no fused multiply-add), so that a rotated
// key has the same bits wherever it is rotated: the 4-bit codes taken from it then do not depend on how the expression
// was compiled.
struct Rotation {
  float c[8], s[8];  // of this lane's 8 pairs
  __device__ __forceinline__ void load(const float* row, int rot, int l) {
    load8(row + 8 * l, c);
    load8(row + (rot >> 1) + 8 * l, s);
  }
  __device__ __forceinline__ void apply(float (&v)[16], bool interleaved) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = interleaved ? v[2 * k] : v[k], b = interleaved ? v[2 * k + 1] : v[8 + k];
      const float y = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k])), z = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
      if (interleaved) {
        v[2 * k] = y;
        v[2 * k + 1] = z;
      } else {
        v[k] = y;
        v[8 + k] = z;
      }
    }
  }
};

// 8 values as they lie in memory, kept packed until they are used
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
