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
// two fp32 values at once (a product and a sum of it may be fused, see Rotation)
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// pair i of a word of codes as bf16 (16 + low, 16 + high): the nibbles moved to the top mantissa bits under the
// exponent of 16
template <int I>
__device__ __forceinline__ uint32_t pair16(uint32_t w) {
  const uint32_t s = I == 0 ? w << 3 : I == 1 ? w >> 1 : I == 2 ? w >> 5 : w >> 9;
  return (s & 0x00780078u) | 0x41804180u;
}
// such a pair as values, minimum + step * code, each rounded once
__device__ __forceinline__ uint32_t value2(uint32_t c16, uint32_t step, uint32_t mn) {
  uint32_t c, r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(c16), "r"(0x41804180u));  // exact
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(c), "r"(step), "r"(mn));
  return r;
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
    if (interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float a = v[2 * k], b = v[2 * k + 1];
        v[2 * k] = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
        v[2 * k + 1] = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
      }
      return;
    }
    // Both results add a product that was taken times -1: the assembler makes one fused operation of a packed product and
    // a packed sum, whatever their rounding says, but leaves this form alone (a test compares the bits).
    const uint64_t minus = pack2(-1.0f, -1.0f);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint64_t a = pack2(v[k], v[k + 1]), b = pack2(v[8 + k], v[9 + k]), cc = pack2(c[k], c[k + 1]), ss = pack2(s[k], s[k + 1]);
      unpack2(fma2(mul2(b, ss), minus, mul2(a, cc)), v[k], v[k + 1]);
      unpack2(fma2(mul2(a, pack2(-s[k], -s[k + 1])), minus, mul2(b, cc)), v[8 + k], v[9 + k]);
    }
  }
};

// 8 values as they lie in memory, kept packed until they are used
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }  // read once
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
