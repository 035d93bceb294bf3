// norm_rope.cu -- norm of queries and keys for each head with the position rotation in the same pass, and the table of
// cosines and sines that the rotation reads.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma + beta          (RMS)
//   y = (x - mean) / sqrt(var + eps) * gamma + beta       (Layer; population variance, two passes over registers)
//   (a, b) -> (a c - b s, b c + a s)                      for each of the rot/2 pairs of channels, angle of the token
//
// One pass: each value is read and written once, so memory bounds it.  A warp takes U * 512/dh rows (heads of tokens, in
// their order); the loads of all of them are in flight before the first is used, and values stay packed as they came
// until their row's turn, so that 24 warps fit an SM.  Statistics and rotation in fp32, one rounding when stored.
// With 8 channels to a lane (half the rows to a warp, partners of a pair 8 lanes apart, one token to a warp) it took 131 us
// where this takes 74 us (16384 x 8 query and 65536 x 8 key rows of 128, bf16).
#include "history.cuh"

namespace rocs {

namespace {

template <int DH, typename T, int U>
__global__ void __launch_bounds__(128, 6) rocs_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = DH / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const int which = w >= p.warps0;
  const NormRopeSide& sd = p.side[which];
  if (which) w -= p.warps0;
  const int l = lane % LPR;
  const bool inter = p.interleaved, turned = p.rope && (inter ? 16 * l < p.rot : 8 * l < p.rot / 2);
  int ch0, ch1;
  groups_of(l, p.rope && !inter ? p.rot / 16 : 0, ch0, ch1);
  const int64_t row0 = w * (RPW * U) + lane / LPR, rows = (int64_t)sd.n * sd.heads;
  Raw8<T> raw[U][2];
  int64_t at[U];  // the row's place in the output
  int tok[U], pos[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * RPW;
    tok[u] = -1;
    at[u] = 0;
    if (row < rows) {
      tok[u] = (int)((uint32_t)row / (uint32_t)sd.heads);
      const int64_t in = (int64_t)(row - (int64_t)tok[u] * sd.heads) * DH;
      at[u] = (int64_t)tok[u] * sd.ld_out + in;
      const T* x = static_cast<const T*>(sd.x) + (int64_t)tok[u] * sd.ld_x + in;
      raw[u][0].load(x + ch0);
      raw[u][1].load(x + ch1);
    } else {
      raw[u][0].zero();
      raw[u][1].zero();
    }
    pos[u] = p.rope && tok[u] >= 0 ? sd.pos[tok[u]] : 0;
  }
  const bool has_g = p.norm != ROCS_NORM_NONE && sd.gamma, has_b = p.norm != ROCS_NORM_NONE && sd.beta;
  float g[16];
  if (has_g) {
    load8(sd.gamma + ch0, g);
    load8(sd.gamma + ch1, g + 8);
  }
  Rotation r;
  int held = -1;  // position that r is of
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (turned && (u == 0 || pos[u] != held)) {
      held = pos[u];
      int at_pos = held;
      if ((unsigned)at_pos >= (unsigned)p.max_pos) {
        record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 901);
        at_pos = 0;
      }
      r.load(p.rope + (int64_t)at_pos * p.rot, p.rot, l);
    }
    float v[16];
    raw[u][0].get(v);
    raw[u][1].get(v + 8);
    if (p.norm != ROCS_NORM_NONE) {
      if (p.norm == ROCS_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += v[k];
        const float mean = row_sum<LPR>(s) * (1.0f / DH);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] -= mean;
      }
      uint64_t sq = 0;
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const uint64_t x2 = pack2(v[k], v[k + 1]);
        sq = fma2(x2, x2, sq);
      }
      float s0, s1;
      unpack2(sq, s0, s1);
      const float ms = row_sum<LPR>(s0 + s1) * (1.0f / DH) + p.eps;
      // rsqrtf is off by 2 units of fp32 at most: nothing beside the rounding to bf16; fp32 outputs take the exact one
      const float inv = sizeof(T) == 2 ? rsqrtf(ms) : 1.0f / sqrtf(ms);
      const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        uint64_t y = mul2(pack2(v[k], v[k + 1]), inv2);
        if (has_g) y = mul2(y, pack2(g[k], g[k + 1]));
        unpack2(y, v[k], v[k + 1]);
      }
      if (has_b) {
        float b[16];
        load8(sd.beta + ch0, b);
        load8(sd.beta + ch1, b + 8);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] += b[k];
      }
    }
    if (turned) {
      if (inter) r.apply(v, true);
      else r.apply(v, false);
    }
    if (tok[u] >= 0) {
      T* out = static_cast<T*>(sd.out) + at[u];
      store8(out + ch0, v);
      store8(out + ch1, v + 8);
    }
  }
}

// angle = position * base^(-2i/rot) in 64 bits: fp32 would lose the angles of far positions
__global__ void rocs_rope_table_kernel(float* table, int64_t n, int half, double log_base) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t pos = i / half;
  const int k = (int)(i - pos * half);
  double s, c;
  sincos((double)pos * exp(-log_base * k / half), &s, &c);
  table[pos * 2 * half + k] = (float)c;
  table[pos * 2 * half + half + k] = (float)s;
}

template <int DH, typename T>
cudaError_t launch_nr(const NormRopeParams& p, int unroll, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.warps + 3) / 4);
  if (unroll == 2) rocs_norm_rope_kernel<DH, T, 2><<<grid, 128, 0, st>>>(p);
  else rocs_norm_rope_kernel<DH, T, 1><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dh, bool f32, int unroll, cudaStream_t st) {
  if (dh == 128) return f32 ? launch_nr<128, float>(p, unroll, st) : launch_nr<128, __nv_bfloat16>(p, unroll, st);
  return f32 ? launch_nr<64, float>(p, unroll, st) : launch_nr<64, __nv_bfloat16>(p, unroll, st);
}

cudaError_t launch_rope_table(float* table, int64_t max_pos, int rot, double base, cudaStream_t st) {
  const int64_t n = max_pos * (rot / 2);
  rocs_rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(table, n, rot / 2, log(base));
  return cudaGetLastError();
}

}  // namespace rocs
