// norm_rope.cu -- norm of queries and keys for each head with the position rotation in the same pass, and the table of
// cosines and sines that the rotation reads.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma + beta          (RMS)
//   y = (x - mean) / sqrt(var + eps) * gamma + beta       (Layer; population variance, two passes over registers)
//   (a, b) -> (a c - b s, b c + a s)                      for each of the rot/2 pairs of channels, angle of the token
//
// One pass: each value is read and written once, so memory bounds it.  A warp takes one token and up to four steps of
// 256/dh heads: its part of the table row and of gamma and beta stay in registers for all of them, and the loads of
// all steps are in flight before the first is used.  Statistics and rotation in fp32, one rounding when stored.
#include "history.cuh"

namespace rocs {

namespace {

template <int DH, typename T, int U>
__global__ void __launch_bounds__(256) rocs_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int LPR = DH / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const int which = w >= p.warps0;
  const NormRopeSide& sd = p.side[which];
  if (which) w -= p.warps0;
  const int t = (int)(w / sd.groups), h0 = (int)(w - (int64_t)t * sd.groups) * (RPW * U) + lane / LPR;
  const int l = lane & (LPR - 1);
  const T* x = static_cast<const T*>(sd.x) + (int64_t)t * sd.ld_x + (int64_t)h0 * DH + 8 * l;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = 0.0f;
    if (h0 + u * RPW < sd.heads) load8(x + u * RPW * DH, v[u]);
  }
  Rotation<DH> r;
  if (p.rope) {
    int pos = sd.pos[t];
    if ((unsigned)pos >= (unsigned)p.max_pos) {
      if (lane == 0) record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 901);
      pos = 0;
    }
    r.load(p.rope + (int64_t)pos * p.rot, p.rot, p.interleaved, lane);
  }
  float g[8], b[8];
  const bool has_g = p.norm != ROCS_NORM_NONE && sd.gamma, has_b = p.norm != ROCS_NORM_NONE && sd.beta;
  if (has_g) load8(sd.gamma + 8 * l, g);
  if (has_b) load8(sd.beta + 8 * l, b);
  T* out = static_cast<T*>(sd.out) + (int64_t)t * sd.ld_out + (int64_t)h0 * DH + 8 * l;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p.norm != ROCS_NORM_NONE) {
      float mean = 0.0f;
      if (p.norm == ROCS_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[u][k];
        mean = row_sum<LPR>(s) * (1.0f / DH);
      }
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[u][k] -= mean;
        s = fmaf(v[u][k], v[u][k], s);
      }
      const float inv = 1.0f / sqrtf(row_sum<LPR>(s) * (1.0f / DH) + p.eps);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[u][k] *= inv;
        if (has_g) v[u][k] *= g[k];
        if (has_b) v[u][k] += b[k];
      }
    }
    if (p.rope) r.apply(v[u], p.interleaved, lane);
    if (h0 + u * RPW < sd.heads) store8(out + u * RPW * DH, v[u]);
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
  const unsigned grid = (unsigned)((p.warps + 7) / 8);
  if (unroll == 4) rocs_norm_rope_kernel<DH, T, 4><<<grid, 256, 0, st>>>(p);
  else if (unroll == 2) rocs_norm_rope_kernel<DH, T, 2><<<grid, 256, 0, st>>>(p);
  else rocs_norm_rope_kernel<DH, T, 1><<<grid, 256, 0, st>>>(p);
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
