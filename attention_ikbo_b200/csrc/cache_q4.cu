// cache_q4.cu -- append to and read from the paged 4-bit cache of request histories.
//
// A row (one head of one token) of dh values x is held as
//   minimum = bf16(min x),  step = bf16((max x - min x) / 15),  code = clamp(rint((x - minimum) / step), 0, 15)
// and stands for  minimum + step * code.  In every 32-bit word of codes (8 channels) nibble i of the low half is
// channel 2i and nibble i of the high half channel 2i + 1, so that one mask picks a pair of neighbouring channels out
// of a word, each in its own half.  A row that holds an infinity or a NaN, or whose range passes fp32, is held with a
// NaN step and minimum: all of it reads as NaN.
//
// Append: a warp takes one token's keys (rotated on the way) or values, up to four steps of 256/dh heads, as in
// norm_rope.cu.  Each value is read once and leaves as 4 bits; a row's statistics are min and max over its dh/8 lanes.
// The step is rounded to bf16 BEFORE the codes are taken, so that codes are nearest to what they will stand for.
#include "history.cuh"

namespace rocs {

namespace {

// The token's place: request r (of its index t), slot in the request's history, row of the cache (head 0).
// A slot outside the page table or a page outside the pool is reported and gives row < 0.
struct Place {
  int64_t row;  // index of (page, head 0, slot within the page) in units of rows
  int slot;
};
__device__ __forceinline__ Place place_of(const CacheMoveParams& p, int t, int lane, int where) {
  const int r = request_of(p.tok_off, p.R, t, lane);
  const int64_t slot = (int64_t)p.base[r] + (t - p.tok_off[r]);
  Place q;
  q.row = -1;
  q.slot = (int)slot;
  const int64_t k = slot >> p.c.page_log2;
  int page = -1;
  if (slot >= 0 && k < p.max_pages) page = p.table[(int64_t)r * p.max_pages + k];
  if ((unsigned)page < (unsigned)p.c.pages)
    q.row = (((int64_t)page * p.c.heads) << p.c.page_log2) + (slot & ((1 << p.c.page_log2) - 1));
  else if (lane == 0)
    record_error(p.ws, ROCS_ERR_DEVICE_INDEX, where);
  return q;
}

template <int LPR>
__device__ __forceinline__ void row_min_max(const float (&v)[8], float& lo, float& hi) {
  lo = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), fminf(fminf(v[4], v[5]), fminf(v[6], v[7])));
  hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

template <int DH, typename T, int U>
__global__ void __launch_bounds__(256) rocs_cache_append_kernel(const __grid_constant__ CacheMoveParams p) {
  constexpr int LPR = DH / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const int t = (int)(w / (2 * p.groups)), item = (int)(w - (int64_t)t * 2 * p.groups);
  const int kv = item >= p.groups;
  const int h0 = (item - kv * p.groups) * (RPW * U) + lane / LPR, l = lane & (LPR - 1);
  const T* x = static_cast<const T*>(p.x[kv]) + (int64_t)t * p.ld[kv] + (int64_t)h0 * DH + 8 * l;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = 0.0f;
    if (h0 + u * RPW < p.c.heads) load8(x + u * RPW * DH, v[u]);
  }
  const Place at = place_of(p, t, lane, 911);
  if (at.row < 0) return;
  Rotation<DH> r;
  const bool rotate = p.rope != nullptr;
  if (rotate) {
    const int pos = p.pos ? p.pos[t] : at.slot;
    if ((unsigned)pos >= (unsigned)p.max_pos) {
      if (lane == 0) record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 912);
      return;
    }
    if (!kv) r.load(p.rope + (int64_t)pos * p.rot, p.rot, p.interleaved, lane);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (rotate && !kv) r.apply(v[u], p.interleaved, lane);
    float lo, hi;
    row_min_max<LPR>(v[u], lo, hi);
    bool bad = false;  // min and max pass over NaN
#pragma unroll
    for (int k = 0; k < 8; ++k) bad |= v[u][k] != v[u][k];
    const unsigned any = __ballot_sync(0xffffffffu, bad);
    const float range = hi - lo;
    const unsigned mine = LPR == 16 ? 0xffffu << (lane & 16) : 0xffu << (lane & 24);
    const bool finite = range < INFINITY && !(any & mine);  // false too where range is NaN
    __nv_bfloat162 sc = __floats2bfloat162_rn(finite ? __fdiv_rn(range, 15.0f) : NAN, finite ? lo : NAN);
    const float step = __low2float(sc), mn = __high2float(sc);
    uint32_t code = 0;
    if (step > 0.0f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(v[u][k] - mn, step)), 0.0f), 15.0f);
        code |= (uint32_t)c << (4 * (k >> 1) + 16 * (k & 1));
      }
    }
    const int h = h0 + u * RPW;
    if (h < p.c.heads) {
      const int64_t row = at.row + ((int64_t)h << p.c.page_log2);
      *reinterpret_cast<uint32_t*>(p.c.codes[kv] + row * (DH / 2) + 4 * l) = code;
      if (l == 0) p.c.scale[kv][row] = sc;
    }
  }
}

template <int DH, int U>
__global__ void __launch_bounds__(256) rocs_cache_read_kernel(const __grid_constant__ CacheMoveParams p) {
  constexpr int LPR = DH / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const int t = (int)(w / (2 * p.groups)), item = (int)(w - (int64_t)t * 2 * p.groups);
  const int kv = item >= p.groups;
  const int h0 = (item - kv * p.groups) * (RPW * U) + lane / LPR, l = lane & (LPR - 1);
  const Place at = place_of(p, t, lane, 921);
  uint32_t code[U];
  __nv_bfloat162 sc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    code[u] = 0;
    sc[u] = __floats2bfloat162_rn(0.0f, 0.0f);
    const int h = h0 + u * RPW;
    if (h < p.c.heads && at.row >= 0) {  // a bad page reads as zeros (and is reported)
      const int64_t row = at.row + ((int64_t)h << p.c.page_log2);
      code[u] = *reinterpret_cast<const uint32_t*>(p.c.codes[kv] + row * (DH / 2) + 4 * l);
      sc[u] = p.c.scale[kv][row];
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.x[kv]) + (int64_t)t * p.ld[kv] + (int64_t)h0 * DH + 8 * l;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float step = __low2float(sc[u]), mn = __high2float(sc[u]);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf(step, (float)((code[u] >> (4 * (k >> 1) + 16 * (k & 1))) & 15u), mn);
    if (h0 + u * RPW < p.c.heads) store8(out + u * RPW * DH, v);
  }
}

template <int DH, typename T>
cudaError_t launch_ap(const CacheMoveParams& p, int unroll, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.warps + 7) / 8);
  if (unroll == 4) rocs_cache_append_kernel<DH, T, 4><<<grid, 256, 0, st>>>(p);
  else if (unroll == 2) rocs_cache_append_kernel<DH, T, 2><<<grid, 256, 0, st>>>(p);
  else rocs_cache_append_kernel<DH, T, 1><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}
template <int DH>
cudaError_t launch_rd(const CacheMoveParams& p, int unroll, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.warps + 7) / 8);
  if (unroll == 4) rocs_cache_read_kernel<DH, 4><<<grid, 256, 0, st>>>(p);
  else if (unroll == 2) rocs_cache_read_kernel<DH, 2><<<grid, 256, 0, st>>>(p);
  else rocs_cache_read_kernel<DH, 1><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheMoveParams& p, int dh, bool f32, int unroll, cudaStream_t st) {
  if (dh == 128) return f32 ? launch_ap<128, float>(p, unroll, st) : launch_ap<128, __nv_bfloat16>(p, unroll, st);
  return f32 ? launch_ap<64, float>(p, unroll, st) : launch_ap<64, __nv_bfloat16>(p, unroll, st);
}
cudaError_t launch_cache_read(const CacheMoveParams& p, int dh, int unroll, cudaStream_t st) {
  return dh == 128 ? launch_rd<128>(p, unroll, st) : launch_rd<64>(p, unroll, st);
}

}  // namespace rocs
