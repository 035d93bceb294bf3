// cache_q4.cu -- append to and read from the paged 4-bit cache of request histories.
//
// A row (one head of one token) of dh values x is held as
//   minimum = bf16(min x),  step = bf16((max x - min x) / 15),  code = clamp(rint((x - minimum) / step), 0, 15)
// and stands for  minimum + step * code.  In every 32-bit word of codes (8 channels) nibble i of the low half is
// channel 2i and nibble i of the high half channel 2i + 1, so that one mask picks a pair of neighbouring channels out
// of a word, each in its own half.  A row that holds an infinity or a NaN, or whose range passes fp32, is held with a
// NaN step and minimum: all of it reads as NaN.
//
// Append: a warp takes U * 512/dh rows (heads of tokens, in their order) of the keys, rotated on the way, or of the values.
// Each value is read once and leaves as 4 bits; a row's statistics are min and max over its dh/16 lanes.  The places of the
// (at most 32) tokens are looked up once for the warp, a token to a lane.  The step is rounded to bf16 BEFORE the codes are
// taken, so that codes are nearest to what they will stand for.  Memory bounds both directions; with one token to a warp and
// a division for every value the two together took 129 us where they take APUS (8 histories of 4096-8192 events, 4 heads of
// 128).
#include "history.cuh"

namespace rocs {

namespace {

// The places of tokens t0 + lane (those below T): request, slot in its history, row of the cache (head 0).  A slot outside
// the page table or a page outside the pool is reported and gives row < 0.
struct Place {
  int64_t row;  // index of (page, head 0, slot within the page) in units of rows
  int slot;
};
__device__ __forceinline__ Place places(const CacheMoveParams& p, int t0, int n, int lane, int where) {
  Place q;
  q.row = -1;
  q.slot = 0;
  int r = request_of(p.tok_off, p.R, t0, lane);
  if (lane < n) {
    const int t = t0 + lane;
    while (r + 1 < p.R && p.tok_off[r + 1] <= t) ++r;
    const int64_t slot = (int64_t)p.base[r] + (t - p.tok_off[r]);
    q.slot = (int)slot;
    const int64_t k = slot >> p.c.page_log2;
    int page = -1;
    if (slot >= 0 && k < p.max_pages) page = p.table[(int64_t)r * p.max_pages + k];
    if ((unsigned)page < (unsigned)p.c.pages)
      q.row = (((int64_t)page * p.c.heads) << p.c.page_log2) + (slot & ((1 << p.c.page_log2) - 1));
    else
      record_error(p.ws, ROCS_ERR_DEVICE_INDEX, where);
  }
  return q;
}

template <int LPR>
__device__ __forceinline__ void row_min_max(const float (&v)[16], float& lo, float& hi) {
  lo = hi = v[0];
#pragma unroll
  for (int k = 1; k < 16; ++k) {
    lo = fminf(lo, v[k]);
    hi = fmaxf(hi, v[k]);
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

// Codes of 8 values, packed: rint((x - mn) / step) held to 0 ... 15.  The quotient by a reciprocal is off by at most 2^-22 of
// itself, so it rounds as the exact one does unless it lies within 2e-5 of a half; then (rare) the values are divided.
__device__ __forceinline__ uint32_t codes8(const float* v, float mn, float step, float inv) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, half to even
  float c[8], far = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = fminf(fmaxf((v[k] - mn) * inv, 0.0f), 15.0f);
    c[k] = __fsub_rn(__fadd_rn(t, kRound), kRound);
    far = fmaxf(far, fabsf(t - c[k]));
  }
  if (far > 0.49998f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = fminf(fmaxf(rintf(__fdiv_rn(v[k] - mn, step)), 0.0f), 15.0f);
  }
  // whole numbers below 2^16 in fp32 are exact, and 2^23 more leaves them in the low bits
  const float even = fmaf(4096.0f, c[6], fmaf(256.0f, c[4], fmaf(16.0f, c[2], c[0]))) + 8388608.0f;
  const float odd = fmaf(4096.0f, c[7], fmaf(256.0f, c[5], fmaf(16.0f, c[3], c[1]))) + 8388608.0f;
  return __byte_perm(__float_as_uint(even), __float_as_uint(odd), 0x5410);
}

template <int DH, typename T, int U>
__global__ void __launch_bounds__(256) rocs_cache_append_kernel(const __grid_constant__ CacheMoveParams p) {
  constexpr int LPR = DH / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= 2 * p.warps) return;
  const int kv = w >= p.warps, heads = p.c.heads;
  if (kv) w -= p.warps;
  const bool rotate = p.rope != nullptr && !kv, inter = p.interleaved;
  const bool turned = rotate && (inter ? 16 * l < p.rot : 8 * l < p.rot / 2);
  int ch0, ch1;
  groups_of(l, rotate && !inter ? p.rot / 16 : 0, ch0, ch1);
  const int64_t first = w * (RPW * U);
  const int t0 = (int)((uint32_t)first / (uint32_t)heads);
  Raw8<T> raw[U][2];
  int tok[U], head[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = first + u * RPW + lane / LPR;
    tok[u] = -1;
    head[u] = 0;
    if (row < p.rows) {
      tok[u] = (int)((uint32_t)row / (uint32_t)heads);
      head[u] = (int)(row - (int64_t)tok[u] * heads);
      const T* x = static_cast<const T*>(p.x[kv]) + (int64_t)tok[u] * p.ld[kv] + (int64_t)head[u] * DH;
      raw[u][0].load(x + ch0);
      raw[u][1].load(x + ch1);
    } else {
      raw[u][0].zero();
      raw[u][1].zero();
    }
  }
  const int64_t last = min(first + RPW * U, p.rows) - 1;
  const int n = (int)((uint32_t)last / (uint32_t)heads) - t0 + 1;
  Place at = places(p, t0, n, lane, 911);
  int pos = at.slot;
  if (p.rope && lane < n) {
    if (p.pos) pos = p.pos[t0 + lane];
    if ((unsigned)pos >= (unsigned)p.max_pos) {
      record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 912);
      at.row = -1;
      pos = 0;
    }
  }
  Rotation r;
  int held = -1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int from = max(tok[u] - t0, 0);
    const int64_t place = __shfl_sync(0xffffffffu, at.row, from);
    const int ps = __shfl_sync(0xffffffffu, pos, from);
    float v[16];
    raw[u][0].get(v);
    raw[u][1].get(v + 8);
    if (turned) {
      if (ps != held) {
        held = ps;
        r.load(p.rope + (int64_t)ps * p.rot, p.rot, l);
      }
      if (inter) r.apply(v, true);
      else r.apply(v, false);
    }
    float lo, hi;
    row_min_max<LPR>(v, lo, hi);
    bool bad = false;  // min and max pass over NaN
#pragma unroll
    for (int k = 0; k < 16; ++k) bad |= v[k] != v[k];
    const unsigned any = __ballot_sync(0xffffffffu, bad);
    const float range = hi - lo;
    const unsigned mine = ((1u << LPR) - 1) << (lane & ~(LPR - 1));
    const bool finite = range < INFINITY && !(any & mine);  // false too where range is NaN
    const __nv_bfloat162 sc = __floats2bfloat162_rn(finite ? __fdiv_rn(range, 15.0f) : NAN, finite ? lo : NAN);
    const float step = __low2float(sc), mn = __high2float(sc);
    uint32_t w0 = 0, w1 = 0;
    if (step > 0.0f) {
      // a step whose reciprocal is not a normal number takes the division for every value
      const float inv = step > 1e-37f && step < 1e37f ? 1.0f / step : NAN;
      if (inv == inv) {
        w0 = codes8(v, mn, step, inv);
        w1 = codes8(v + 8, mn, step, inv);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t c = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[k] - mn, step)), 0.0f), 15.0f) << (4 * ((k & 7) >> 1) + 16 * (k & 1));
          if (k < 8) w0 |= c;
          else w1 |= c;
        }
      }
    }
    if (tok[u] >= 0 && place >= 0) {
      const int64_t row = place + ((int64_t)head[u] << p.c.page_log2);
      uint8_t* to = p.c.codes[kv] + row * (DH / 2);
      *reinterpret_cast<uint32_t*>(to + ch0 / 2) = w0;
      *reinterpret_cast<uint32_t*>(to + ch1 / 2) = w1;
      if (l == 0) p.c.scale[kv][row] = sc;
    }
  }
}

template <int DH, int U>
__global__ void __launch_bounds__(256) rocs_cache_read_kernel(const __grid_constant__ CacheMoveParams p) {
  constexpr int LPR = DH / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= 2 * p.warps) return;
  const int kv = w >= p.warps, heads = p.c.heads;
  if (kv) w -= p.warps;
  const int64_t first = w * (RPW * U), last = min(first + RPW * U, p.rows) - 1;
  const int t0 = (int)((uint32_t)first / (uint32_t)heads), n = (int)((uint32_t)last / (uint32_t)heads) - t0 + 1;
  const Place at = places(p, t0, n, lane, 921);
  uint2 code[U];
  __nv_bfloat162 sc[U];
  int64_t to[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = first + u * RPW + lane / LPR;
    const bool have = row <= last;
    const int tok = have ? (int)((uint32_t)row / (uint32_t)heads) : t0, head = have ? (int)(row - (int64_t)tok * heads) : 0;
    const int64_t place = __shfl_sync(0xffffffffu, at.row, tok - t0);
    to[u] = have ? (int64_t)tok * p.ld[kv] + (int64_t)head * DH + 16 * l : -1;
    code[u] = make_uint2(0, 0);
    sc[u] = __floats2bfloat162_rn(0.0f, 0.0f);
    if (have && place >= 0) {  // a bad page reads as zeros (and is reported)
      const int64_t from = place + ((int64_t)head << p.c.page_log2);
      code[u] = *reinterpret_cast<const uint2*>(p.c.codes[kv] + from * (DH / 2) + 8 * l);
      sc[u] = p.c.scale[kv][from];
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.x[kv]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (to[u] < 0) continue;
    const float step = __low2float(sc[u]), mn = __high2float(sc[u]);
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = fmaf(step, (float)(((k < 8 ? code[u].x : code[u].y) >> (4 * ((k & 7) >> 1) + 16 * (k & 1))) & 15u), mn);
    store8(out + to[u], v);
    store8(out + to[u] + 8, v + 8);
  }
}

template <int DH, typename T>
cudaError_t launch_ap(const CacheMoveParams& p, int unroll, cudaStream_t st) {
  const unsigned grid = (unsigned)((2 * p.warps + 7) / 8);
  if (unroll == 2) rocs_cache_append_kernel<DH, T, 2><<<grid, 256, 0, st>>>(p);
  else rocs_cache_append_kernel<DH, T, 1><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}
template <int DH>
cudaError_t launch_rd(const CacheMoveParams& p, int unroll, cudaStream_t st) {
  const unsigned grid = (unsigned)((2 * p.warps + 7) / 8);
  if (unroll == 4) rocs_cache_read_kernel<DH, 4><<<grid, 256, 0, st>>>(p);
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
