// cache_q4.cu -- append to and read from the paged 4-bit cache of request histories.
//
// A row (one head of one token) of dh values x is held as
//   minimum = bf16(min x),  step = bf16((max x - min x) * (1/15)),  code = clamp(rint((x - minimum) / step), 0, 15)
// in fp32, and stands for  minimum + step * code.  In every 32-bit word of codes (8 channels) nibble i of the low half is
// channel 2i and nibble i of the high half channel 2i + 1, so that one mask picks a pair of neighbouring channels out
// of a word, each in its own half.  A row that holds an infinity or a NaN, or whose range passes fp32, is held with a
// NaN step and minimum: all of it reads as NaN.
//
// Append: a warp takes U * 512/dh rows (heads of tokens, in their order) of the keys, rotated on the way, or of the values.
// Each value is read once and leaves as 4 bits; a row's statistics are min and max over its dh/16 lanes.  The places of the
// (at most 32) tokens are looked up once for the warp, a token to a lane.  The step is rounded to bf16 BEFORE the codes are
// taken, so that codes are nearest to what they will stand for.  Memory bounds both directions; with one token to a warp and
// a division for every value the two together took 129 us where they take 76 us (8 histories of 4096-8192 events, 4 heads of
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
    if (r + 1 < p.R && p.tok_off[r + 1] <= t) {  // a later request's, perhaps behind many without tokens
      int hi = p.R;
      while (hi - r > 1) {
        const int mid = r + (hi - r) / 2;
        if (p.tok_off[mid] <= t) r = mid;
        else hi = mid;
      }
    }
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
  lo = fminf(v[0], v[1]);
  hi = fmaxf(v[0], v[1]);
#pragma unroll
  for (int k = 2; k < 16; k += 2) {
    asm("min.f32 %0, %0, %1, %2;" : "+f"(lo) : "f"(v[k]), "f"(v[k + 1]));
    asm("max.f32 %0, %0, %1, %2;" : "+f"(hi) : "f"(v[k]), "f"(v[k + 1]));
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}

// Codes of 8 values, packed: rint((x - mn) / step), held to 0 ... 15 where CLAMP.  The quotient by the reciprocal is
// corrected with its own remainder (exact, a fused multiply-add), which rounds it as the division does (Markstein's
// method); bf16 values lie on a grid, so quotients of exactly a half are common and have to come out as such.
template <bool CLAMP>
__device__ __forceinline__ uint32_t codes8(const float* v, float mn, float step, float inv) {
  const uint64_t mn2 = pack2(-mn, -mn), step2 = pack2(-step, -step), inv2 = pack2(inv, inv);
  // adding 1.5 * 2^23 rounds to a whole number, half to even, and leaves it in the low bits
  const uint64_t round2 = pack2(12582912.0f, 12582912.0f);
  uint32_t c[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t d = add2(pack2(v[k], v[k + 1]), mn2), t = mul2(d, inv2);
    uint64_t q = fma2(fma2(t, step2, d), inv2, t);
    float a, b;
    if (CLAMP) {
      unpack2(q, a, b);
      q = pack2(fminf(fmaxf(a, 0.0f), 15.0f), fminf(fmaxf(b, 0.0f), 15.0f));
    }
    unpack2(add2(q, round2), a, b);
    c[k] = __float_as_uint(a);
    c[k + 1] = __float_as_uint(b);
  }
  // the low halves of the words of 1.5 * 2^23 are zero: only codes meet there
  const uint32_t even = c[0] + (c[2] << 4) + (c[4] << 8) + (c[6] << 12), odd = c[1] + (c[3] << 4) + (c[5] << 8) + (c[7] << 12);
  return __byte_perm(even, odd, 0x5410);
}

template <int DH, typename T, int U>
__global__ void __launch_bounds__(256, 4) rocs_cache_append_kernel(const __grid_constant__ CacheMoveParams p) {
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
    uint64_t z = 0;  // min and max pass over NaN; times zero and summed it stays (and an infinity becomes one)
#pragma unroll
    for (int k = 0; k < 16; k += 2) z = fma2(pack2(v[k], v[k + 1]), 0, z);
    float z0, z1;
    unpack2(z, z0, z1);
    const unsigned any = __ballot_sync(0xffffffffu, !(z0 + z1 == 0.0f));
    const float range = hi - lo;
    const unsigned mine = ((1u << LPR) - 1) << (lane & ~(LPR - 1));
    const bool finite = range < INFINITY && !(any & mine);  // false too where range is NaN
    // The format takes a fifteenth by the product: off by one unit of fp32 at most, so that only quotients midway between two
    // bf16 values may round to the other one, which is as near.
    const __nv_bfloat162 sc = __floats2bfloat162_rn(finite ? range * (1.0f / 15.0f) : NAN, finite ? lo : NAN);
    const float step = __low2float(sc), mn = __high2float(sc);
    uint32_t w0 = 0, w1 = 0;
    if (step > 1e-36f && step < 1e36f) {
      const float inv = 1.0f / step;
      // the row's ends say whether a value can pass 0 ... 15 (the minimum was rounded up, or the step down)
      if ((lo - mn) * inv > -0.49f && (hi - mn) * inv < 15.49f) {
        w0 = codes8<false>(v, mn, step, inv);
        w1 = codes8<false>(v + 8, mn, step, inv);
      } else {
        w0 = codes8<true>(v, mn, step, inv);
        w1 = codes8<true>(v + 8, mn, step, inv);
      }
    } else if (step > 0.0f) {  // so small or large that the reciprocal is no normal number
#pragma unroll 1
      for (int k = 0; k < 16; ++k) {
        float x = v[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) x = k == i ? v[i] : x;
        const uint32_t c = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(x - mn, step)), 0.0f), 15.0f) << (4 * ((k & 7) >> 1) + 16 * (k & 1));
        if (k < 8) w0 |= c;
        else w1 |= c;
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
    const uint32_t rsc = *reinterpret_cast<const uint32_t*>(&sc[u]);
    const uint32_t st = __byte_perm(rsc, rsc, 0x1010), mn = __byte_perm(rsc, rsc, 0x3232);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t c = k ? code[u].y : code[u].x;
      st_global_v4(out + to[u] + 8 * k, value2(pair16<0>(c), st, mn), value2(pair16<1>(c), st, mn), value2(pair16<2>(c), st, mn),
                   value2(pair16<3>(c), st, mn));
    }
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
