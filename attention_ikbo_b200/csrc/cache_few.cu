// cache_few.cu -- attention over the paged 4-bit cache for few query rows (single tokens, a handful of candidates).
//
//   O_i = softmax_j(scale q_i . k_j) v_j,   k_j = mK_j + sK_j cK_j,   v_j = mV_j + sV_j cV_j      (codes c in 0..15)
//
// The codes go to the tensor core as they are: 16 + c is exact in bf16 (four mantissa bits under a leading one), and so is
// c - 8, which one packed subtraction makes of it.  So
//   q_i . k_j = sK_j (q_i . (16 + cK_j)) + (mK_j - 16 sK_j) sum(q_i)
//   O_i       = sum_j P'_ij (cV_j - 8) + sum_j (p_ij mV_j + 8 P'_ij),     P'_ij = p_ij sV_j
// and unpacking costs a shift and one three-input logic operation for two values.  Scores are exact up to fp32 sums.  P'
// goes to the tensor core in two bf16 parts (16 bits), so that O carries no rounding beside its own (0.00166 of its norm,
// for 65,536 keys as for 300,000); the second product costs 10 us of the case below.
//
// Sums over the keys have to stay small and short.  The tensor core cuts off what falls below its accumulator instead of
// rounding, always towards zero, so an accumulator that grows with the number of keys loses a little of itself with each
// step.  With 16 + c in place of c - 8 it grew whatever the values, and the error of O was 0.046 of its norm for 65,536
// keys and 0.44 for 300,000.  Centred codes leave it as large as the result is, and every kWindow granules it is added
// to fp32 sums in shared memory (rounded to nearest) and begins anew, as the sums of P and of p mV + 8 P' do.
//
// With a few rows to a pair of (request, key head) each 4-bit value is used a few times: the bytes of the cache and the
// unpacking bound it.  mma.sync takes its operands from registers, so codes go from shared memory through the logic
// operations straight into fragments, with no second trip through shared memory as a tcgen05 operand tile would need.
// Keys (in Q K^T) and channels (in P V) are the instruction's 16 rows and query rows its 8 columns, so 8 rows fill it,
// where a tcgen05 tile has at least 64: S^T = K Q^T, O^T = V^T P^T, and an 8 x 8 transposition (movmatrix) turns S^T's
// layout into that of P^T.  NB = 1 or 2 blocks of 8 rows share the unpacked codes.  With query rows as the 16 rows of the
// instruction (8 keys or channels to each) it issued twice the products and exponentials for up to 8 rows, and took 204
// us where this form took 144 us (P in one part, 16 + c in the sums) and takes 158 us as it is (32 histories of 8192-16384
// keys, 8 heads of 128, 4 rows; the centring and the windows are 4 us of it).
//
// Each warp takes 16 keys at a time through its own ring of cp.async stages (a 16-key granule never crosses a page) with its
// own running softmax: no block-wide synchronisation until the unit's end, where the four warps' results are joined in
// shared memory.  A row's maximum is only taken where a score passes the running one by more than 2^8 (a vote finds that).
//
// Fragments without shuffles: the contraction index may be permuted freely as long as both operands agree.  Lane
// (g, t) = (lane / 4, lane % 4) owns channels t*DH/4 ... of keys g and g + 8 (and of query row g) in Q K^T, and channels
// g*DH/8 ... of its keys 2t, 2t + 1, 2t + 8, 2t + 9 in P V, which leaves it with DH/8 contiguous channels of O for rows 2t
// and 2t + 1.
#include "cache_work.cuh"

namespace rocs {

namespace {

constexpr int kWarps = 4, kThreadsFew = kWarps * 32, kStages = 4, kGran = 16, kKeys = kWarps * kGran;
constexpr int kWindow = 64;  // granules of a warp between two additions to its sums

template <int DH, int NB>
struct FewSmem {
  static constexpr int kRow = DH / 2;                         // bytes of codes in a row
  static constexpr int kStage = 2 * kGran * kRow + 2 * kGran * 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kLd = DH + 4;                          // O of a row, its sum of P and its maximum (two words unused)
  static constexpr int kSums = kWarps * 8 * NB * kLd * 4;     // of every warp
  static constexpr int kBuf = kRing + kSums;
};
// a pair of 16 + c as c - 8, exact
__device__ __forceinline__ uint32_t centred(uint32_t c16) {
  uint32_t c;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(c16), "r"(0x41C041C0u));
  return c;
}
template <int DH>
constexpr int few_part() { return kFewRows * (DH + 2); }  // floats of one partial result

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // of an 8 x 8 matrix of 16-bit values over the warp
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int DH, int NB>
__global__ void __launch_bounds__(kThreadsFew, 3) rocs_cache_few_kernel(const __grid_constant__ CacheAttnParams p) {
  using L = FewSmem<DH, NB>;
  constexpr int KS = DH / 16;   // contraction steps of Q K^T, and 16-channel tiles of O
  constexpr int CH = DH / 4;    // channels of a row that a lane holds in Q K^T
  constexpr int OC = DH / 8;    // channels of O that a lane holds
  constexpr int kRows = 8 * NB;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_sum[33], s_out[3];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  Work<kKeys> w;
  if (!w.start(p, kRows, s_sum, s_out, 2)) return;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * L::kStage);
  float* const sums = reinterpret_cast<float*>(smem + L::kRing), *const mine = sums + warp * kRows * L::kLd;
  const float c = p.scale_log2;

  for (bool more = true; more;) {
    const Request& q = w.q;
    const int row0 = w.chunk * kRows, n_steps = w.count();
    const int tpr = p.G;  // rows of one token
    // Q fragments: row g of each block, this lane's CH channels; sums and limits of rows 2t and 2t + 1
    uint32_t qb[NB][KS][2];
    float qsum[NB][2];
    int lim[NB][2], lim_min = q.L;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row = row0 + 8 * b + g;
      const int tok = row < q.rows ? row / tpr : 0, hh = w.head * p.G + (row < q.rows ? row - tok * tpr : 0);
      const int64_t token = (int64_t)q.c0 * p.q_tokens + tok;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + token * p.q_ld + (int64_t)hh * DH + t * CH);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < CH / 8; ++k) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < q.rows) u = src[k];
        qb[b][2 * k][0] = u.x;
        qb[b][2 * k][1] = u.y;
        qb[b][2 * k + 1][0] = u.z;
        qb[b][2 * k + 1][1] = u.w;
        s += (bf_lo(u.x) + bf_hi(u.x)) + (bf_lo(u.y) + bf_hi(u.y)) + (bf_lo(u.z) + bf_hi(u.z)) + (bf_lo(u.w) + bf_hi(u.w));
      }
      s = quad_sum(s);
      const int mine = row_limit(p, q, row);
      lim_min = min(lim_min, mine);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // row 2t + e is that of lanes with g = 2t + e
        qsum[b][e] = __shfl_sync(0xffffffffu, s, 4 * (2 * t + e));
        lim[b][e] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + e));
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);

    float o[NB][KS][4], m[NB][2], l[NB][2], corr[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[b][e] = -INFINITY;
        l[b][e] = corr[b][e] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[b][k][i] = 0.0f;
    }

    // this warp's granules: step*4 + warp, those with keys in them
    const int first = w.step * kWarps + warp, all = (q.L + kGran - 1) / kGran;
    const int n = max(0, min(n_steps, (all - first + kWarps - 1) / kWarps));
    const int32_t* table = p.table + (int64_t)w.r * p.max_pages;
    auto page_of = [&](int i) { return i < n ? table[((first + i * kWarps) * kGran) >> p.c.page_log2] : 0; };
    auto issue = [&](int i, int page) {
      if (i < n) {
        if ((unsigned)page >= (unsigned)p.c.pages) {
          if (lane == 0) record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 933);
          page = 0;
        }
        const int slot = ((first + i * kWarps) * kGran) & ((1 << p.c.page_log2) - 1);
        const int64_t row = (((int64_t)page * p.c.heads + w.head) << p.c.page_log2) + slot;
        const uint32_t st = ring + (i % kStages) * L::kStage;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint8_t* src = p.c.codes[kv] + row * L::kRow;
#pragma unroll
          for (int k = 0; k < kGran * L::kRow / 512; ++k) {
            const int ch = lane + 32 * k, key = ch / (L::kRow / 16), part = ch % (L::kRow / 16);
            const int to = DH == 128 ? part ^ (key & 2) : part;
            cp_async16(st + kv * kGran * L::kRow + key * L::kRow + to * 16, src + ch * 16);
          }
        }
        if (lane < 8)
          cp_async16(st + 2 * kGran * L::kRow + lane * 16,
                     reinterpret_cast<const uint8_t*>(p.c.scale[lane >> 2] + row) + (lane & 3) * 16);
      }
      cp_commit();
    };
    int ahead = page_of(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int pg = ahead;
      ahead = page_of(i + 1);
      issue(i, pg);
    }
    int i = 0;
    bool begun = false;  // this warp's sums hold something of the unit
    do {
      for (const int stop = min(n, i + kWindow); i < stop; ++i) {
        cp_wait<kStages - 2>();
        __syncwarp();  // the granule has landed for every lane, and every lane is done with the stage refilled next
        const int pg = ahead;
        ahead = page_of(i + kStages);
        issue(i + kStages - 1, pg);
        const uint32_t st = ring + (i % kStages) * L::kStage;
        const int key0 = (first + i * kWarps) * kGran;
        // scores: keys g and g + 8, rows 2t and 2t + 1 of each block
        float s[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.0f;
        {
          uint32_t cw[2][CH / 8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = g + 8 * h;
            if constexpr (DH == 128) {
              const uint4 u = ld_shared_v4(st + key * L::kRow + ((t ^ (key & 2)) << 4));
              cw[h][0] = u.x; cw[h][1] = u.y; cw[h][2] = u.z; cw[h][3] = u.w;
            } else {
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(cw[h][0]), "=r"(cw[h][1]) : "r"(st + key * L::kRow + (t << 3)) : "memory");
            }
          }
#pragma unroll
          for (int k = 0; k < KS / 2; ++k) {
            const uint32_t a0[4] = {pair16<0>(cw[0][k]), pair16<0>(cw[1][k]), pair16<1>(cw[0][k]), pair16<1>(cw[1][k])};
            const uint32_t a1[4] = {pair16<2>(cw[0][k]), pair16<2>(cw[1][k]), pair16<3>(cw[0][k]), pair16<3>(cw[1][k])};
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              mma16816(s[b], a0, qb[b][2 * k][0], qb[b][2 * k][1]);
              mma16816(s[b], a1, qb[b][2 * k + 1][0], qb[b][2 * k + 1][1]);
            }
          }
        }
        // x = log2-domain scores
        uint32_t sk[2], sv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sk[h]) : "r"(st + 2 * kGran * L::kRow + (g + 8 * h) * 4) : "memory");
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sv[h]) : "r"(st + 2 * kGran * L::kRow + (kGran + g + 8 * h) * 4) : "memory");
        }
        const bool cut = key0 + kGran > lim_min;  // some row does not see some key of the granule
        bool grown = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = c * bf_lo(sk[h]), d = fmaf(-16.0f, a, c * bf_hi(sk[h]));
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaf(a, s[b][2 * h + e], d * qsum[b][e]);
              if (cut && key0 + g + 8 * h >= lim[b][e]) x = -INFINITY;
              s[b][2 * h + e] = x;
              grown |= x > m[b][e] + 8.0f;
            }
        }
        // O and the sums move to a new maximum only where it grew by more than 2^8 (P stays far below overflow)
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(m[b][e], fmaxf(s[b][e], s[b][2 + e]));
#pragma unroll
              for (int i2 = 4; i2 < 32; i2 *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i2));
              f[e] = mx == -INFINITY ? 1.0f : ex2(m[b][e] - mx);
              m[b][e] = mx;
              l[b][e] *= f[e];
              corr[b][e] *= f[e];
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[b][k][0] *= f[0];
              o[b][k][1] *= f[1];
              o[b][k][2] *= f[0];
              o[b][k][3] *= f[1];
            }
          }
        }
        uint32_t pb[NB][2], pl[NB][2];  // high and low parts
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float mu[2] = {m[b][0] == -INFINITY ? 0.0f : m[b][0], m[b][1] == -INFINITY ? 0.0f : m[b][1]};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(s[b][2 * h] - mu[0]), p1 = ex2(s[b][2 * h + 1] - mu[1]);
            l[b][0] += p0;
            l[b][1] += p1;
            float w0 = p0 * bf_lo(sv[h]), w1 = p1 * bf_lo(sv[h]), c0 = p0 * bf_hi(sv[h]), c1 = p1 * bf_hi(sv[h]);
            if (cut) {  // a key that the row does not see counts for nothing, whatever its scale holds
              if (key0 + g + 8 * h >= lim[b][0]) w0 = c0 = 0.0f;
              if (key0 + g + 8 * h >= lim[b][1]) w1 = c1 = 0.0f;
            }
            const uint32_t pk = pack_bf16x2(w0, w1);
            // what the two parts leave of P' is below 2^-17 of it: the sum of P' is taken as it is
            corr[b][0] += fmaf(8.0f, w0, c0);
            corr[b][1] += fmaf(8.0f, w1, c1);
            pb[b][h] = transpose8(pk);
            pl[b][h] = transpose8(pack_bf16x2(w0 - bf_lo(pk), w1 - bf_hi(pk)));
          }
        }
        // P V: keys 2t, 2t + 1 of both halves; this lane's DH/8 channels of each
        const uint32_t vst = st + kGran * L::kRow;
        constexpr int VW = DH / 64;  // words of DH/8 channels
        uint32_t v[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 8 * (e >> 1) + 2 * t + (e & 1);
          if constexpr (DH == 128)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[e][0]), "=r"(v[e][VW - 1])
                         : "r"(vst + key * L::kRow + (((g >> 1) ^ (key & 2)) << 4) + ((g & 1) << 3)) : "memory");
          else
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[e][0]) : "r"(vst + key * L::kRow + (g << 2)) : "memory");
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
          const uint32_t lo0 = __byte_perm(v[0][k], v[1][k], 0x5410), hi0 = __byte_perm(v[0][k], v[1][k], 0x7632);
          const uint32_t lo1 = __byte_perm(v[2][k], v[3][k], 0x5410), hi1 = __byte_perm(v[2][k], v[3][k], 0x7632);
          // tile 4k + i: channels 2i (its rows 0-7) and 2i + 1 (8-15) of the word, two keys to a register
          const uint32_t a0[4] = {centred(pair16<0>(lo0)), centred(pair16<0>(hi0)), centred(pair16<0>(lo1)),
                                  centred(pair16<0>(hi1))};
          const uint32_t a1[4] = {centred(pair16<1>(lo0)), centred(pair16<1>(hi0)), centred(pair16<1>(lo1)),
                                  centred(pair16<1>(hi1))};
          const uint32_t a2[4] = {centred(pair16<2>(lo0)), centred(pair16<2>(hi0)), centred(pair16<2>(lo1)),
                                  centred(pair16<2>(hi1))};
          const uint32_t a3[4] = {centred(pair16<3>(lo0)), centred(pair16<3>(hi0)), centred(pair16<3>(lo1)),
                                  centred(pair16<3>(hi1))};
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            mma16816(o[b][4 * k + 0], a0, pb[b][0], pb[b][1]);
            mma16816(o[b][4 * k + 1], a1, pb[b][0], pb[b][1]);
            mma16816(o[b][4 * k + 2], a2, pb[b][0], pb[b][1]);
            mma16816(o[b][4 * k + 3], a3, pb[b][0], pb[b][1]);
            mma16816(o[b][4 * k + 0], a0, pl[b][0], pl[b][1]);
            mma16816(o[b][4 * k + 1], a1, pl[b][0], pl[b][1]);
            mma16816(o[b][4 * k + 2], a2, pl[b][0], pl[b][1]);
            mma16816(o[b][4 * k + 3], a3, pl[b][0], pl[b][1]);
          }
        }
      }
      // To this warp's sums.  Lane (g, t) alone has rows 2t and 2t + 1 of each block, channels g*OC ...: tile k holds channels
      // 2k and 2k + 1 of them.  The row's sum of P and its maximum stand behind its channels.
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i2 = 4; i2 < 32; i2 *= 2) {
            l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], i2);
            corr[b][e] += __shfl_xor_sync(0xffffffffu, corr[b][e], i2);
          }
          float* const row = mine + (8 * b + 2 * t + e) * L::kLd;
          float f = 0.0f;  // a maximum of -infinity: no key so far, sums of zero (or NaN, which stay)
          if (begun && row[DH + 1] != -INFINITY) f = ex2(row[DH + 1] - m[b][e]);
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            float4* const dst = reinterpret_cast<float4*>(row + g * OC + 2 * k);
            float4 v = make_float4(o[b][k][e] + corr[b][e], o[b][k][2 + e] + corr[b][e], o[b][k + 1][e] + corr[b][e],
                                   o[b][k + 1][2 + e] + corr[b][e]);
            if (begun) {
              const float4 was = *dst;
              v = make_float4(fmaf(was.x, f, v.x), fmaf(was.y, f, v.y), fmaf(was.z, f, v.z), fmaf(was.w, f, v.w));
            }
            *dst = v;
            o[b][k][e] = o[b][k][2 + e] = o[b][k + 1][e] = o[b][k + 1][2 + e] = 0.0f;
          }
          const float sum = begun ? fmaf(row[DH], f, l[b][e]) : l[b][e];
          __syncwarp();  // every lane has read the row's old maximum
          if (g == 0) {
            row[DH] = sum;
            row[DH + 1] = m[b][e];
          }
          l[b][e] = corr[b][e] = 0.0f;
        }
      __syncwarp();
      begun = true;
    } while (i < n);
    cp_wait<0>();
    __syncthreads();
    // kTpr threads to a row, TC channels each
    {
      constexpr int kTpr = kThreadsFew / kRows, TC = DH / kTpr;
      const int row = threadIdx.x / kTpr, d0 = (threadIdx.x % kTpr) * TC;
      float mm = -INFINITY, ll = 0.0f, acc[TC];
#pragma unroll
      for (int k = 0; k < TC; ++k) acc[k] = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, sums[(x * kRows + row) * L::kLd + DH + 1]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float* const from = sums + (x * kRows + row) * L::kLd;
        const float f = mm == -INFINITY ? 0.0f : ex2(from[DH + 1] - mm);
        // a warp without a key for the row has l = 0 and O = 0 (m = -inf, f = 0), but NaN must not be lost
        ll += f * from[DH];
        const float* src = from + d0;
#pragma unroll
        for (int k = 0; k < TC; k += 4) {
          const float4 v4 = *reinterpret_cast<const float4*>(src + k);
          acc[k] = fmaf(f, v4.x, acc[k]);
          acc[k + 1] = fmaf(f, v4.y, acc[k + 1]);
          acc[k + 2] = fmaf(f, v4.z, acc[k + 2]);
          acc[k + 3] = fmaf(f, v4.w, acc[k + 3]);
        }
      }
      bool write = true;
      const int c0 = w.first_cta(), c1 = w.last_cta();
      if (c0 != c1) {
        const int slot = w.step == 0 ? 1 : 0;  // the unit's first part is its CTA's last run of steps
        float* dst = p.part + ((int64_t)blockIdx.x * 2 + slot) * few_part<DH>();
#pragma unroll
        for (int k = 0; k < TC; k += 4)
          __stcg(reinterpret_cast<float4*>(dst + row * DH + d0 + k), make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]));
        if (threadIdx.x % kTpr == 0) {
          __stcg(dst + kFewRows * DH + row, mm);
          __stcg(dst + kFewRows * DH + kFewRows + row, ll);
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(&p.cnt[c0], 1) == c1 - c0;
        __syncthreads();
        write = s_last != 0;
        if (write) {
          __threadfence();
          mm = -INFINITY;
          ll = 0.0f;
#pragma unroll
          for (int k = 0; k < TC; ++k) acc[k] = 0.0f;
          for (int x = c0; x <= c1; ++x) {
            const float* src = p.part + ((int64_t)x * 2 + (x == c0 ? 1 : 0)) * few_part<DH>();
            const float mx2 = __ldcg(src + kFewRows * DH + row), lx = __ldcg(src + kFewRows * DH + kFewRows + row);
            const float mn = fmaxf(mm, mx2);
            const float fo = mn == -INFINITY ? 0.0f : ex2(mm - mn), fn = mn == -INFINITY ? 0.0f : ex2(mx2 - mn);
            mm = mn;
            ll = ll * fo + lx * fn;
#pragma unroll
            for (int k = 0; k < TC; k += 4) {
              const float4 v4 = __ldcg(reinterpret_cast<const float4*>(src + row * DH + d0 + k));
              acc[k] = acc[k] * fo + v4.x * fn;
              acc[k + 1] = acc[k + 1] * fo + v4.y * fn;
              acc[k + 2] = acc[k + 2] * fo + v4.z * fn;
              acc[k + 3] = acc[k + 3] * fo + v4.w * fn;
            }
          }
        }
      }
      const int i = row0 + row;
      if (write && i < q.rows) {
        const int tok = i / tpr, hh = w.head * p.G + (i - tok * tpr);
        const size_t at = ((size_t)((int64_t)q.c0 * p.q_tokens + tok)) * p.H + hh;
        // no key: O = 0, LSE = -inf.  A row whose scores are NaN has m = -inf and l = NaN, and stays NaN.
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        __nv_bfloat16* dst = p.o + at * DH + d0;
#pragma unroll
        for (int k = 0; k < TC; k += 4)
          *reinterpret_cast<uint2*>(dst + k) = make_uint2(pack_bf16x2(acc[k] * inv, acc[k + 1] * inv), pack_bf16x2(acc[k + 2] * inv, acc[k + 3] * inv));
        if (p.lse && threadIdx.x % kTpr == 0) p.lse[at] = ll == 0.0f ? -INFINITY : (mm + lg2(ll)) * kLn2;
      }
    }
    __syncthreads();  // the sums become the next unit's
    more = w.next(p);
  }
}

template <int DH, int NB>
cudaError_t launch_few(const CacheAttnParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> optin_done{0};
  auto k = rocs_cache_few_kernel<DH, NB>;
  const cudaError_t e = ensure_smem_optin(optin_done, k, FewSmem<DH, NB>::kBuf);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreadsFew, FewSmem<DH, NB>::kBuf, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int cache_few_grid(int sms) { return 3 * sms; }
size_t cache_few_part_bytes(int dh) { return (size_t)(dh == 128 ? few_part<128>() : few_part<64>()) * sizeof(float); }

cudaError_t launch_cache_few(const CacheAttnParams& p, int dh, int rows, int grid, cudaStream_t st) {
  if (rows <= 8) return dh == 128 ? launch_few<128, 1>(p, grid, st) : launch_few<64, 1>(p, grid, st);
  return dh == 128 ? launch_few<128, 2>(p, grid, st) : launch_few<64, 2>(p, grid, st);
}

}  // namespace rocs
