// cache_few.cu -- attention over the paged 4-bit cache for few query rows (single tokens, a handful of candidates).
//
//   O_i = softmax_j(scale q_i . k_j) v_j,   k_j = mK_j + sK_j cK_j,   v_j = mV_j + sV_j cV_j      (codes c in 0..15)
//
// The codes go to the tensor core as they are: 16 + c is exact in bf16 (four mantissa bits under a leading one), so
//   q_i . k_j = sK_j (q_i . (16 + cK_j)) + (mK_j - 16 sK_j) sum(q_i)
//   O_i       = sum_j P'_ij (16 + cV_j) - 16 sum_j P'_ij + sum_j p_ij mV_j,     P'_ij = bf16(p_ij sV_j)
// and unpacking costs a shift and one three-input logic operation for two values.  Scores are exact up to fp32 sums;
// the one rounding to fewer bits is that of P' (it multiplies codes on the tensor core in bf16).
//
// With at most 16 rows to a pair of (request, key head) each 4-bit value is used 16 times at most: the bytes of the
// cache bound it.  mma.sync (16 rows x 8 keys) takes its operands from registers, so codes go from shared memory
// through the logic operations straight into fragments, with no second trip through shared memory as a tcgen05 operand
// tile would need, and 16 rows fill an instruction where a tcgen05 tile has at least 64.  Each warp takes 16 keys at a
// time through its own ring of cp.async stages (a 16-key granule never crosses a page) with its own running softmax:
// no block-wide synchronisation until the unit's end, where the four warps' results are joined in shared memory.
//
// Fragments without shuffles: the contraction index may be permuted freely as long as both operands agree.  Lane
// (g, t) = (lane / 4, lane % 4) owns channels t*DH/4 ... of key g in Q K^T (one 16-byte load), and channels
// g*DH/8 ... of its keys in P V, which leaves it with DH/4 contiguous channels of O for rows g and g + 8.
#include "cache_work.cuh"

namespace rocs {

namespace {

constexpr int kWarps = 4, kThreadsFew = kWarps * 32, kStages = 4, kGran = 16, kKeys = kWarps * kGran;

template <int DH>
struct FewSmem {
  static constexpr int kRow = DH / 2;                         // bytes of codes in a row
  static constexpr int kStage = 2 * kGran * kRow + 2 * kGran * 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = kWarps * kFewRows * (DH + 4) * 4;  // O of every warp (rows padded by 16 bytes)
  static constexpr int kBuf = kRing > kMerge ? kRing : kMerge;
};
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

template <int DH>
__global__ void __launch_bounds__(kThreadsFew, 3) rocs_cache_few_kernel(const __grid_constant__ CacheAttnParams p) {
  using L = FewSmem<DH>;
  constexpr int KS = DH / 16;   // contraction steps of Q K^T
  constexpr int NT = DH / 8;    // 8-channel tiles of O
  constexpr int CH = DH / 4;    // channels of a row that a lane holds
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][kFewRows], s_l[kWarps][kFewRows];
  __shared__ int64_t s_sum[33], s_out[3];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  Work<kKeys> w;
  if (!w.start(p, kFewRows, s_sum, s_out, 2)) return;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * L::kStage);
  // keys of a granule's half that this lane's score columns are (and its V rows): neighbours, in an order that spreads
  // the four lanes' V rows over all banks
  const int ka = (2 * t) ^ (t >> 1), kb = ka ^ 1;
  const float c = p.scale_log2;

  for (bool more = true; more;) {
    const Request& q = w.q;
    const int row0 = w.chunk * kFewRows, n_steps = w.count();
    const int tpr = p.G;  // rows of one token
    // Q fragments: rows g and g + 8, this lane's CH channels
    uint32_t qa[KS][4];
    float qsum[2];
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + g + 8 * i;
      lim[i] = row_limit(p, q, row);
      const int tok = row < q.rows ? row / tpr : 0, hh = w.head * p.G + (row < q.rows ? row - tok * tpr : 0);
      const int64_t token = (int64_t)q.c0 * p.q_tokens + tok;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + token * p.q_ld + (int64_t)hh * DH + t * CH);
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < CH / 8; ++k) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < q.rows) u = src[k];
        qa[2 * k][i] = u.x;
        qa[2 * k][2 + i] = u.y;
        qa[2 * k + 1][i] = u.z;
        qa[2 * k + 1][2 + i] = u.w;
        s += (bf_lo(u.x) + bf_hi(u.x)) + (bf_lo(u.y) + bf_hi(u.y)) + (bf_lo(u.z) + bf_hi(u.z)) + (bf_lo(u.w) + bf_hi(u.w));
      }
      qsum[i] = quad_sum(s);
    }
    int lim_min = min(lim[0], lim[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, corr[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k][i] = 0.0f;

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
    for (int i = 0; i < n; ++i) {
      cp_wait<kStages - 2>();
      __syncwarp();  // the granule has landed for every lane, and every lane is done with the stage refilled next
      const int pg = ahead;
      ahead = page_of(i + kStages);
      issue(i + kStages - 1, pg);
      const uint32_t st = ring + (i % kStages) * L::kStage;
      const int key0 = (first + i * kWarps) * kGran;
      // scores of 2 x 8 keys
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
        const int key = 8 * j + (g ^ ((g >> 2) & 1));
        uint32_t cw[CH / 8];
        if constexpr (DH == 128) {
          const uint4 u = ld_shared_v4(st + key * L::kRow + ((t ^ (key & 2)) << 4));
          cw[0] = u.x; cw[1] = u.y; cw[2] = u.z; cw[3] = u.w;
        } else {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(cw[0]), "=r"(cw[1]) : "r"(st + key * L::kRow + (t << 3)) : "memory");
        }
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          mma16816(s[j], qa[2 * k], pair16<0>(cw[k]), pair16<1>(cw[k]));
          mma16816(s[j], qa[2 * k + 1], pair16<2>(cw[k]), pair16<3>(cw[k]));
        }
      }
      // x = log2-domain scores; steps and minima of this lane's 4 keys
      uint32_t sk[4], sv[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = st + 2 * kGran * L::kRow + (8 * j + 2 * t) * 4;
        uint32_t a, b;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at) : "memory");
        sk[2 * j] = t < 2 ? a : b;
        sk[2 * j + 1] = t < 2 ? b : a;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at + kGran * 4) : "memory");
        sv[2 * j] = t < 2 ? a : b;
        sv[2 * j + 1] = t < 2 ? b : a;
      }
      const bool cut = key0 + kGran > lim_min;  // some row does not see some key of the granule
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = c * bf_lo(sk[2 * j + e]), b = fmaf(-16.0f, a, c * bf_hi(sk[2 * j + e]));
          const int key = key0 + 8 * j + (e ? kb : ka);
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            float x = fmaf(a, s[j][2 * i2 + e], b * qsum[i2]);
            if (cut && key >= lim[i2]) x = -INFINITY;
            s[j][2 * i2 + e] = x;
            mx[i2] = fmaxf(mx[i2], x);
          }
        }
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        mx[i2] = fmaxf(mx[i2], __shfl_xor_sync(0xffffffffu, mx[i2], 1));
        mx[i2] = fmaxf(mx[i2], __shfl_xor_sync(0xffffffffu, mx[i2], 2));
      }
      // O and the sums move to a new maximum only where it grew by more than 2^8 (P stays far below overflow)
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f)) {
        float f[2];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const float mn = fmaxf(m[i2], mx[i2]);
          f[i2] = mn == -INFINITY ? 1.0f : ex2(m[i2] - mn);
          m[i2] = mn;
          l[i2] *= f[i2];
          corr[i2] *= f[i2];
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          o[k][0] *= f[0];
          o[k][1] *= f[0];
          o[k][2] *= f[1];
          o[k][3] *= f[1];
        }
      }
      uint32_t pa[4];
      const float mu[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const float p0 = ex2(s[j][2 * i2] - mu[i2]), p1 = ex2(s[j][2 * i2 + 1] - mu[i2]);
          l[i2] += p0 + p1;
          float w0 = p0 * bf_lo(sv[2 * j]), w1 = p1 * bf_lo(sv[2 * j + 1]);
          float c0 = p0 * bf_hi(sv[2 * j]), c1 = p1 * bf_hi(sv[2 * j + 1]);
          if (cut) {  // a key that the row does not see counts for nothing, whatever its scale holds
            if (key0 + 8 * j + ka >= lim[i2]) w0 = c0 = 0.0f;
            if (key0 + 8 * j + kb >= lim[i2]) w1 = c1 = 0.0f;
          }
          const uint32_t pk = pack_bf16x2(w0, w1);
          pa[2 * j + i2] = pk;
          corr[i2] += fmaf(-16.0f, bf_lo(pk) + bf_hi(pk), c0 + c1);
        }
      // P V: keys ka, kb of both halves; this lane's DH/8 channels of each
      const uint32_t vst = st + kGran * L::kRow;
      constexpr int VW = DH / 64;  // words of DH/8 channels
      uint32_t v[4][VW];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = 8 * (e >> 1) + ((e & 1) ? kb : ka);
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
        mma16816(o[8 * k + 0], pa, pair16<0>(lo0), pair16<0>(lo1));
        mma16816(o[8 * k + 1], pa, pair16<0>(hi0), pair16<0>(hi1));
        mma16816(o[8 * k + 2], pa, pair16<1>(lo0), pair16<1>(lo1));
        mma16816(o[8 * k + 3], pa, pair16<1>(hi0), pair16<1>(hi1));
        mma16816(o[8 * k + 4], pa, pair16<2>(lo0), pair16<2>(lo1));
        mma16816(o[8 * k + 5], pa, pair16<2>(hi0), pair16<2>(hi1));
        mma16816(o[8 * k + 6], pa, pair16<3>(lo0), pair16<3>(lo1));
        mma16816(o[8 * k + 7], pa, pair16<3>(hi0), pair16<3>(hi1));
      }
    }
    cp_wait<0>();
    __syncthreads();  // the ring becomes the merge buffer
    // lane (g, t): tile n holds O of channels 2t*NT + n and (2t+1)*NT + n, rows g and g + 8
    float* mine = reinterpret_cast<float*>(smem) + warp * kFewRows * (DH + 4);
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
      l[i2] = quad_sum(l[i2]);
      corr[i2] = quad_sum(corr[i2]);
      float* dst = mine + (g + 8 * i2) * (DH + 4) + t * CH;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < NT; k += 4)
          *reinterpret_cast<float4*>(dst + e * NT + k) =
              make_float4(o[k][2 * i2 + e] + corr[i2], o[k + 1][2 * i2 + e] + corr[i2], o[k + 2][2 * i2 + e] + corr[i2],
                          o[k + 3][2 * i2 + e] + corr[i2]);
      if (t == 0) {
        s_m[warp][g + 8 * i2] = m[i2];
        s_l[warp][g + 8 * i2] = l[i2];
      }
    }
    __syncthreads();
    // 8 threads to a row, DH/8 channels each
    {
      constexpr int TC = DH / 8;
      const int row = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * TC;
      float mm = -INFINITY, ll = 0.0f, acc[TC];
#pragma unroll
      for (int k = 0; k < TC; ++k) acc[k] = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, s_m[x][row]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = mm == -INFINITY ? 0.0f : ex2(s_m[x][row] - mm);
        // a warp without a key for the row has l = 0 and O = 0 (m = -inf, f = 0), but NaN must not be lost
        ll += f * s_l[x][row];
        const float* src = reinterpret_cast<const float*>(smem) + (x * kFewRows + row) * (DH + 4) + d0;
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
        if ((threadIdx.x & 7) == 0) {
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
        for (int k = 0; k < TC; k += 8)
          st_global_v4(dst + k, pack_bf16x2(acc[k] * inv, acc[k + 1] * inv), pack_bf16x2(acc[k + 2] * inv, acc[k + 3] * inv),
                       pack_bf16x2(acc[k + 4] * inv, acc[k + 5] * inv), pack_bf16x2(acc[k + 6] * inv, acc[k + 7] * inv));
        if (p.lse && (threadIdx.x & 7) == 0) p.lse[at] = ll == 0.0f ? -INFINITY : (mm + lg2(ll)) * kLn2;
      }
    }
    __syncthreads();  // the merge buffer becomes the ring again
    more = w.next(p);
  }
}

template <int DH>
cudaError_t launch_few(const CacheAttnParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> optin_done{0};
  auto k = rocs_cache_few_kernel<DH>;
  const cudaError_t e = ensure_smem_optin(optin_done, k, FewSmem<DH>::kBuf);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreadsFew, FewSmem<DH>::kBuf, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int cache_few_grid(int sms) { return 3 * sms; }
size_t cache_few_part_bytes(int dh) { return (size_t)(dh == 128 ? few_part<128>() : few_part<64>()) * sizeof(float); }

cudaError_t launch_cache_few(const CacheAttnParams& p, int dh, int grid, cudaStream_t st) {
  return dh == 128 ? launch_few<128>(p, grid, st) : launch_few<64>(p, grid, st);
}

}  // namespace rocs
