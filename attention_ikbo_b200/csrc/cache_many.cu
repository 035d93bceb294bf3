// cache_many.cu -- attention over the paged 4-bit cache for many query rows (hundreds of candidates to a request).
//
//   O_i = softmax_j(scale q_i . k_j) v_j,   k_j = mK_j + sK_j cK_j,   v_j = mV_j + sV_j cV_j      (codes c in 0..15)
//
// Each 4-bit value is used by up to 256 rows, so the tensor core and the exponentials bound it.  Per K/V block of 128
// keys, from L2 once for both 128-row query tiles:
//   * K goes to the tensor core as 16 + c, exact in bf16 (four mantissa bits under a leading one; a shift and one logic
//     operation for two values), and the softmax applies the key's step and minimum to the fp32 product,
//         x_ij = a_j (q_i . (16 + c_j)) + b_j sum(q_i),   a_j = sK_j scale log2(e),  b_j = (mK_j - 16 sK_j) scale log2(e),
//     two packed FMAs for two scores where a plain softmax has one: scores are exact up to fp32 sums.  Rounding the
//     keys to bf16 instead would put 2^-9 of every product into the scores.
//   * V is rounded to bf16 once, as P is and as the output is: its error is a weighted mean of such roundings.
// Warp roles (512 threads): warp 0 loads query tiles by TMA, warp 1 issues tcgen05.mma, warps 4-7 and 8-11 are the
// softmax and the epilogue of query tiles A and B (S in TMEM; P in bf16 over S, the A operand of P V; O in TMEM), warps
// 12-15 turn codes into the tensor core's 128-byte-swizzled operand tiles: codes go from global memory into registers
// one block ahead, through the logic operations, into a ring of shared-memory slots in the order of their use.
// setmaxnreg moves registers to the softmax warps, which hold a row's 128 scores.
// Work is shared out by cache_work.cuh: equal runs of blocks, partial results merged by the last to finish.
//
// The rows of a tile are whole query tokens of the G heads that share the key head: row = token * G + head, 128 / G
// tokens to a tile, loaded as one box {64 channels, G heads, 128 / G tokens} for each half of the channels.
#include "cache_work.cuh"

namespace rocs {

namespace {

constexpr int kThreadsMany = 512, BM = 128, BN = 128;
constexpr int kSoftWarp = 4, kDeqWarp = 12;
constexpr int kSlots = 8;  // of the scale ring and the per-unit records: far more than the K/V ring lets run ahead
// 4 warpgroups launched at 128 registers a thread; the shares add up to what was launched
constexpr uint32_t kLaunchRegs = 128, kRegsCtl = 56, kRegsDeq = 88, kRegsSoft = 184;
static_assert(kRegsCtl + kRegsDeq + 2 * kRegsSoft == 4 * kLaunchRegs, "register split");

template <int DH>
struct ManySmem {
  static constexpr uint32_t kTile = BM * DH * 2;  // a query tile, or one block of K or V (bf16)
  static constexpr int kRing = DH == 128 ? 4 : 6;
  static constexpr uint32_t kStage = 32 * 64;     // per softmax warp: 32 rows x 32 columns of O (bf16)
  static constexpr uint32_t off_q = 0;
  static constexpr uint32_t off_ring = 2 * kTile;
  static constexpr uint32_t off_stage = off_ring + kRing * kTile;
  static constexpr uint32_t off_scale = off_stage + 8 * kStage;  // kSlots x 64 key pairs x {a0, a1, b0, b1}
  static constexpr uint32_t off_bar = off_scale + kSlots * BN * 8;
  static constexpr uint32_t n_bars = 2 * kRing + 2 * 8 + 1 + 2 * kSlots;
  static constexpr uint32_t off_misc = off_bar + n_bars * 8;
  static constexpr uint32_t alloc_bytes = off_misc + 64 + 1024;
  static_assert(alloc_bytes <= 232448 - 1024, "shared memory budget");
};
template <int DH>
constexpr int many_slab() { return 32 * (DH + 2); }  // floats of a partial result of 32 rows: O [dh/4][32][4], m, l

__device__ __forceinline__ void wait_ld_regs(uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]),
                 "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]), "+r"(a[31]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15]),
                 "+r"(b[16]), "+r"(b[17]), "+r"(b[18]), "+r"(b[19]), "+r"(b[20]), "+r"(b[21]), "+r"(b[22]), "+r"(b[23]),
                 "+r"(b[24]), "+r"(b[25]), "+r"(b[26]), "+r"(b[27]), "+r"(b[28]), "+r"(b[29]), "+r"(b[30]), "+r"(b[31])
               :
               : "memory");
}
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
  asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ void ld_shared_2x64(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

// One block of K or V on its way into a ring slot.
struct Item {
  int page0, page1;  // pages of this warp's two 16-key granules
  int key0, left;    // first key, keys of the history from there on
  int head;
  int flags;         // bit 0: V, 1: last block of the unit's run, 2: there is an item; from bit 4: unit
};

}  // namespace

template <int DH>
__global__ void __launch_bounds__(kThreadsMany, 1) rocs_cache_many_kernel(const __grid_constant__ CacheManyParams mp) {
  using L = ManySmem<DH>;
  constexpr int kRing = L::kRing;
  const CacheAttnParams& p = mp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem + L::off_q;
  uint8_t* s_ring = smem + L::off_ring;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t* ring_full = bars;
  uint64_t* ring_empty = bars + kRing;
  uint64_t* q_full = bars + 2 * kRing;  // [2] query tile landed
  uint64_t* q_empty = q_full + 2;       // [2] its last S computed and its rows' sums taken
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_empty = o_full + 2;
  uint64_t* s_free = o_empty + 2;    // [2] separate P: S read into registers
  uint64_t* pv_done = s_free + 2;    // [2] separate P: P V complete (P may be rewritten)
  uint64_t* drain_bar = pv_done + 2;
  uint64_t* sc_full = drain_bar + 1;      // [kSlots] steps and minima of a K block are there
  uint64_t* unit_done = sc_full + kSlots;  // [kSlots] all V blocks of a unit have been looked through
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::off_misc);
  int* s_abort = reinterpret_cast<int*>(smem + L::off_misc + 4);
  int* s_bad = reinterpret_cast<int*>(smem + L::off_misc + 16);  // [kSlots] first key of the unit whose V is not finite
  __shared__ int64_t s_sum[33], s_out[3];

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const Ctl ctl{s_abort, p.ws, (unsigned long long)mp.wait_limit_ns};
  const int tile_tokens = BM / p.G, tile_rows = tile_tokens * p.G;

  Work<BN> w;
  if (!w.start(p, 2 * tile_rows, s_sum, s_out, mp.min_share)) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 4);
      mbar_init(&ring_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1 + 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], 4);
      mbar_init(&s_free[x], 4);
      mbar_init(&pv_done[x], 1);
    }
    mbar_init(drain_bar, 1);
    for (int k = 0; k < kSlots; ++k) {
      mbar_init(&sc_full[k], 4);
      mbar_init(&unit_done[k], 4);
      s_bad[k] = 0x7fffffff;
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (tile_rows < BM) {  // rows that no query token fills
    for (uint32_t i = threadIdx.x; i < 2 * L::kTile / 16; i += kThreadsMany) reinterpret_cast<uint4*>(s_q)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  // TMEM columns: S_A [0,128) S_B [128,256) O_A [256,256+DH) O_B [256+DH,256+2DH).  dh = 128: P_X over S_X [0,64), so S
  // of the next block waits for P V.  dh = 64 leaves 128 columns free: P_A [384,448), P_B [448,512) of their own.
  constexpr bool kSepP = 256 + 2 * DH + 128 <= 512;
  constexpr uint32_t kPCol = 256 + 2 * DH;

  if (warp < kSoftWarp) {
    reg_dealloc<kRegsCtl>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------------ query tiles
      tma_prefetch_desc(&mp.tm_q);
      uint32_t ph[2] = {0, 0}, n[2] = {0, 0};
      bool ok = true;
      for (bool more = true; more && ok; more = w.next(p)) {
        if (w.q.L == 0) continue;
        const int row0 = w.chunk * 2 * tile_rows, nx = row0 + tile_rows < w.q.rows ? 2 : 1;
        const int tok0 = w.q.c0 * p.q_tokens + w.chunk * 2 * tile_tokens;
        for (int x = 0; x < nx; ++x) {
          if (!mbar_wait(&q_empty[x], ph[x] ^ 1, ctl, 941)) { ok = false; break; }
          ph[x] ^= 1;
          ++n[x];
          mbar_arrive_expect_tx(&q_full[x], (uint32_t)tile_rows * DH * 2);
#pragma unroll
          for (int cc = 0; cc < DH / 64; ++cc)
            tma_load_3d(s_q + x * L::kTile + cc * (BM * 128), &mp.tm_q, &q_full[x], cc * 64, w.head * p.G, tok0 + x * tile_tokens);
        }
      }
      if (!ok)
        for (int x = 0; x < 2; ++x)
          if (n[x]) mbar_drain(&q_full[x], (n[x] - 1) & 1, 20000000ull);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------------ tcgen05 issuer
      constexpr uint32_t idesc_s = idesc_bf16(BM, BN, false, false);  // S = Q (16 + c)^T: both K-major
      constexpr uint32_t idesc_o = idesc_bf16(BM, DH, false, true);   // O += P V: V is MN-major
      uint32_t rs = 0, rph = 0, qph = 0, pph = 0, oeph = 0, sfph = 0;  // phase bits of the two tiles
      bool s_pend[2] = {false, false}, b_pend = false;
      bool ok = true;
      const uint32_t q0 = smem_u32(s_q), ring0 = smem_u32(s_ring);
      uint32_t slot = 0;
      auto take = [&](int where) -> bool {  // the next ring slot, in order of use
        if (!mbar_wait(&ring_full[rs], rph, ctl, where)) return false;
        slot = rs;
        if (++rs == kRing) { rs = 0; rph ^= 1; }
        tc_fence_after();
        return true;
      };
      auto issue_s = [&](int x) -> bool {
        if (kSepP) {
          if (s_pend[x]) {
            if (!mbar_wait(&s_free[x], (sfph >> x) & 1, ctl, 942)) return false;
            sfph ^= 1u << x;
            tc_fence_after();
          }
          s_pend[x] = true;
        }
        const uint64_t ad = sdesc_sw128(q0 + x * L::kTile, 16, 1024), bd = sdesc_sw128(ring0 + slot * L::kTile, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          umma_ss(tmem_base + x * 128, sdesc_add(ad, (kk >> 2) * (BM * 128) + (kk & 3) * 32),
                  sdesc_add(bd, (kk >> 2) * (BN * 128) + (kk & 3) * 32), idesc_s, kk != 0);
        umma_commit(&s_full[x]);
        return true;
      };
      auto issue_pv = [&](int x, uint32_t vslot, bool first) -> bool {
        if (!mbar_wait(&p_full[x], (pph >> x) & 1, ctl, 943)) return false;
        pph ^= 1u << x;
        if (first) {  // O_x of the tile's last unit must have been read out
          if (!mbar_wait(&o_empty[x], ((oeph >> x) & 1) ^ 1, ctl, 944)) return false;
          oeph ^= 1u << x;
        }
        tc_fence_after();
        const uint64_t vd = sdesc_sw128(ring0 + vslot * L::kTile, BN * 128, 1024);
        const uint32_t pa = tmem_base + (kSepP ? kPCol + x * 64 : x * 128);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_ts(tmem_base + 256 + x * DH, pa + kk * 8, sdesc_add(vd, kk * 2048), idesc_o, (!first || kk != 0) ? 1u : 0u);
        if (kSepP) umma_commit(&pv_done[x]);
        return true;
      };
      for (bool more = true; more; more = w.next(p)) {
        if (w.q.L == 0) continue;
        const int nx = w.chunk * 2 * tile_rows + tile_rows < w.q.rows ? 2 : 1, n = w.count();
        for (int x = 0; x < nx && ok; ++x) {
          ok = mbar_wait(&q_full[x], (qph >> x) & 1, ctl, 945);
          qph ^= 1u << x;
        }
        if (!ok || !(ok = take(946))) break;
        for (int x = 0; x < nx && ok; ++x) ok = issue_s(x);
        if (!ok) break;
        umma_commit(&ring_empty[slot]);
        // a unit without tile B still waits for the end of B's last unit, so that no record of an older unit is reused
        if (nx == 2) b_pend = true;
        else if (b_pend) {
          if (!(ok = mbar_wait(&o_empty[1], ((oeph >> 1) & 1) ^ 1, ctl, 947))) break;
        }
        for (int j = 1; j < n && ok; ++j) {
          if (!(ok = take(948))) break;
          const uint32_t kslot = slot;
          if (kSepP) {  // S of the next block as soon as the softmax has read the current one, then P V
            for (int x = 0; x < nx && ok; ++x) ok = issue_s(x);
            if (!ok) break;
            umma_commit(&ring_empty[kslot]);
            if (!(ok = take(949))) break;
            const uint32_t vslot = slot;
            for (int x = 0; x < nx && ok; ++x) ok = issue_pv(x, vslot, j == 1);
            if (!ok) break;
            umma_commit(&ring_empty[vslot]);
          } else {
            if (!(ok = take(949))) break;
            const uint32_t vslot = slot;
            slot = kslot;
            for (int x = 0; x < nx && ok; ++x) ok = issue_pv(x, vslot, j == 1) && issue_s(x);
            if (!ok) break;
            umma_commit(&ring_empty[kslot]);
            umma_commit(&ring_empty[vslot]);
          }
        }
        if (!ok) break;
        for (int x = 0; x < nx; ++x) umma_commit(&q_empty[x]);
        if (!(ok = take(950))) break;
        const uint32_t vslot = slot;
        for (int x = 0; x < nx && ok; ++x) {
          ok = issue_pv(x, vslot, n == 1);
          if (ok) umma_commit(&o_full[x]);
        }
        if (!ok) break;
        umma_commit(&ring_empty[vslot]);
      }
      umma_commit(drain_bar);
      mbar_drain(drain_bar, 0, 50000000ull);
    }
  } else if (warp >= kDeqWarp) {
    // ------------------------------------------------------------------ codes to operand tiles
    reg_dealloc<kRegsDeq>();
    constexpr int PARTS = DH / 32;     // 16-byte parts of a row of codes
    constexpr int RPI = 32 / PARTS;    // rows of one load instruction
    constexpr int ITER = 32 / RPI;     // loads for this warp's 32 keys
    const int dw = warp - kDeqWarp, part = lane % PARTS, sub = lane / PARTS;
    const int page_mask = (1 << p.c.page_log2) - 1;
    const float cl = p.scale_log2;
    // blocks in the order of their use: K0, K1, V0, K2, V1, ..., V_last of every unit
    bool more = true;
    int n = 0, i = 0, unit = -1;
    auto unit_start = [&]() {
      while (more && w.q.L == 0) more = w.next(p);
      if (more) {
        n = w.count();
        i = 0;
        ++unit;
      }
    };
    unit_start();
    auto gen = [&](Item& it) {
      it.flags = 0;
      it.left = 0;
      if (!more) return;
      const int v = i > 0 && ((i & 1) == 0 || i == 2 * n - 1);
      const int j = i == 2 * n - 1 ? n - 1 : v ? i / 2 - 1 : (i + 1) / 2;
      it.key0 = (w.step + j) * BN;
      it.left = w.q.L - it.key0;
      it.head = w.head;
      it.flags = v | (i == 2 * n - 1 ? 2 : 0) | 4 | (unit << 4);
      const int32_t* t = p.table + (int64_t)w.r * p.max_pages;
      const int k0 = it.key0 + 32 * dw;
      it.page0 = 32 * dw < it.left ? t[k0 >> p.c.page_log2] : 0;
      it.page1 = 32 * dw + 16 < it.left ? t[(k0 + 16) >> p.c.page_log2] : 0;
      if (++i == 2 * n) {
        more = w.next(p);
        unit_start();
      }
    };
    auto load = [&](Item& it, uint4 (&c)[ITER], uint32_t& sc) {
      if (!(it.flags & 4)) return;
      if ((unsigned)it.page0 >= (unsigned)p.c.pages || (unsigned)it.page1 >= (unsigned)p.c.pages) {
        if (lane == 0) record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 951);
        if ((unsigned)it.page0 >= (unsigned)p.c.pages) it.page0 = 0;
        if ((unsigned)it.page1 >= (unsigned)p.c.pages) it.page1 = 0;
      }
      const int kv = it.flags & 1, k0 = it.key0 + 32 * dw;
      const int64_t row0 = (((int64_t)it.page0 * p.c.heads + it.head) << p.c.page_log2) + (k0 & page_mask);
      const int64_t row1 = (((int64_t)it.page1 * p.c.heads + it.head) << p.c.page_log2) + ((k0 + 16) & page_mask) - 16;
#pragma unroll
      for (int s = 0; s < ITER; ++s) {
        const int key = RPI * s + sub;
        c[s] = make_uint4(0, 0, 0, 0);
        if (32 * dw + key < it.left)
          c[s] = *reinterpret_cast<const uint4*>(p.c.codes[kv] + ((key < 16 ? row0 : row1) + key) * (DH / 2) + part * 16);
      }
      sc = 0;
      if (32 * dw + (int)lane < it.left)
        sc = *reinterpret_cast<const uint32_t*>(p.c.scale[kv] + ((int)lane < 16 ? row0 : row1) + lane);
    };
    uint32_t rs = 0, rph = 0, kord = 0;
    auto convert = [&](const Item& it, const uint4 (&c)[ITER], uint32_t sc) -> bool {
      if (!mbar_wait(&ring_empty[rs], rph ^ 1, ctl, 952)) return false;
      const uint32_t slot = smem_u32(s_ring) + rs * L::kTile;
      float st = __uint_as_float(sc << 16), mn = __uint_as_float(sc & 0xffff0000u);
      const int u = (it.flags >> 4) & (kSlots - 1);
      if (!(it.flags & 1)) {
        // a and b of this lane's key, in pairs {a0, a1, b0, b1}
        const uint32_t at = smem_u32(smem + L::off_scale) + (kord & (kSlots - 1)) * (BN * 8) + (16 * dw + (lane >> 1)) * 16 + (lane & 1) * 4;
        const float a = cl * st, b = fmaf(-16.0f, a, cl * mn);
        st_shared_u32(at, __float_as_uint(a));
        st_shared_u32(at + 8, __float_as_uint(b));
      } else {
        // a row with values that are not finite: zeros here, and NaN for the rows that see it (in the epilogue)
        const bool bad = !(fabsf(mn) + 15.0f * fabsf(st) <= 3.38e38f);
        const unsigned any = __ballot_sync(0xffffffffu, bad);
        if (any) {
          if (lane == 0) atomicMin(&s_bad[u], it.key0 + 32 * dw + __ffs(any) - 1);
          if (bad) sc = 0;
        }
      }
#pragma unroll
      for (int s = 0; s < ITER; ++s) {
        const int key = RPI * s + sub, row = 32 * dw + key;
        const uint32_t base = slot + (part >> 1) * (BN * 128) + row * 128;
        const uint32_t x4 = (part & 1) * 4, sw = row & 7;
        const uint32_t cw[4] = {c[s].x, c[s].y, c[s].z, c[s].w};
        if (!(it.flags & 1)) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared_v4(base + (((x4 + k) ^ sw) << 4), pair16<0>(cw[k]), pair16<1>(cw[k]), pair16<2>(cw[k]), pair16<3>(cw[k]));
        } else {
          const uint32_t rsc = __shfl_sync(0xffffffffu, sc, key);
          const uint32_t st2 = __byte_perm(rsc, rsc, 0x1010), mn2 = __byte_perm(rsc, rsc, 0x3232);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared_v4(base + (((x4 + k) ^ sw) << 4), value2(pair16<0>(cw[k]), st2, mn2), value2(pair16<1>(cw[k]), st2, mn2),
                         value2(pair16<2>(cw[k]), st2, mn2), value2(pair16<3>(cw[k]), st2, mn2));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (!(it.flags & 1)) mbar_arrive(&sc_full[kord & (kSlots - 1)]);
        if (it.flags & 2) {
          // the record of a unit four further on: its last reader is long done, its first writer not there yet
          if (dw == 0) s_bad[(u + 4) & (kSlots - 1)] = 0x7fffffff;
          mbar_arrive(&unit_done[u]);
        }
        mbar_arrive(&ring_full[rs]);
      }
      if (!(it.flags & 1)) ++kord;
      if (++rs == kRing) { rs = 0; rph ^= 1; }
      return true;
    };
    Item it0, it1, it2;
    uint4 c0[ITER], c1[ITER];
    uint32_t sc0 = 0, sc1 = 0;
    gen(it0);
    load(it0, c0, sc0);
    gen(it1);
    load(it1, c1, sc1);
    gen(it2);
    while (it0.flags & 4) {
      if (!convert(it0, c0, sc0)) break;
      it0 = it1;
#pragma unroll
      for (int s = 0; s < ITER; ++s) c0[s] = c1[s];
      sc0 = sc1;
      it1 = it2;
      load(it1, c1, sc1);
      gen(it2);
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    reg_alloc<kRegsSoft>();
    const int x = (warp - kSoftWarp) >> 2;  // 0: tile A, 1: tile B
    const int quarter = warp & 3;           // TMEM lanes 32*quarter .. +31
    const uint32_t t_lane = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_addr = tmem_base + t_lane + x * 128;
    const uint32_t p_addr = kSepP ? tmem_base + t_lane + kPCol + x * 64 : s_addr;
    const uint32_t o_addr = tmem_base + t_lane + 256 + x * DH;
    const uint32_t stage = smem_u32(smem + L::off_stage) + (warp - kSoftWarp) * L::kStage;
    const uint32_t scales = smem_u32(smem + L::off_scale);
    const int trow = 32 * quarter + (int)lane;
    const uint32_t qrow = smem_u32(s_q) + x * L::kTile + trow * 128;
    uint32_t kord = 0, unit = 0, qph = 0, sph = 0, oph = 0, n_sig = 0;
    bool ok = true;
    for (bool more = true; more; more = w.next(p)) {
      const Request& q = w.q;
      const int row0 = (w.chunk * 2 + x) * tile_rows, n = w.count();
      const bool row_ok = trow < tile_rows && row0 + trow < q.rows;
      // index of the row's (token, head) in the outputs, -1 for padding
      int at = -1, lim = q.L;
      if (row_ok) {
        const int tok = (row0 + trow) / p.G;
        at = (q.c0 * p.q_tokens + tok) * p.H + w.head * p.G + (row0 + trow - tok * p.G);
        if (p.key_limit) lim = min(lim, max(0, p.key_limit[q.c0 + tok / p.q_tokens]));
      }
      if (q.L == 0) {
        if (row_ok) {
#pragma unroll
          for (int k = 0; k < DH / 8; ++k) st_global_v4(p.o + (size_t)at * DH + 8 * k, 0u, 0u, 0u, 0u);
          if (p.lse) p.lse[at] = -INFINITY;
        }
        continue;
      }
      const int u = unit & (kSlots - 1), uph = (unit / kSlots) & 1;
      ++unit;
      if (x == 1 && row0 >= q.rows) {
        kord += n;
        continue;
      }
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      // sum of the row's query values
      if (!(ok = mbar_wait(&q_full[x], qph, ctl, 961))) break;
      qph ^= 1;
      float qs = 0.0f;
#pragma unroll
      for (int cc = 0; cc < DH / 64; ++cc)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 v = ld_shared_v4(qrow + cc * (BM * 128) + ((k ^ (trow & 7)) << 4));
          qs += ((bf_lo(v.x) + bf_hi(v.x)) + (bf_lo(v.y) + bf_hi(v.y))) + ((bf_lo(v.z) + bf_hi(v.z)) + (bf_lo(v.w) + bf_hi(v.w)));
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[x]);
      const uint64_t qs2 = pack2(qs, qs);

      float m_used = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j, ++kord) {
        const uint32_t sc = scales + (kord & (kSlots - 1)) * (BN * 8);
        if (!(ok = mbar_wait(&sc_full[kord & (kSlots - 1)], (kord / kSlots) & 1, ctl, 962))) break;
        if (!(ok = mbar_wait(&s_full[x], sph, ctl, 963))) break;
        sph ^= 1;
        tc_fence_after();
        const int key0 = (w.step + j) * BN;
        const bool careful = j == 0 || key0 + BN > lim_min;  // a first block, or one that some row does not see all of
        uint32_t sv[4][32];
        // first half of S, then the second half in flight while the first half's exponentials run
        const bool split_ld = !kSepP && !careful;
        tmem_ld32(s_addr, sv[0]);
        tmem_ld32(s_addr + 32, sv[1]);
        tmem_ld_wait();
        tmem_ld32(s_addr + 64, sv[2]);
        tmem_ld32(s_addr + 96, sv[3]);
        if (!split_ld) wait_ld_regs(sv[2], sv[3]);
        if constexpr (kSepP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[x]);
          if (n_sig > 0) {
            if (!(ok = mbar_wait(&pv_done[x], (n_sig - 1) & 1, ctl, 964))) break;
            tc_fence_after();
          }
        }
        uint64_t ls0 = 0, ls1 = 0;
        float mq[4];
        // O and the sum move to a new maximum (a block's first maximum needs no O yet)
        auto rescale = [&](float m_new) {
          const float f = m_new == -INFINITY ? 1.0f : ex2(m_used - m_new);
          l *= f;
          if (j > 0) {
            tmem_st_wait();
#pragma unroll 1
            for (int cc = 0; cc < DH / 32; ++cc) {
              uint32_t ov[32];
              tmem_ld32(o_addr + cc * 32, ov);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
              tmem_st32(o_addr + cc * 32, ov);
            }
          }
          m_used = m_new;
        };
        // P = exp2(x - m) over S.  The exponentials use the running maximum at once and the block's own maximum is
        // taken alongside; if a row's grows by more than 2^8 the block is done again after O has been rescaled
        // (rare).  Until then P <= 2^8, which bf16 and the fp32 sums hold.
        auto fast = [&](bool with_max) {
          const float nm = m_used == -INFINITY ? 0.0f : -m_used;
          const uint64_t nm2 = pack2(nm, nm);
          ls0 = 0;
          ls1 = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) mq[k] = -INFINITY;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            if (c4 == 2 && split_ld && with_max) wait_ld_regs(sv[2], sv[3]);
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint64_t a2, b2, xp, sp;
              ld_shared_2x64(sc + (c4 * 16 + k) * 16, a2, b2);
              asm("mov.b64 %0, {%1, %2};" : "=l"(sp) : "r"(sv[c4][2 * k]), "r"(sv[c4][2 * k + 1]));
              xp = fma2(sp, a2, fma2(b2, qs2, nm2));
              float x0, x1;
              unpack2(xp, x0, x1);
              if (with_max) mq[k & 3] = max3(mq[k & 3], x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              if (k & 1) ls1 = add2(ls1, pack2(p0, p1));
              else ls0 = add2(ls0, pack2(p0, p1));
              pk[k] = pack_bf16x2(p0, p1);
            }
            tmem_st16(p_addr + c4 * 16, pk);
          }
        };
        if (!careful) {
          fast(true);
          const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));  // relative to m_used
          if (__any_sync(0xffffffffu, mx > 8.0f)) {
            const float base = m_used == -INFINITY ? 0.0f : m_used;
            rescale(fmaxf(m_used, base + mx));
            fast(false);
          }
        } else {
          // scores in place, those of keys that the row does not see at -infinity
#pragma unroll
          for (int k = 0; k < 4; ++k) mq[k] = -INFINITY;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint64_t a2, b2, sp;
              ld_shared_2x64(sc + (c4 * 16 + k) * 16, a2, b2);
              asm("mov.b64 %0, {%1, %2};" : "=l"(sp) : "r"(sv[c4][2 * k]), "r"(sv[c4][2 * k + 1]));
              float x0, x1;
              unpack2(fma2(sp, a2, fma2(b2, qs2, 0)), x0, x1);
              if (key0 + c4 * 32 + 2 * k >= lim) x0 = -INFINITY;
              if (key0 + c4 * 32 + 2 * k + 1 >= lim) x1 = -INFINITY;
              mq[k & 3] = max3(mq[k & 3], x0, x1);
              sv[c4][2 * k] = __float_as_uint(x0);
              sv[c4][2 * k + 1] = __float_as_uint(x1);
            }
          const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
          if (__any_sync(0xffffffffu, mx > m_used + 8.0f)) rescale(fmaxf(m_used, mx));
          const float nm = m_used == -INFINITY ? 0.0f : -m_used;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float p0 = ex2(__uint_as_float(sv[c4][2 * k]) + nm), p1 = ex2(__uint_as_float(sv[c4][2 * k + 1]) + nm);
              ls0 = add2(ls0, pack2(p0, p1));
              pk[k] = pack_bf16x2(p0, p1);
            }
            tmem_st16(p_addr + c4 * 16, pk);
          }
        }
        float la, lb;
        unpack2(add2(ls0, ls1), la, lb);
        l += la + lb;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        ++n_sig;
      }
      if (!ok) break;
      if (!(ok = mbar_wait(&unit_done[u], uph, ctl, 965))) break;
      const bool poison = s_bad[u] < lim;  // the row sees a key whose V is not finite
      if (!(ok = mbar_wait(&o_full[x], oph, ctl, 966))) break;
      oph ^= 1;
      tc_fence_after();

      // A unit cut by the border of a run: each part leaves its unnormalised O, maxima and sums and counts itself in;
      // the last one (it waits for nobody) merges all parts in their order.
      const int cta0 = w.first_cta(), cta1 = w.last_cta(), slab = x * 4 + quarter;
      const float* parts = nullptr;
      if (cta0 != cta1) {
        constexpr int kSlab = many_slab<DH>();
        float* mine = p.part + (((int64_t)blockIdx.x * 2 + (w.step == 0 ? 1 : 0)) * 8 + slab) * kSlab;
#pragma unroll 1
        for (int cc = 0; cc < DH / 32; ++cc) {  // [column/4][row][4]: each store a contiguous 512 bytes
          uint32_t ov[32];
          tmem_ld32(o_addr + cc * 32, ov);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float4 v = make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]), __uint_as_float(ov[4 * k + 2]),
                                   __uint_as_float(ov[4 * k + 3]));
            if (poison) v = make_float4(NAN, NAN, NAN, NAN);
            __stcg(reinterpret_cast<float4*>(mine + ((cc * 8 + k) * 32 + lane) * 4), v);
          }
        }
        __stcg(mine + DH * 32 + lane, m_used);
        __stcg(mine + DH * 32 + 32 + lane, l);
        __threadfence();
        __syncwarp();
        int order = 0;
        if (lane == 0) order = atomicAdd(&p.cnt[cta0 * 8 + slab], 1);
        order = __shfl_sync(0xffffffffu, order, 0);
        if (order != cta1 - cta0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[x]);
          continue;
        }
        __threadfence();
        parts = p.part + ((int64_t)cta0 * 2 * 8 + slab) * kSlab;  // part of run c: + (c - cta0) * 2 * 8 slabs, the first one's + 8
        m_used = -INFINITY;
        l = 0.0f;
        for (int c = cta0; c <= cta1; ++c) {
          const float* src = parts + ((int64_t)(c - cta0) * 16 + (c == cta0 ? 8 : 0)) * kSlab + DH * 32 + lane;
          const float mc = __ldcg(src), lc = __ldcg(src + 32), mn = fmaxf(m_used, mc);
          l = l * (mn == -INFINITY ? 1.0f : ex2(m_used - mn)) + lc * (mn == -INFINITY ? 1.0f : ex2(mc - mn));
          m_used = mn;
        }
      }
      // no key seen: O = 0, LSE = -inf.  Scores that are NaN leave l = NaN, and stay NaN.
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      // 32 columns at a time through this warp's slab of shared memory, out in rows of 64 bytes
#pragma unroll 1
      for (int cc = 0; cc < DH / 32; ++cc) {
        uint32_t ov[32];
        if (!parts) {
          tmem_ld32(o_addr + cc * 32, ov);
          tmem_ld_wait();
        } else {
          constexpr int kSlab = many_slab<DH>();
#pragma unroll
          for (int k = 0; k < 32; ++k) ov[k] = 0;
          for (int c = cta0; c <= cta1; ++c) {
            const float* src = parts + ((int64_t)(c - cta0) * 16 + (c == cta0 ? 8 : 0)) * kSlab;
            const float f = m_used == -INFINITY ? 1.0f : ex2(__ldcg(src + DH * 32 + lane) - m_used);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src + ((cc * 8 + k) * 32 + lane) * 4));
              ov[4 * k] = __float_as_uint(fmaf(f, v.x, __uint_as_float(ov[4 * k])));
              ov[4 * k + 1] = __float_as_uint(fmaf(f, v.y, __uint_as_float(ov[4 * k + 1])));
              ov[4 * k + 2] = __float_as_uint(fmaf(f, v.z, __uint_as_float(ov[4 * k + 2])));
              ov[4 * k + 3] = __float_as_uint(fmaf(f, v.w, __uint_as_float(ov[4 * k + 3])));
            }
          }
        }
        __syncwarp();  // the slab's last rows have been read
        const float scale = poison ? NAN : inv;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_shared_v4(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4),
                       pack_bf16x2(__uint_as_float(ov[8 * k]) * scale, __uint_as_float(ov[8 * k + 1]) * scale),
                       pack_bf16x2(__uint_as_float(ov[8 * k + 2]) * scale, __uint_as_float(ov[8 * k + 3]) * scale),
                       pack_bf16x2(__uint_as_float(ov[8 * k + 4]) * scale, __uint_as_float(ov[8 * k + 5]) * scale),
                       pack_bf16x2(__uint_as_float(ov[8 * k + 6]) * scale, __uint_as_float(ov[8 * k + 7]) * scale));
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 8 * k + (int)(lane >> 2), to = __shfl_sync(0xffffffffu, at, row);
          const uint4 v = ld_shared_v4(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
          if (to >= 0) st_global_v4(p.o + (size_t)to * DH + cc * 32 + (lane & 3) * 8, v.x, v.y, v.z, v.w);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[x]);
      if (row_ok && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m_used + lg2(l)) * kLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int DH>
static cudaError_t launch_many(const CacheManyParams& p, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> optin_done{0};
  static std::atomic<int> regs_checked{0};
  auto k = rocs_cache_many_kernel<DH>;
  if (!regs_checked.load(std::memory_order_acquire)) {
    // the setmaxnreg split is only valid for the register count it was computed for
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, k) != cudaSuccess || fa.numRegs != (int)kLaunchRegs) return cudaErrorInvalidConfiguration;
    regs_checked.store(1, std::memory_order_release);
  }
  const cudaError_t e = ensure_smem_optin(optin_done, k, (int)ManySmem<DH>::alloc_bytes);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreadsMany, ManySmem<DH>::alloc_bytes, st>>>(p);
  return cudaGetLastError();
}

size_t cache_many_part_bytes(int dh) { return 8 * sizeof(float) * (size_t)(dh == 128 ? many_slab<128>() : many_slab<64>()); }

cudaError_t launch_cache_many(const CacheManyParams& p, int dh, int grid, cudaStream_t st) {
  return dh == 128 ? launch_many<128>(p, grid, st) : launch_many<64>(p, grid, st);
}

}  // namespace rocs
