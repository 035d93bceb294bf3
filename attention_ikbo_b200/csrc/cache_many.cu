// cache_many.cu -- attention over the paged 4-bit cache for many query rows (hundreds of candidates to a request).
//
//   O_i = softmax_j(scale q_i . k_j) v_j,   k_j = mK_j + sK_j cK_j,   v_j = mV_j + sV_j cV_j      (codes c in 0..15)
//
// Each 4-bit value is used by up to 256 rows, so the tensor core and the exponentials bound it.  Per K/V block of 128
// keys, from L2 once for both 128-row query tiles:
//   * K goes to the tensor core as 16 + c, exact in bf16 (four mantissa bits under a leading one; a shift and one logic
//     operation for two values).  With t_j = mK_j / sK_j - 16 the score is
//         x_ij = a_j (q_i . (16 + c_j) + t_j sum(q_i)),   a_j = sK_j scale log2(e).
//     The product t_j sum(q_i) is one more contraction step of the tensor core: both factors in three bf16 parts (24
//     bits), the six products that matter in six of its 16 columns.  So the softmax has one packed FMA for two scores,
//     as one without codes would have, and scores are exact up to fp32 sums.  Applying the minimum in the softmax
//     instead, a second packed FMA and twice the shared-memory reads, took 1016 us where this took 908 us (8 histories
//     of 4096-8192 keys, 4 heads, 8192 rows each); rounding the keys to bf16 would put 2^-9 of every product into the
//     scores.
//   * V is rounded to bf16 once, as P is and as the output is: its error is a weighted mean of such roundings.
//   * The tensor core cuts off what falls below its accumulator, always towards zero: with values of one sign O lost 0.0004
//     of itself in 131,072 keys and 0.008 in 2,000,000.  So a run over more than kWindow blocks of a unit goes through the
//     roles in windows, each with an O of its own, joined in fp32 in memory (the place of the run's partial result): 868 ->
//     874 us for the case above, whose runs have one window.  Windows made in the softmax loop itself took 905 us there.
// Warp roles (512 threads): warp 0 loads query tiles by TMA, warp 1 issues tcgen05.mma, warp 2 walks the work and copies
// codes, steps and minima into staging buffers (cp.async.bulk, one copy for each page), warps 4-7 and 8-11 are the
// softmax and the epilogue of query tiles A and B (S in TMEM; P in bf16 over S, the A operand of P V; O in TMEM), warps
// 12-15 turn staged codes into the tensor core's 128-byte-swizzled operand tiles, into a ring of slots in the order of
// their use.  setmaxnreg moves registers to the softmax warps.
// Work is shared out by cache_work.cuh: equal runs of blocks, partial results merged by the last to finish.
//
// What bounds it is what runs beside the tensor work (870-910 us for the case above, 0.55 of the bf16 rate; 205 us for 512
// candidates to each of 32 histories of 2048 keys with 8 heads): S products read all the shared-memory bandwidth there is
// and go first, so a block's conversion, some 200 instructions a warp, takes 1500 cycles, and the roles' code together does
// not fit the instruction cache, which is why conversion loops are rolled (unrolled: 1127 us) and load one row ahead.
//
// The rows of a tile are whole query tokens of the G heads that share the key head: row = token * G + head, 128 / G
// tokens to a tile, loaded as one box {64 channels, G heads, 128 / G tokens} for each half of the channels.
#include "cache_work.cuh"

namespace rocs {

namespace {

constexpr int kThreadsMany = 512, BM = 128, BN = 128;
constexpr int kSoftWarp = 4, kDeqWarp = 12;
constexpr int kRecs = 4;  // records of units on their way through the roles
constexpr int kWindow = 256;  // blocks of keys of a record, at most
// 4 warpgroups launched at 128 registers a thread; the shares add up to what was launched
constexpr uint32_t kLaunchRegs = 128, kRegsCtl = 64, kRegsDeq = 64, kRegsSoft = 192;
static_assert(kRegsCtl + kRegsDeq + 2 * kRegsSoft == 4 * kLaunchRegs, "register split");

// One unit's run of key blocks, or a window of it, as warp 2 hands it to the other roles.
struct Rec {
  int c0, rows, L, head;  // first candidate, query rows of the key head, keys of the history, key head
  int row0, step, n;      // first row of tile A, first block of 128 keys, blocks (-1: no more units)
  int cta0, cta1;         // CTAs whose runs hold blocks of the unit
  int bad;                // first key whose V is not finite
  int slot;               // place of the run's partial result: 1 for a unit's first part, 0 otherwise
  int window;             // 1: a window of the run came before, + 2: another comes behind
  int pad[4];
};

template <int DH>
struct ManySmem {
  static constexpr uint32_t kTile = BM * DH * 2;  // a query tile, or one block of K or V (bf16)
  static constexpr int kRing = DH == 128 ? 4 : 6;
  static constexpr int kStaged = DH == 128 ? 2 : 4;
  static constexpr uint32_t kStaging = BN * DH / 2 + BN * 4;  // codes, then steps and minima
  // A K block's a and t: a block is converted once the ring slot kRing items before it is free, at the earliest that of
  // the K block before the last (dh = 64: the one before that), whose S was issued after P of the block before it: four
  // (eight) slots are enough for both tiles' softmax to be done with the old one.
  static constexpr int kScales = DH == 128 ? 4 : 8;
  static constexpr uint32_t kAug = BM * 16;       // 8 columns of the extra contraction step; the other 8 are zeros
  static constexpr uint32_t off_q = 0;
  static constexpr uint32_t off_ring = 2 * kTile;
  static constexpr uint32_t off_staging = off_ring + kRing * kTile;
  static constexpr uint32_t off_aug_q = off_staging + kStaged * kStaging;
  static constexpr uint32_t off_aug_k = off_aug_q + 2 * kAug;
  static constexpr uint32_t off_zero = off_aug_k + kScales * kAug;
  static constexpr uint32_t off_scale = off_zero + kAug;  // kScales x 128 x a
  static constexpr uint32_t off_rec = off_scale + kScales * BN * 4;
  static constexpr uint32_t off_bar = off_rec + kRecs * sizeof(Rec);
  static constexpr uint32_t n_bars = 2 * kRing + 2 * 7 + 1 + kScales + 3 * kRecs + 2 * kStaged;
  static constexpr uint32_t off_misc = off_bar + n_bars * 8;
  static constexpr uint32_t alloc_bytes = off_misc + 16 + 1024;
  static_assert(alloc_bytes <= 232448 - 288, "shared memory budget");
};
template <int DH>
constexpr int many_slab() { return 32 * (DH + 2); }  // floats of a partial result of 32 rows: O [dh/4][32][4], m, l

// tcgen05.wait::ld that names the loaded registers, so that no use of them moves before it
__device__ __forceinline__ void wait_ld_regs(uint32_t (&a)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]), "+r"(a[22]), "+r"(a[23]),
                 "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]), "+r"(a[29]), "+r"(a[30]), "+r"(a[31])
               :
               : "memory");
}
// operand descriptor without swizzle, K-major: 8-row groups of 16-byte rows 128 bytes apart, the second 8 columns lbo on
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}
// x in three bf16 parts, most significant first, as bits
__device__ __forceinline__ void split3(float x, uint32_t& a, uint32_t& b, uint32_t& c) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  const float r = x - __bfloat162float(h);
  const __nv_bfloat16 m = __float2bfloat16_rn(r), l = __float2bfloat16_rn(r - __bfloat162float(m));
  a = __bfloat16_as_ushort(h);
  b = __bfloat16_as_ushort(m);
  c = __bfloat16_as_ushort(l);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ void ld_shared_2x64(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// A window's O (32 rows of a tile in TMEM), maxima and sums joined with those of the run's earlier windows, which stand in
// memory.  A function of its own, out of the softmax warps' way: inlined it slowed their loop by 4 % though it never ran.
template <int DH>
__device__ __noinline__ float2 join_window(uint32_t o_addr, const float* kept, float m, float l) {
  const int lane = threadIdx.x & 31;
  const float was_m = __ldcg(kept + DH * 32 + lane), m_new = fmaxf(was_m, m);
  float was_f = 0.0f, f = 1.0f;  // no key in either: sums of zero (or NaN, which stay)
  if (m_new > -INFINITY) {
    was_f = ex2(was_m - m_new);
    f = ex2(m - m_new);
  }
#pragma unroll 1
  for (int cc = 0; cc < DH / 16; ++cc) {
    uint32_t ov[16];
    tmem_ld16(o_addr + cc * 16, ov);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 was = __ldcg(reinterpret_cast<const float4*>(kept + ((cc * 4 + k) * 32 + lane) * 4));
      ov[4 * k] = __float_as_uint(fmaf(was.x, was_f, __uint_as_float(ov[4 * k]) * f));
      ov[4 * k + 1] = __float_as_uint(fmaf(was.y, was_f, __uint_as_float(ov[4 * k + 1]) * f));
      ov[4 * k + 2] = __float_as_uint(fmaf(was.z, was_f, __uint_as_float(ov[4 * k + 2]) * f));
      ov[4 * k + 3] = __float_as_uint(fmaf(was.w, was_f, __uint_as_float(ov[4 * k + 3]) * f));
    }
    tmem_st16(o_addr + cc * 16, ov);
  }
  tmem_st_wait();
  return make_float2(m_new, fmaf(__ldcg(kept + DH * 32 + 32 + lane), was_f, l * f));
}

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
  uint64_t* q_empty = q_full + 2;       // [2] its last S computed
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_empty = o_full + 2;
  uint64_t* qa_full = o_empty + 2;   // [2] the query rows' sums are there
  uint64_t* drain_bar = qa_full + 2;
  uint64_t* sc_full = drain_bar + 1;           // [kScales] steps and minima of a K block are there
  uint64_t* rec_full = sc_full + L::kScales;   // [kRecs]
  uint64_t* rec_empty = rec_full + kRecs;      // [kRecs] read by every role, and the unit's epilogues done
  uint64_t* rec_v = rec_empty + kRecs;         // [kRecs] all V blocks of the unit have been looked through
  uint64_t* st_full = rec_v + kRecs;           // [kStaged]
  uint64_t* st_empty = st_full + L::kStaged;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::off_misc);
  int* s_abort = reinterpret_cast<int*>(smem + L::off_misc + 4);
  volatile Rec* recs = reinterpret_cast<volatile Rec*>(smem + L::off_rec);
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
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], 4);
      mbar_init(&qa_full[x], 4);
    }
    mbar_init(drain_bar, 1);
    for (int k = 0; k < L::kScales; ++k) mbar_init(&sc_full[k], 4);
    for (int k = 0; k < kRecs; ++k) {
      mbar_init(&rec_full[k], 1);
      mbar_init(&rec_empty[k], 1 + 1 + 4 + 8);  // query tiles, issuer, conversion warps, softmax warps
      mbar_init(&rec_v[k], 4);  // conversion warps
    }
    for (int k = 0; k < L::kStaged; ++k) {
      mbar_init(&st_full[k], 1);
      mbar_init(&st_empty[k], 4);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (tile_rows < BM)  // rows that no query token fills
    for (uint32_t i = threadIdx.x; i < 2 * L::kTile / 16; i += kThreadsMany) reinterpret_cast<uint4*>(s_q)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < L::kAug / 16) reinterpret_cast<uint4*>(smem + L::off_zero)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  // TMEM columns: S_A [0,128) S_B [128,256) O_A [256,256+DH) O_B [256+DH,256+2DH); P_X over S_X [0,64), so S of the next
  // block waits for P V.
  int ri = 0;
  uint32_t rec_ph = 0;  // this role's place among the unit records
  // the next unit's record; null after the last one, or when a wait has run out
  auto next_rec = [&](int where) -> volatile Rec* {
    if (!mbar_wait(&rec_full[ri], rec_ph, ctl, where)) return nullptr;
    return recs[ri].n < 0 ? nullptr : &recs[ri];
  };
  auto rec_step = [&]() {
    if (++ri == kRecs) { ri = 0; rec_ph ^= 1; }
  };

  if (warp < kSoftWarp) {
    reg_dealloc<kRegsCtl>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------------ query tiles
      tma_prefetch_desc(&mp.tm_q);
      uint32_t ph[2] = {0, 0}, n[2] = {0, 0};
      bool ok = true;
      while (volatile Rec* r = next_rec(940)) {
        const int keys = r->L, nx = r->row0 + tile_rows < r->rows ? 2 : 1, head = r->head;
        const int tok0 = r->c0 * p.q_tokens + r->row0 / p.G;
        mbar_arrive(&rec_empty[ri]);
        rec_step();
        if (keys == 0) continue;
        for (int x = 0; x < nx && ok; ++x) {
          if (!(ok = mbar_wait_sleep<200>(&q_empty[x], ph[x] ^ 1, ctl, 941))) break;
          ph[x] ^= 1;
          ++n[x];
          mbar_arrive_expect_tx(&q_full[x], (uint32_t)tile_rows * DH * 2);
#pragma unroll
          for (int cc = 0; cc < DH / 64; ++cc)
            tma_load_3d(s_q + x * L::kTile + cc * (BM * 128), &mp.tm_q, &q_full[x], cc * 64, head * p.G, tok0 + x * tile_tokens);
        }
        if (!ok) break;
      }
      if (ctl.aborted())
        for (int x = 0; x < 2; ++x)
          if (n[x]) mbar_drain(&q_full[x], (n[x] - 1) & 1, 20000000ull);
    } else if (warp == 2) {
      // ------------------------------------------------------------------ work, codes
      int si = 0, n_issued = 0;
      uint32_t sph = 0;
      const int page = 1 << p.c.page_log2;
      const bool mine = lane < 8 && (lane * 16 & (page - 1)) == 0;  // a page starts at this lane's 16 keys of the block
      const uint32_t code_bytes = page * (DH / 2), scale_bytes = page * 4;
      const uint32_t staging = smem_u32(smem + L::off_staging);
      bool ok = true;
      int from = 0;  // blocks of the run that earlier windows have taken
      for (bool more = true; more && ok;) {
        if (!(ok = mbar_wait_sleep<200>(&rec_empty[ri], rec_ph ^ 1, ctl, 952))) break;
        const int left = w.count() - from, n = min(left, kWindow), first = w.step + from, keys = w.q.L;
        if (lane == 0) {
          volatile Rec& r = recs[ri];
          r.c0 = w.q.c0;
          r.rows = w.q.rows;
          r.L = keys;
          r.head = w.head;
          r.row0 = w.chunk * 2 * tile_rows;
          r.step = first;
          r.n = n;
          r.cta0 = w.first_cta();
          r.cta1 = w.last_cta();
          r.bad = 0x7fffffff;
          r.slot = w.step == 0 ? 1 : 0;
          r.window = (from > 0 ? 1 : 0) | (n < left ? 2 : 0);
          mbar_arrive(&rec_full[ri]);
        }
        rec_step();
        const int32_t* table = p.table + (int64_t)w.r * p.max_pages;
        auto page_at = [&](int j) {
          const int key = (first + j) * BN + (int)lane * 16;
          return j < n && mine && key < keys ? table[key >> p.c.page_log2] : 0;
        };
        auto copy = [&](int kv, int j, int pg) -> bool {
          if (!mbar_wait_sleep<200>(&st_empty[si], sph ^ 1, ctl, 953)) return false;
          const int key = (first + j) * BN + (int)lane * 16;
          const bool go = mine && key < keys;
          if (go && (unsigned)pg >= (unsigned)p.c.pages) {
            record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 951);
            pg = 0;
          }
          const uint32_t count = __popc(__ballot_sync(0xffffffffu, go));
          if (lane == 0) mbar_arrive_expect_tx(&st_full[si], count * (code_bytes + scale_bytes));
          __syncwarp();
          if (go) {
            const int64_t row = ((int64_t)pg * p.c.heads + w.head) << p.c.page_log2;
            const uint32_t dst = staging + si * L::kStaging;
            bulk_load(dst + lane * 16 * (DH / 2), p.c.codes[kv] + row * (DH / 2), code_bytes, &st_full[si]);
            bulk_load(dst + BN * (DH / 2) + lane * 64, p.c.scale[kv] + row, scale_bytes, &st_full[si]);
          }
          ++n_issued;
          if (++si == L::kStaged) { si = 0; sph ^= 1; }
          return true;
        };
        // blocks in the order of their use: K0, K1, V0, K2, V1, ..., V_last
        int now = 0, next = page_at(0);
        for (int j = 0; j < n && keys > 0 && ok; ++j) {
          const int before = now;
          now = next;
          next = page_at(j + 1);
          ok = copy(0, j, now) && (j == 0 || copy(1, j - 1, before));
        }
        if (ok && keys > 0) ok = copy(1, n - 1, now);
        from += n;
        if (n == left) {
          from = 0;
          more = w.next(p);
        }
      }
      if (ok && mbar_wait_sleep<200>(&rec_empty[ri], rec_ph ^ 1, ctl, 954) && lane == 0) {
        recs[ri].n = -1;
        mbar_arrive(&rec_full[ri]);
      }
      if (ctl.aborted())
        for (int k = n_issued > L::kStaged ? n_issued - L::kStaged : 0; k < n_issued; ++k)
          mbar_drain(&st_full[k % L::kStaged], (k / L::kStaged) & 1, 20000000ull);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------------ tcgen05 issuer
      constexpr uint32_t idesc_s = idesc_bf16(BM, BN, false, false);  // S = Q (16 + c)^T: both K-major
      constexpr uint32_t idesc_o = idesc_bf16(BM, DH, false, true);   // O += P V: V is MN-major
      uint32_t rs = 0, rph = 0, qph = 0, pph = 0, oeph = 0;  // phase bits of the two tiles
      uint32_t kord = 0;
      bool ok = true;
      const uint32_t q0 = smem_u32(s_q), ring0 = smem_u32(s_ring), aug_q = smem_u32(smem + L::off_aug_q);
      const uint32_t aug_k = smem_u32(smem + L::off_aug_k), zero = smem_u32(smem + L::off_zero);
      uint32_t slot = 0;
      auto take = [&](int where) -> bool {  // the next ring slot, in order of use
        if (!mbar_wait(&ring_full[rs], rph, ctl, where)) return false;
        slot = rs;
        if (++rs == kRing) { rs = 0; rph ^= 1; }
        tc_fence_after();
        return true;
      };
      auto issue_s = [&](int x) {
        const uint64_t ad = sdesc_sw128(q0 + x * L::kTile, 16, 1024), bd = sdesc_sw128(ring0 + slot * L::kTile, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          umma_ss(tmem_base + x * 128, sdesc_add(ad, (kk >> 2) * (BM * 128) + (kk & 3) * 32),
                  sdesc_add(bd, (kk >> 2) * (BN * 128) + (kk & 3) * 32), idesc_s, kk != 0);
        const uint32_t qa = aug_q + x * L::kAug, ka = aug_k + (kord % L::kScales) * L::kAug;
        umma_ss(tmem_base + x * 128, sdesc_plain(qa, zero - qa), sdesc_plain(ka, zero - ka), idesc_s, 1u);
        umma_commit(&s_full[x]);
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
        const uint32_t pa = tmem_base + x * 128;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_ts(tmem_base + 256 + x * DH, pa + kk * 8, sdesc_add(vd, kk * 2048), idesc_o, (!first || kk != 0) ? 1u : 0u);
        return true;
      };
      while (volatile Rec* r = next_rec(955)) {
        const int keys = r->L, nx = r->row0 + tile_rows < r->rows ? 2 : 1, n = r->n;
        mbar_arrive(&rec_empty[ri]);
        rec_step();
        if (keys == 0) continue;
        for (int x = 0; x < nx && ok; ++x) {
          ok = mbar_wait(&q_full[x], (qph >> x) & 1, ctl, 945) && mbar_wait(&qa_full[x], (qph >> x) & 1, ctl, 947);
          qph ^= 1u << x;
        }
        if (!ok || !(ok = take(946))) break;
        for (int x = 0; x < nx; ++x) issue_s(x);
        umma_commit(&ring_empty[slot]);
        ++kord;
        for (int j = 1; j < n && ok; ++j, ++kord) {
          if (!(ok = take(948))) break;
          const uint32_t kslot = slot;
          if (!(ok = take(949))) break;
          const uint32_t vslot = slot;
          slot = kslot;
          for (int x = 0; x < nx && ok; ++x) {
            ok = issue_pv(x, vslot, j == 1);
            if (ok) issue_s(x);
          }
          if (!ok) break;
          umma_commit(&ring_empty[kslot]);
          umma_commit(&ring_empty[vslot]);
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
    // this lane's part of a row and row of a load: the 8 lanes of a 16-byte store's phase are four rows and the two parts
    // of one 128-byte half, which the swizzle spreads over all banks
    const int dw = warp - kDeqWarp;
    const int part = DH == 128 ? (lane & 1) | ((lane >> 2) & 2) : lane & 1;
    const int sub = DH == 128 ? ((lane >> 1) & 3) | ((lane >> 2) & 4) : lane >> 1;
    const uint32_t staging = smem_u32(smem + L::off_staging), scales = smem_u32(smem + L::off_scale), ring = smem_u32(s_ring);
    const float cl = p.scale_log2;
    uint32_t rs = 0, rph = 0, si = 0, sph = 0, kord = 0, qph = 0;
    const int trow = 32 * dw + (int)lane;
    bool ok = true;
    while (ok) {
      volatile Rec* r = next_rec(956);
      if (!r) break;
      const int step = r->step, n = r->n, keys = r->L, rec = ri, nx = r->row0 + tile_rows < r->rows ? 2 : 1;
      __syncwarp();
      if (lane == 0) {
        // every use of a record turns rec_v's phase, for a unit without keys too: its readers count uses of the record
        if (keys == 0) mbar_arrive(&rec_v[ri]);
        mbar_arrive(&rec_empty[ri]);
      }
      rec_step();
      if (keys == 0) continue;
      for (int i = 0; i < 2 * n; ++i) {
        const bool v = i > 0 && ((i & 1) == 0 || i == 2 * n - 1);
        const int j = i == 2 * n - 1 ? n - 1 : v ? i / 2 - 1 : (i + 1) / 2;
        const int key0 = (step + j) * BN + 32 * dw, left = keys - key0;  // this warp's 32 keys, and how many there are
        if (!(ok = mbar_wait_sleep<100>(&st_full[si], sph, ctl, 957))) break;
        const uint32_t src = staging + si * L::kStaging;
        uint32_t sc;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc) : "r"(src + BN * (DH / 2) + (32 * dw + lane) * 4) : "memory");
        if ((int)lane >= left) sc = 0;  // places past the history: codes are always finite, a zero step makes zeros of V
        if (!(ok = mbar_wait_sleep<100>(&ring_empty[rs], rph ^ 1, ctl, 958))) break;
        const uint32_t slot = ring + rs * L::kTile + (part >> 1) * (BN * 128) + (32 * dw + sub) * 128;
        const uint32_t codes = src + (32 * dw + sub) * (DH / 2) + part * 16;
        uint4 nx4 = ld_shared_v4(codes);
        if (!v) {
          // a and t of this lane's key.  A step of zero, or too small to count beside its minimum, is taken as a tiny one:
          // then t carries the minimum alone.
          float st = bf_lo(sc);
          const float mn = bf_hi(sc), least = fmaxf(fabsf(mn) * 8.673617e-19f, 7.888609e-31f);  // 2^-60, 2^-100
          if (fabsf(st) < least) st = least;
          uint32_t t1, t2, t3;
          split3(mn / st - 16.0f, t1, t2, t3);
          st_shared_u32(scales + ((kord % L::kScales) * BN + trow) * 4, __float_as_uint(cl * st));
          st_shared_v4(smem_u32(smem + L::off_aug_k) + (kord % L::kScales) * L::kAug + trow * 16, t1 | t2 << 16, t3 | t1 << 16,
                       t2 | t1 << 16, 0u);
#pragma unroll 1
          for (int s = 0; s < ITER; ++s) {
            const uint4 c = nx4;
            if (s + 1 < ITER) nx4 = ld_shared_v4(codes + (s + 1) * RPI * (DH / 2));
            const uint32_t cw[4] = {c.x, c.y, c.z, c.w}, sw = (RPI * s + sub) & 7;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4(slot + s * RPI * 128 + ((((part & 1) << 2 | k) ^ sw) << 4), pair16<0>(cw[k]), pair16<1>(cw[k]), pair16<2>(cw[k]),
                           pair16<3>(cw[k]));
          }
        } else {
          // a row with values that are not finite: zeros here, and NaN for the rows that see it (in the epilogue).  Its values
          // lie between the minimum and 15 steps above it; bf16 holds what is below 0x1.ffp127.
          const float mn = bf_hi(sc), end = fmaf(15.0f, bf_lo(sc), mn);
          const bool bad = !(fabsf(mn) < 0x1.ffp127f && fabsf(end) < 0x1.ffp127f);
          const unsigned any = __ballot_sync(0xffffffffu, bad);
          if (any) {
            if (lane == 0) atomicMin(const_cast<int*>(&recs[rec].bad), key0 + __ffs(any) - 1);
            if (bad) sc = 0;
          }
#pragma unroll 1
          for (int s = 0; s < ITER; ++s) {
            const uint4 c = nx4;
            if (s + 1 < ITER) nx4 = ld_shared_v4(codes + (s + 1) * RPI * (DH / 2));
            const uint32_t cw[4] = {c.x, c.y, c.z, c.w}, sw = (RPI * s + sub) & 7;
            const uint32_t rsc = __shfl_sync(0xffffffffu, sc, RPI * s + sub);
            const uint32_t st2 = __byte_perm(rsc, rsc, 0x1010), mn2 = __byte_perm(rsc, rsc, 0x3232);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared_v4(slot + s * RPI * 128 + ((((part & 1) << 2 | k) ^ sw) << 4), value2(pair16<0>(cw[k]), st2, mn2),
                           value2(pair16<1>(cw[k]), st2, mn2), value2(pair16<2>(cw[k]), st2, mn2), value2(pair16<3>(cw[k]), st2, mn2));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&st_empty[si]);
          if (!v) mbar_arrive(&sc_full[kord % L::kScales]);
          if (i == 2 * n - 1) mbar_arrive(&rec_v[rec]);
          mbar_arrive(&ring_full[rs]);
        }
        if (!v) ++kord;
        if (++rs == kRing) { rs = 0; rph ^= 1; }
        if (++si == L::kStaged) { si = 0; sph ^= 1; }
        if (i > 0) continue;
        // after a unit's first K block: sums of the query rows, the other factor of the extra contraction step
        for (int x = 0; x < nx && ok; ++x) {
          if (!(ok = mbar_wait_sleep<100>(&q_full[x], (qph >> x) & 1, ctl, 959))) break;
          qph ^= 1u << x;
          const uint32_t qrow = smem_u32(s_q) + x * L::kTile + trow * 128;
          float qs = 0.0f;
#pragma unroll 1
          for (int cc = 0; cc < DH / 64; ++cc)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 u = ld_shared_v4(qrow + cc * (BM * 128) + ((k ^ (trow & 7)) << 4));
              qs += ((bf_lo(u.x) + bf_hi(u.x)) + (bf_lo(u.y) + bf_hi(u.y))) + ((bf_lo(u.z) + bf_hi(u.z)) + (bf_lo(u.w) + bf_hi(u.w)));
            }
          uint32_t q1, q2, q3;
          split3(qs, q1, q2, q3);
          st_shared_v4(smem_u32(smem + L::off_aug_q) + x * L::kAug + trow * 16, q1 | q1 << 16, q1 | q2 << 16, q2 | q3 << 16, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&qa_full[x]);
        }
        if (!ok) break;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    reg_alloc<kRegsSoft>();
    const int x = (warp - kSoftWarp) >> 2;  // 0: tile A, 1: tile B
    const int quarter = warp & 3;           // TMEM lanes 32*quarter .. +31
    const uint32_t t_lane = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_addr = tmem_base + t_lane + x * 128;
    const uint32_t o_addr = tmem_base + t_lane + 256 + x * DH;
    const uint32_t scales = smem_u32(smem + L::off_scale);
    const int trow = 32 * quarter + (int)lane;
    uint32_t kord = 0, sph = 0, oph = 0;
    bool ok = true;
    while (ok) {
      volatile Rec* const r = next_rec(960);
      if (!r) break;
      const int rec = ri, v_ph = rec_ph, n = r->n, step = r->step;
      const int row0 = r->row0 + x * tile_rows;
      rec_step();
      // index of the row's (token, head) in the outputs, -1 for padding
      int at = -1, lim = r->L;
      const bool empty = lim == 0;
      if (trow < tile_rows && row0 + trow < r->rows) {
        const int tok = (row0 + trow) / p.G;
        at = (r->c0 * p.q_tokens + tok) * p.H + r->head * p.G + (row0 + trow - tok * p.G);
        if (p.key_limit) lim = min(lim, max(0, p.key_limit[r->c0 + tok / p.q_tokens]));
      }
      if (empty) {
        if (at >= 0) {
#pragma unroll
          for (int k = 0; k < DH / 8; ++k) st_global_v4(p.o + (size_t)at * DH + 8 * k, 0u, 0u, 0u, 0u);
          if (p.lse) p.lse[at] = -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_empty[rec]);
        continue;
      }
      if (x == 1 && row0 >= r->rows) {
        kord += n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&rec_empty[rec]);
        continue;
      }
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      float m_used = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j, ++kord) {
        const uint32_t sc = scales + (kord % L::kScales) * (BN * 4);
        if (!(ok = mbar_wait(&sc_full[kord % L::kScales], (kord / L::kScales) & 1, ctl, 962))) break;
        if (!(ok = mbar_wait(&s_full[x], sph, ctl, 963))) break;
        sph ^= 1;
        tc_fence_after();
        const int left = lim - (step + j) * BN;            // keys of the block that the row sees
        const bool cut = (step + j + 1) * BN > lim_min;   // some row does not see all of the block
        // P = exp2(x - m) over S.  Mostly the exponentials use the running maximum m as it stands: P may grow to 2^20
        // and the sums with it, which fp32 and bf16 hold without loss.  The first block of a run, one that some row does
        // not see all of, and one where a row's sum passes that bound (rare; S is put back first) take the careful way:
        // the maximum first, O and the sum moved to it where it grew by more than 2^8, then the exponentials.  It reads S
        // in quarters from TMEM, in rolled loops: P of quarter c lies over quarter c / 2, so quarters in order never
        // overwrite an unread one.
        bool careful = j == 0 || cut;
        float sum = 0.0f;
        if (!careful) {
          const float nm = -m_used;
          const uint64_t nm2 = pack2(nm, nm);
          uint32_t sv[4][32];
          tmem_ld32(s_addr, sv[0]);
          tmem_ld32(s_addr + 32, sv[1]);
          wait_ld_regs(sv[0]);
          wait_ld_regs(sv[1]);
          tmem_ld32(s_addr + 64, sv[2]);  // in flight while the first half's exponentials run
          tmem_ld32(s_addr + 96, sv[3]);
          uint64_t ls[2] = {0, 0};
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            if (c4 == 2) {
              wait_ld_regs(sv[2]);
              wait_ld_regs(sv[3]);
            }
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint64_t a2[2];
              ld_shared_2x64(sc + (c4 * 8 + k) * 16, a2[0], a2[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint64_t sp;
                asm("mov.b64 %0, {%1, %2};" : "=l"(sp) : "r"(sv[c4][4 * k + 2 * e]), "r"(sv[c4][4 * k + 2 * e + 1]));
                float x0, x1;
                unpack2(fma2(sp, a2[e], nm2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                ls[e] = add2(ls[e], pack2(p0, p1));
                pk[2 * k + e] = pack_bf16x2(p0, p1);
              }
            }
            tmem_st16(s_addr + c4 * 16, pk);
          }
          float la, lb;
          unpack2(add2(ls[0], ls[1]), la, lb);
          sum = la + lb;
          careful = __any_sync(0xffffffffu, sum > 1048576.0f || m_used == -INFINITY);
          if (careful) {
            tmem_st_wait();
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) tmem_st32(s_addr + c4 * 32, sv[c4]);
            tmem_st_wait();
          }
        }
        if (careful) {
          uint32_t s[32];
          auto scores = [&](int c4, float nm, float (&xs)[32]) {  // of quarter c4, relative to m; not seen: -infinity
            tmem_ld32(s_addr + c4 * 32, s);
            wait_ld_regs(s);
            const uint64_t nm2 = pack2(nm, nm);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint64_t a2[2];
              ld_shared_2x64(sc + (c4 * 8 + k) * 16, a2[0], a2[1]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint64_t sp;
                asm("mov.b64 %0, {%1, %2};" : "=l"(sp) : "r"(s[4 * k + 2 * e]), "r"(s[4 * k + 2 * e + 1]));
                unpack2(fma2(sp, a2[e], nm2), xs[4 * k + 2 * e], xs[4 * k + 2 * e + 1]);
              }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c4 * 32 + k >= left) xs[k] = -INFINITY;
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            float xs[32], mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            scores(c4, 0.0f, xs);
#pragma unroll
            for (int k = 0; k < 16; ++k) mq[k & 3] = max3(mq[k & 3], xs[2 * k], xs[2 * k + 1]);
            mx = fmaxf(mx, fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])));
          }
          if (__any_sync(0xffffffffu, mx > m_used + 8.0f)) {
            const float m_new = fmaxf(m_used, mx), f = m_new == -INFINITY ? 1.0f : ex2(m_used - m_new);
            m_used = m_new;
            l *= f;
            if (j > 0) {  // before the first P V there is no O
              uint32_t v[16];
#pragma unroll 1
              for (int cc = 0; cc < DH / 16; ++cc) {
                tmem_ld16(o_addr + cc * 16, v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                tmem_st16(o_addr + cc * 16, v);
              }
            }
          }
          const float nm = m_used == -INFINITY ? 0.0f : -m_used;
          sum = 0.0f;
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            float xs[32];
            scores(c4, nm, xs);
            uint32_t pk[16];
            uint64_t ls = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float p0 = ex2(xs[2 * k]), p1 = ex2(xs[2 * k + 1]);
              ls = add2(ls, pack2(p0, p1));
              pk[k] = pack_bf16x2(p0, p1);
            }
            float la, lb;
            unpack2(ls, la, lb);
            sum += la + lb;
            tmem_st16(s_addr + c4 * 16, pk);
          }
        }
        l += sum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      if (!(ok = mbar_wait(&rec_v[rec], v_ph, ctl, 965))) break;
      const bool poison = r->bad < lim;  // the row sees a key whose V is not finite
      if (!(ok = mbar_wait(&o_full[x], oph, ctl, 966))) break;
      oph ^= 1;
      tc_fence_after();

      // A unit cut by the border of a run: each part leaves its unnormalised O, maxima and sums and counts itself in;
      // the last one (it waits for nobody) merges all parts in their order.  Windows of a run are joined in the same place
      // one by one; a unit that is not cut takes that of a unit's first part, which only the CTA's last unit needs, later.
      const int cta0 = r->cta0, cta1 = r->cta1, slab = x * 4 + quarter;
      const float* parts = nullptr;
      if (cta0 != cta1 || r->window) {
        constexpr int kSlab = many_slab<DH>();
        float* mine = p.part + (((int64_t)blockIdx.x * 2 + r->slot) * 8 + slab) * kSlab;
        if (r->window & 1) {
          const float2 ml = join_window<DH>(o_addr, mine, m_used, l);
          m_used = ml.x;
          l = ml.y;
        }
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
        int order = r->window & 2 ? -1 : 0;
        if (order == 0 && cta0 != cta1) {
          if (lane == 0) order = atomicAdd(&p.cnt[cta0 * 8 + slab], 1);
          order = __shfl_sync(0xffffffffu, order, 0);
        }
        if (order != cta1 - cta0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&o_empty[x]);
            mbar_arrive(&rec_empty[rec]);
          }
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
      // 16 columns at a time, each row's 32 bytes a whole sector
#pragma unroll 1
      for (int cc = 0; cc < DH / 16; ++cc) {
        uint32_t ov[16];
        if (!parts) {
          tmem_ld16(o_addr + cc * 16, ov);
          tmem_ld_wait();
        } else {
          constexpr int kSlab = many_slab<DH>();
#pragma unroll
          for (int k = 0; k < 16; ++k) ov[k] = 0;
          for (int c = cta0; c <= cta1; ++c) {
            const float* src = parts + ((int64_t)(c - cta0) * 16 + (c == cta0 ? 8 : 0)) * kSlab;
            const float f = m_used == -INFINITY ? 1.0f : ex2(__ldcg(src + DH * 32 + lane) - m_used);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src + ((cc * 4 + k) * 32 + lane) * 4));
              ov[4 * k] = __float_as_uint(fmaf(f, v.x, __uint_as_float(ov[4 * k])));
              ov[4 * k + 1] = __float_as_uint(fmaf(f, v.y, __uint_as_float(ov[4 * k + 1])));
              ov[4 * k + 2] = __float_as_uint(fmaf(f, v.z, __uint_as_float(ov[4 * k + 2])));
              ov[4 * k + 3] = __float_as_uint(fmaf(f, v.w, __uint_as_float(ov[4 * k + 3])));
            }
          }
        }
        const float scale = poison ? NAN : inv;
        if (at >= 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            st_global_v4(p.o + (size_t)at * DH + cc * 16 + k * 8,
                         pack_bf16x2(__uint_as_float(ov[8 * k]) * scale, __uint_as_float(ov[8 * k + 1]) * scale),
                         pack_bf16x2(__uint_as_float(ov[8 * k + 2]) * scale, __uint_as_float(ov[8 * k + 3]) * scale),
                         pack_bf16x2(__uint_as_float(ov[8 * k + 4]) * scale, __uint_as_float(ov[8 * k + 5]) * scale),
                         pack_bf16x2(__uint_as_float(ov[8 * k + 6]) * scale, __uint_as_float(ov[8 * k + 7]) * scale));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_empty[x]);
        mbar_arrive(&rec_empty[rec]);
      }
      if (at >= 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m_used + lg2(l)) * kLn2;
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
