// cache_work.cuh -- how the attention over the cache is shared out among the CTAs.
//
// A unit is (request, key head, chunk of its query rows); the rows of a key head are the request's query tokens times
// the G query heads that share it.  A unit takes one step for each block of keys (one also for a history without keys:
// its outputs are written).  All steps of all units, in order (request, key head, chunk, keys), are numbered 0 ... W-1
// and each CTA takes an equal run of S of them, so the shares are equal however ragged requests and histories are.  A
// unit that is cut by the border between runs leaves partial results (unnormalised O, row maxima and sums); the part
// that counts itself in last merges all of them in order, so results do not depend on which CTA that is.  No CTA waits
// for another.  Each CTA finds its first unit by itself from the offsets and lengths on the device: no scheduling
// kernel runs first, and lengths may change between replays of a captured call.
#pragma once

#include "history.cuh"

namespace rocs {

struct Request {
  int c0, rows, L;  // first candidate, query rows of one key head, keys
};

// The request's sizes; what does not fit the call's bounds is reported and taken as empty.
__device__ __forceinline__ Request request_at(const CacheAttnParams& p, int r) {
  Request q;
  q.c0 = p.cand_off[r];
  const int64_t end = p.cand_off[r + 1];
  int n = (int)(end - q.c0);
  q.L = p.seq_len[r];
  if (q.c0 < 0 || end < q.c0 || end > p.C) {
    record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 931);
    q.c0 = n = 0;
  }
  q.rows = n * p.q_tokens * p.G;
  if (q.rows <= p.rows_lo || q.rows > p.rows_hi) q.rows = 0;
  if (q.rows > 0 && (q.L < 0 || q.L > p.capacity)) {
    record_error(p.ws, ROCS_ERR_DEVICE_INDEX, 932);
    q.L = q.L < 0 ? 0 : p.capacity;
  }
  return q;
}

template <int KEYS>
struct Work {
  int unit_rows;                      // rows of a chunk
  int r, head, chunk, chunks, steps;  // request, key head, chunk of rows, chunks and steps of the request's units
  Request q;
  int64_t pos, end, share;  // next step, end of this CTA's run, run length S
  int step;                 // next step within the unit

  __device__ __forceinline__ void enter(const CacheAttnParams& p, int request) {
    r = request;
    q = request_at(p, r);
    chunks = (q.rows + unit_rows - 1) / unit_rows;
    steps = q.L > 0 ? (q.L + KEYS - 1) / KEYS : 1;
  }
  __device__ __forceinline__ int64_t steps_of(const CacheAttnParams& p, int r) const {
    const Request q = request_at(p, r);
    return (int64_t)((q.rows + unit_rows - 1) / unit_rows) * p.c.heads * (q.L > 0 ? (q.L + KEYS - 1) / KEYS : 1);
  }
  // The first unit of this CTA's run.  All threads of the block (a multiple of 32, at most 1024) call it.
  // min_share: runs are not made shorter than this.
  __device__ __forceinline__ bool start(const CacheAttnParams& p, int rows, int64_t (&s_sum)[33], int64_t (&s_out)[3], int min_share) {
    unit_rows = rows;
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (p.R + T - 1) / T, b0 = min(p.R, t * per), b1 = min(p.R, b0 + per);
    int64_t sum = 0;
    for (int k = b0; k < b1; ++k) sum += steps_of(p, k);
    int64_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) s_sum[warp] = run;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) before += s_sum[w];
      total += s_sum[w];
    }
    run += before;  // steps up to and with this thread's requests
    share = (total + gridDim.x - 1) / gridDim.x;
    if (share < min_share) share = min_share;
    pos = (int64_t)blockIdx.x * share;
    end = min(pos + share, total);
    if (pos >= total) return false;
    if (run - sum <= pos && pos < run) {  // one thread's requests hold the first step
      int64_t at = run - sum;
      for (int k = b0; k < b1; ++k) {
        const int64_t n = steps_of(p, k);
        if (pos < at + n) {
          s_out[0] = k;
          s_out[1] = pos - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    enter(p, (int)s_out[0]);
    const int64_t within = s_out[1];
    const int unit = (int)(within / steps);
    step = (int)(within - (int64_t)unit * steps);
    head = unit / chunks;
    chunk = unit - head * chunks;
    return true;
  }
  // steps of the current unit that belong to this CTA: [step, step + n)
  __device__ __forceinline__ int count() const { return (int)min((int64_t)(steps - step), end - pos); }
  // on to the next unit; false at the end of the run
  __device__ __forceinline__ bool next(const CacheAttnParams& p) {
    pos += count();
    if (pos >= end) return false;
    step = 0;
    if (++chunk == chunks) {
      chunk = 0;
      if (++head == p.c.heads) {
        head = 0;
        int k = r;
        do enter(p, ++k);
        while (chunks == 0 && k + 1 < p.R);
      }
    }
    return true;
  }
  // CTAs whose runs hold steps of the current unit
  __device__ __forceinline__ int first_cta() const { return (int)((pos - step) / share); }
  __device__ __forceinline__ int last_cta() const { return (int)((pos - step + steps - 1) / share); }
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// mbar_wait that sleeps between polls.  A failed poll comes back after some 40 cycles and costs about ten instructions;
// with a dozen waiting warps these were more than half of all instructions issued.
template <int NS>
__device__ __forceinline__ bool mbar_wait_sleep(uint64_t* bar, uint32_t parity, const Ctl& ctl, int where) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    __nanosleep(NS);
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (ctl.aborted()) return false;
      if (globaltimer() - t0 > ctl.limit_ns) {
        ctl.fail(ROCS_ERR_TIMEOUT, where);
        return false;
      }
    }
  }
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLn2 = 0.69314718055994531f;

// Keys that a row sees: row `i` of a key head (of `rows`) belongs to query token i / G.  Rows past the last one are
// padding of a tile and see all keys, so that they do not make a block of keys look cut.
__device__ __forceinline__ int row_limit(const CacheAttnParams& p, const Request& q, int i) {
  if (i >= q.rows || !p.key_limit) return q.L;
  return min(q.L, max(0, p.key_limit[q.c0 + i / (p.q_tokens * p.G)]));
}

}  // namespace rocs
