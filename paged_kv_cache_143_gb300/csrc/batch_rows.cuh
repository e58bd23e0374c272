// batch_rows.cuh — which request a row of a ragged batch belongs to, found on
// the device from query_start_loc alone (no host mirror, so a captured call
// follows device lengths that change between replays).
#pragma once

#include "pa_device.cuh"

namespace pa {

// The longest list of tokens, candidates or places: below 2^31 by more than any loop here
// goes past its end.
constexpr int64_t kMostTokens = 0x7fff0000;

// The last i of [0, n) with f(i) <= x, for f that does not fall (0 if there is
// none). The lanes of a warp try 32 places at once: one round for up to 32
// requests, two for 1024, each a load and a vote. All lanes get the answer.
template <class F>
__device__ __forceinline__ int warp_last_le(int n, int64_t x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int64_t at = (int64_t)lane * step;
    const bool le = at < len && (int64_t)f(lo + (int)at) <= x;
    const int c = max(__popc(__ballot_sync(0xffffffffu, le)), 1);
    const int skip = (c - 1) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  return lo;
}

// Request r's rows and lengths, or false (with kErrBounds) where they leave the
// batch's buffers.
struct ReqSpan {
  int q0, q_len, seq;
};
__device__ __forceinline__ bool span_fits(const ReqSpan& s, int T, int64_t capacity, unsigned* err) {
  if (s.q0 >= 0 && s.q_len >= 0 && (int64_t)s.q0 + s.q_len <= T &&
      (s.q_len == 0 || (s.seq >= s.q_len && s.seq <= capacity)))
    return true;
  raise_error(err, kErrBounds);
  return false;
}
__device__ __forceinline__ bool request_span(const int32_t* qsl, const int32_t* seq_lens, int r,
                                             int T, int64_t capacity, unsigned* err, ReqSpan& s) {
  s.q0 = qsl[r];
  s.q_len = qsl[r + 1] - s.q0;
  s.seq = seq_lens[r];
  return span_fits(s, T, capacity, err);
}

// A worker's run [begin, end) of a batch's units of work, of which request r has
// units(r): the requests' units one after the other, equal runs for all workers. Unit
// `begin` is request r's, whose first unit is `base`. Found from the device lengths by
// each worker for itself (the whole warp calls it): every lane sums a part of the
// requests, and the part that holds `begin` is gone through in the same way.
struct BatchRun {
  int64_t begin, end, base;
  int r;
};
template <class F>
__device__ __forceinline__ BatchRun batch_run(int R, int64_t workers, int64_t worker, F units) {
  const int lane = threadIdx.x & 31;
  BatchRun run{0, 0, 0, 0};
  int lo = 0, len = R;
  for (bool top = true; top || len > 1; top = false) {
    const int step = (len + 31) >> 5;
    const int from = (int)min((int64_t)lane * step, (int64_t)len), to = min(from + step, len);
    int64_t mine = 0;
#pragma unroll 4
    for (int i = from; i < to; ++i) mine += units(lo + i);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (top) {
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31), per = (all + workers - 1) / workers;
      run.begin = min(worker * per, all);
      run.end = min(run.begin + per, all);
      if (run.begin == run.end) return run;
    }
    const unsigned past = __ballot_sync(0xffffffffu, run.base + upto > run.begin);
    const int who = __ffs(past) - 1;  // (there is one: begin < the units up to the last lane's)
    run.base += __shfl_sync(0xffffffffu, upto - mine, who);
    lo += who * step;
    len = min(step, len - who * step);
  }
  run.r = lo;
  return run;
}

// The request of row t and its rows and lengths, or -1 for a row behind the last sequence.
// The whole warp calls it. One trip to memory for up to 32 requests, and for row t of
// request t (a batch of decodes); else the search after it.
__device__ __forceinline__ int span_of_row(const int32_t* qsl, const int32_t* seq_lens, int R, int t,
                                           ReqSpan& s) {
  const int lane = threadIdx.x & 31;
  const int at = R <= 32 ? min(lane, R - 1) : min(t, R - 1);
  int q0 = __ldg(qsl + at), q1 = __ldg(qsl + at + 1), seq = __ldg(seq_lens + at), r = at;
  if (R <= 32) {
    r = max(__popc(__ballot_sync(0xffffffffu, lane < R && q0 <= t)) - 1, 0);
    q0 = __shfl_sync(0xffffffffu, q0, r);
    q1 = __shfl_sync(0xffffffffu, q1, r);
    seq = __shfl_sync(0xffffffffu, seq, r);
  } else if (t < q0 || t >= q1) {
    r = warp_last_le(R, t, [&](int i) { return __ldg(qsl + i); });
    q0 = __ldg(qsl + r);
    q1 = __ldg(qsl + r + 1);
    seq = __ldg(seq_lens + r);
  }
  s.q0 = q0;
  s.q_len = q1 - q0;
  s.seq = seq;
  return t >= q0 && t < q1 ? r : -1;
}

}  // namespace pa
