// select_top.cu — pa_select_blocks (the blocks that each query attends to) and
// pa_select_tokens (the tokens of a request that stay in the cache): of each
// row's candidates the first and last ones and the greatest others, listed in
// ascending order.
//
// One CTA per row. Scores become 32-bit keys in the order of the numbers (NaN
// above all, forced candidates above NaN, -0 as 0), which each thread holds in
// registers for a run of consecutive candidates. The k-th greatest key is found
// bit by bit from the top: a bit stays set while at least k keys reach the
// prefix with it, 32 votes of the CTA in all and no atomics, so nothing depends
// on timing. Keys above the threshold are taken, and of those equal to it as
// many as are left, from the lowest index: one scan of both counts gives every
// thread the place of its candidates in the list.
// Rows longer than the registers hold (32768 candidates) read their scores again
// for every two bits.
#include "batch_rows.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kForced = 0xffffffffu;

struct SelectParams {
  const float* scores;       // row x at scores + x * stride
  int64_t stride;
  const int32_t* qsl;        // NULL: row r is request r, all its tokens are candidates
  const int32_t* seq_lens;
  const int32_t* idx;        // row of request r (qsl == NULL), NULL: r
  int max_rows;              // rows of scores (qsl == NULL)
  int R, T, H, unit;         // candidates are units of `unit` tokens
  int limit;                 // candidates that a row has room for
  int first, last, k;
  int32_t* out;              // [rows][k]
  int32_t* counts;           // [R] or NULL
  unsigned* err;
};

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return kForced - 1;  // NaN
  if (u == 0x80000000u) return 0x80000000u;                 // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sums over the CTA's threads of two counts; the scratch is [2][32].
template <int THREADS>
__device__ __forceinline__ void scan2(int& a, int& b, int (*scratch)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, x, o), v = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    scratch[0][warp] = x;
    scratch[1][warp] = y;
  }
  __syncthreads();
  int before_x = 0, before_y = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w)
    if (w < warp) {
      before_x += scratch[0][w];
      before_y += scratch[1][w];
    }
  a = before_x + x - a;
  b = before_y + y - b;
}

template <int THREADS, int M>
__global__ void __launch_bounds__(THREADS) select_kernel(SelectParams p) {
  __shared__ int scratch[2][32];
  __shared__ int votes[2][3];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float* src;
  int n;  // candidates
  if (p.qsl) {
    const int t = (int)(row / p.H);
    const int r = request_of_row(p.qsl, p.R, t);
    if (r < 0) return;  // a row behind the last sequence
    ReqSpan s;
    if (!request_span(p.qsl, p.seq_lens, r, p.T, (int64_t)p.limit * p.unit, p.err, s)) return;
    n = (s.seq - s.q_len + (t - s.q0)) / p.unit + 1;
    src = p.scores + row * p.stride;
  } else {
    const int r = (int)row;
    n = p.seq_lens[r];
    const int at = p.idx ? p.idx[r] : r;
    if (n < 0 || n > p.limit || at < 0 || at >= p.max_rows) {
      if (tid == 0) raise_error(p.err, kErrBounds);
      return;
    }
    src = p.scores + (int64_t)at * p.stride;
  }
  int32_t* out = p.out + row * p.k;
  if (p.counts && tid == 0) p.counts[row] = min(n, p.k);
  if (n <= p.k) {
    for (int i = tid; i < p.k; i += THREADS) out[i] = i < n ? i : -1;
    return;
  }
  const int tail = n - p.last;
  auto key_at = [&](int i) -> uint32_t {
    return i < p.first || i >= tail ? kForced : key_of(__ldg(src + i));
  };
  if (n <= THREADS * M) {
    uint32_t key[M];
    const int i0 = tid * M;
    const bool wide = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
#pragma unroll
    for (int m = 0; m < M; m += 4) {
      if (wide && i0 + m + 4 <= n) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(src + i0 + m));
        key[m] = key_of(v.x);
        key[m + 1] = key_of(v.y);
        key[m + 2] = key_of(v.z);
        key[m + 3] = key_of(v.w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) key[m + e] = i0 + m + e < n ? key_of(__ldg(src + i0 + m + e)) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + m + e;
        if (i < n && (i < p.first || i >= tail)) key[m + e] = kForced;
      }
    }
    // places past n hold 0, below every candidate's key (the lowest, of -inf, is 0x007fffff)
    uint32_t thr = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t want = thr | (1u << bit);
      int c = 0;
#pragma unroll
      for (int m = 0; m < M; ++m) c += key[m] >= want;
      c = __reduce_add_sync(kFull, c);
      // one slot of `scratch` per warp, two rows in turn: the next bit's counts
      // do not overtake the reading of this one's
      if ((tid & 31) == 0) scratch[bit & 1][tid >> 5] = c;
      __syncthreads();
      int sum = (tid & 31) < THREADS / 32 ? scratch[bit & 1][tid & 31] : 0;
      sum = __reduce_add_sync(kFull, sum);
      if (sum >= p.k) thr = want;
    }
    int above = 0, equal = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      above += key[m] > thr;
      equal += key[m] == thr && i0 + m < n;
    }
    const int mine = above;
    __syncthreads();
    int before = above, ties = equal;
    scan2<THREADS>(before, ties, scratch);
    // all keys above the threshold: the last thread's sums
    if (tid == THREADS - 1) votes[0][0] = before + mine;
    __syncthreads();
    const int room = p.k - votes[0][0];  // ties that are taken
    int at = before + min(ties, room);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const bool tie = key[m] == thr && i0 + m < n;
      if (key[m] > thr || (tie && ties < room)) out[at++] = i0 + m;
      ties += tie;
    }
    return;
  }
  // A row too long for the registers.
  uint32_t thr = 0;
  for (int bit = 30; bit >= 0; bit -= 2) {
    int c[3] = {0, 0, 0};
    for (int i = tid; i < n; i += THREADS) {
      const uint32_t key = key_at(i);
#pragma unroll
      for (int v = 0; v < 3; ++v) c[v] += key >= (thr | ((uint32_t)(v + 1) << bit));
    }
    const int turn = (bit >> 1) & 1;
    if (tid < 3) votes[turn][tid] = 0;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 3; ++v) {
      const int w = __reduce_add_sync(kFull, c[v]);
      if ((tid & 31) == 0) atomicAdd(&votes[turn][v], w);  // whole numbers: any order
    }
    __syncthreads();
    const uint32_t digit = (votes[turn][0] >= p.k) + (votes[turn][1] >= p.k) + (votes[turn][2] >= p.k);
    thr |= digit << bit;
  }
  int done = 0;   // listed so far
  int seen = 0;   // ties met so far
  int above = 0;  // keys above the threshold in all
  for (int i = tid; i < n; i += THREADS) above += key_at(i) > thr;
  above = __reduce_add_sync(kFull, above);
  __syncthreads();
  if ((tid & 31) == 0) scratch[0][tid >> 5] = above;
  __syncthreads();
  above = (tid & 31) < THREADS / 32 ? scratch[0][tid & 31] : 0;
  above = __reduce_add_sync(kFull, above);
  const int room = p.k - above;
  for (int base = 0; base < n; base += THREADS) {
    const int i = base + tid;
    const uint32_t key = i < n ? key_at(i) : 0u;
    const int up = i < n && key > thr, tie = i < n && key == thr;
    int a = up, e = tie;
    __syncthreads();
    scan2<THREADS>(a, e, scratch);
    const bool taken = up || (tie && seen + e < room);
    if (taken) out[done + a + min(e, max(room - seen, 0))] = i;
    if (tid == THREADS - 1) {
      votes[0][0] = a + up;
      votes[0][1] = e + tie;
    }
    __syncthreads();
    done += votes[0][0] + min(votes[0][1], max(room - seen, 0));
    seen += votes[0][1];
  }
}

pa_status launch_select(SelectParams& p, int64_t rows, cudaStream_t s) {
  if (rows > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  if (p.limit <= 1024)
    select_kernel<128, 8><<<(unsigned)rows, 128, 0, s>>>(p);
  else if (p.limit <= 4096)
    select_kernel<256, 16><<<(unsigned)rows, 256, 0, s>>>(p);
  else
    select_kernel<512, 64><<<(unsigned)rows, 512, 0, s>>>(p);
  return launch_status();
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_select_blocks(const float* scores, const int32_t* query_start_loc,
                                      const int32_t* seq_lens, int32_t num_reqs,
                                      int32_t num_tokens, int32_t num_kv_heads,
                                      int32_t max_blocks, int32_t block_size, int32_t first,
                                      int32_t last, int32_t k, int32_t* selected,
                                      pa_stream_t stream) {
  using namespace pa;
  if (num_reqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || max_blocks < 0 || block_size <= 0 ||
      first < 0 || last < 0 || k < 1 || (int64_t)first + last > k)
    return PA_ERR_INVALID;
  if (num_reqs == 0 || num_tokens == 0) return PA_OK;
  if (!scores || (reinterpret_cast<uintptr_t>(scores) & 3u) || !query_start_loc || !seq_lens ||
      !selected)
    return PA_ERR_INVALID;
  SelectParams p{};
  p.scores = scores;
  p.stride = max_blocks;
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.R = num_reqs;
  p.T = num_tokens;
  p.H = num_kv_heads;
  p.unit = block_size;
  p.limit = max_blocks;
  p.first = first;
  p.last = last;
  p.k = k;
  p.out = selected;
  return launch_select(p, (int64_t)num_tokens * num_kv_heads, as_stream(stream));
}

extern "C" pa_status pa_select_tokens(const float* mass, int64_t mass_stride, int32_t max_reqs,
                                      const int32_t* idx_mapping, const int32_t* seq_lens,
                                      int32_t num_reqs, int32_t first, int32_t last, int32_t k,
                                      int32_t* kept, int32_t* kept_lens, pa_stream_t stream) {
  using namespace pa;
  if (num_reqs < 0 || max_reqs < 0 || mass_stride < 0 || mass_stride > 0x7fffffff || first < 0 ||
      last < 0 || k < 1 || (int64_t)first + last > k)
    return PA_ERR_INVALID;
  if (num_reqs == 0) return PA_OK;
  if (!mass || (reinterpret_cast<uintptr_t>(mass) & 3u) || !seq_lens || !kept || !kept_lens)
    return PA_ERR_INVALID;
  SelectParams p{};
  p.scores = mass;
  p.stride = mass_stride;
  p.seq_lens = seq_lens;
  p.idx = idx_mapping;
  p.max_rows = max_reqs;
  p.R = num_reqs;
  p.H = 1;
  p.unit = 1;
  p.limit = (int)mass_stride;
  p.first = first;
  p.last = last;
  p.k = k;
  p.out = kept;
  p.counts = kept_lens;
  return launch_select(p, num_reqs, as_stream(stream));
}
