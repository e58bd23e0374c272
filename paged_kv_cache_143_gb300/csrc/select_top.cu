// select_top.cu — pa_select_blocks (the blocks that each query attends to) and
// pa_select_tokens (the tokens of a request that stay in the cache): of each
// row's candidates the first and last ones and the greatest others, listed in
// ascending order.
//
// Scores become 32-bit keys in the order of the numbers (NaN above all, forced
// candidates above NaN, -0 as 0). The k-th greatest key is found eight bits at a time
// from the top: of the keys that agree with what is found so far, a histogram in shared
// memory counts the next eight bits, and the digit is the one in which the k-th falls
// (the search ends early where all keys of the digit are taken). Keys above the threshold
// are taken, and of those equal to it as many as are left, from the lowest index: one
// running count of both gives each candidate its place in the list. Counts are whole
// numbers, so nothing depends on the order of the atomics.
//  - A CTA of 128 threads (256 for more than 1024 candidates, 512 for more than 2048)
//    holds eight candidates a thread in registers, a warp a run of them in the row, so
//    that places follow from votes and one sum over the warps; a row of more than 4096
//    is shared by a cluster of 2, 4 or 8 CTAs (histograms joined through distributed
//    shared memory, with them what the CTAs before take), and one of more than 32768
//    read again for every pass.
//  - What bounds it is latency (a few hundred kilobytes for a whole batch): two trips to
//    memory until the keys are there, and a pass is an atomic a candidate and the digit,
//    which one warp works out for all (every warp for itself took more issue slots than
//    the candidates): 1450 cycles, 2900 in a cluster. Replayed from a graph, 256 rows of
//    up to 900, 2300 and 4063 candidates take 6.4, 7.5 and 8.4 us, 24 rows of 32000
//    12, one of 100000 38, rows that are taken whole 2 to 3; 16000 rows of 900 68.
//    1024 bins between the least and the greatest key, and the last few ranked one by
//    one: 9.2 and 17.
#include <cooperative_groups.h>

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
  int split;                 // CTAs (a cluster) a row
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

constexpr int kBins = 256;
constexpr int kThreadsAtOnce = 1536;  // of an SM

template <int THREADS>
struct SelectTail {
  alignas(16) int hist[4][kBins];  // of this CTA, pass by pass
  alignas(16) int total[kBins];    // of the cluster
  int digit, rest, in_bin;         // a pass's digit, which of its keys is wanted, and of how many
  int2 ahead[THREADS / 32];        // of a warp's bins: keys that the CTAs before take, and ties
  int2 counts[THREADS / 32];       // of a warp's keys of a round: those above the threshold, and equal to it
  int row_state, row_n;            // what the row is: 0 nothing to do, 1 candidates
  const float* row_src;
};

// One more in a bin, where `on`: predicated, so that a thread's candidates go out one
// after the other (a branch for each costs several times as much).
__device__ __forceinline__ void count_if(bool on, int* bin) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p red.shared::cta.add.u32 [%0], 1;\n\t}" ::"r"(smem_u32(bin)),
      "r"((uint32_t)on)
      : "memory");
}

// The digit into which the `left`-th key from the top falls, and which of that digit's
// keys it is (from 1), of how many. The whole warp calls it; lane l has bins 255 - 8 l and
// below.
__device__ __forceinline__ void find_digit(const int* hist, int& left, int& digit, int& in_bin) {
  const int lane = threadIdx.x & 31;
  const int4 hi = *reinterpret_cast<const int4*>(hist + kBins - 4 - 8 * lane);
  const int4 lo = *reinterpret_cast<const int4*>(hist + kBins - 8 - 8 * lane);
  const int c[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += c[i];
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += y;
  }
  const unsigned reached = __ballot_sync(kFull, before >= left);
  const int who = __ffs(reached) - 1;  // (left is at most the number of keys)
  before -= sum;
  int d = 0, rest = 0, size = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (before < left && before + c[i] >= left) {
      d = kBins - 1 - 8 * lane - i;
      rest = left - before;
      size = c[i];
    }
    before += c[i];
  }
  digit = __shfl_sync(kFull, d, who);
  in_bin = __shfl_sync(kFull, size, who);
  left = __shfl_sync(kFull, rest, who);
}

template <int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS, kThreadsAtOnce / THREADS) select_kernel(SelectParams p) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = THREADS / 32, kRound = THREADS * EACH;
  __shared__ SelectTail<THREADS> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = p.split;
  const unsigned row = blockIdx.x / (unsigned)split;
  const int rank = (int)(blockIdx.x - row * split);
  for (int i = tid; i < 4 * kBins / 4; i += THREADS)
    reinterpret_cast<int4*>(sm.hist)[i] = make_int4(0, 0, 0, 0);
  if (warp == 0) {  // the row's candidates (every CTA of a cluster finds the same)
    int n = 0;
    const float* src = nullptr;
    bool ok = true;
    if (p.qsl) {
      const int t = (int)(row / (unsigned)p.H);
      ReqSpan s;
      const int r = span_of_row(p.qsl, p.seq_lens, p.R, t, s);
      ok = r >= 0 &&  // else a row behind the last sequence
           span_fits(s, p.T, (int64_t)p.limit * p.unit, p.err);
      if (ok) n = (s.seq - s.q_len + (t - s.q0)) / p.unit + 1;
      src = p.scores + (int64_t)row * p.stride;
    } else {
      n = p.seq_lens[row];
      const int at = p.idx ? p.idx[row] : (int)row;
      ok = n >= 0 && n <= p.limit && at >= 0 && at < p.max_rows;
      if (!ok && lane == 0) raise_error(p.err, kErrBounds);
      src = p.scores + (int64_t)at * p.stride;
    }
    if (lane == 0) {
      sm.row_state = ok;
      sm.row_n = n;
      sm.row_src = src;
    }
  }
  __syncthreads();
  if (!sm.row_state) return;
  const int n = sm.row_n;
  const float* src = sm.row_src;
  int32_t* out = p.out + (int64_t)row * p.k;
  if (p.counts && tid == 0 && rank == 0) p.counts[row] = min(n, p.k);
  if (n <= p.k) {
    for (int i = rank * THREADS + tid; i < p.k; i += THREADS * split) out[i] = i < n ? i : -1;
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  // This CTA's run of candidates. Of a round a warp has `held` times 32 in a row, a thread
  // every 32nd of them.
  const int share = (n + split - 1) / split;
  const int begin = min(n, rank * share), end = min(n, begin + share);
  const int tail = n - p.last;
  const bool one_round = share <= kRound;
  const int held = min(EACH, (end - begin + THREADS - 1) / THREADS);
  uint32_t key[EACH];  // (0 where there is no candidate: the lowest key, of -inf, is greater)
  auto index = [&](int base, int j) { return base + (warp * held + j) * 32 + lane; };
  auto read = [&](int base) {
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int i = index(base, j);
      key[j] = j >= held || i >= end ? 0u : i < p.first || i >= tail ? kForced : key_of(__ldg(src + i));
    }
  };
  // Each round's keys in turn: those of the one round stay where they are.
  auto rounds = [&](auto f) {
    for (int base = begin; base < end; base += kRound) {
      if (!one_round) read(base);
      f(base);
    }
  };
  read(begin);
  uint32_t thr = 0;
  int left = p.k;  // of the k, those among the keys that agree with thr so far
  // (of a cluster, the first 256 threads:) keys of the thread's bins that the CTAs before
  // this one take, and of ties that they have
  int ahead = 0, ahead_ties = 0;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* hist = sm.hist[pass];
    rounds([&](int) {
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        if (j % 4 == 0 && j >= held) break;
        const bool agrees = key[j] != 0u && (pass == 0 || ((key[j] ^ thr) >> (shift + 8)) == 0u);
        count_if(agrees, &hist[(key[j] >> shift) & (kBins - 1)]);
      }
    });
    int before = 0;
    if (split > 1) {
      cluster.sync();
      if (tid < kBins) {
        int c = 0;
#pragma unroll
        for (int o = 0; o < 8; ++o) {
          const int x = o < split ? *cluster.map_shared_rank(&hist[tid], o) : 0;
          c += x;
          before += o < rank ? x : 0;
        }
        sm.total[tid] = c;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int digit, in_bin;
      find_digit(split > 1 ? sm.total : hist, left, digit, in_bin);
      if (lane == 0) {
        sm.digit = digit;
        sm.rest = left;
        sm.in_bin = in_bin;
      }
    }
    __syncthreads();
    left = sm.rest;
    const int digit = sm.digit;
    const bool all = left == sm.in_bin;  // of this digit: no need to tell them apart
    thr |= (uint32_t)digit << shift;
    ahead += tid > digit || (all && tid == digit) ? before : 0;
    if (all) {
      thr = max(thr, 1u) - 1u;  // (all keys are above 0)
      left = 0;
      break;
    }
    if (pass == 3 && tid == digit) ahead_ties = before;
  }
  // Keys above thr are taken, and `left` of those equal to it.
  int above0 = 0, equal0 = 0;
  if (split > 1) {
    cluster.barrier_arrive();
    ahead = __reduce_add_sync(kFull, ahead);
    ahead_ties = __reduce_add_sync(kFull, ahead_ties);
    if (lane == 0) sm.ahead[warp] = make_int2(ahead, ahead_ties);
    __syncthreads();
    const int2 c = lane < kWarps ? sm.ahead[lane] : make_int2(0, 0);
    above0 = __reduce_add_sync(kFull, c.x);
    equal0 = __reduce_add_sync(kFull, c.y);
  }
  rounds([&](int base) {
    unsigned ups[EACH], ties[EACH];
    int a = 0, e = 0;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      ups[j] = __ballot_sync(kFull, key[j] > thr);
      ties[j] = __ballot_sync(kFull, key[j] == thr);
      a += __popc(ups[j]);
      e += __popc(ties[j]);
    }
    if (lane == 0) sm.counts[warp] = make_int2(a, e);
    __syncthreads();
    const int2 c = lane < kWarps ? sm.counts[lane] : make_int2(0, 0);
    int x = above0 + __reduce_add_sync(kFull, lane < warp ? c.x : 0);
    int y = equal0 + __reduce_add_sync(kFull, lane < warp ? c.y : 0);
    const unsigned lower = (1u << lane) - 1u;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int up = x + __popc(ups[j] & lower), tie = y + __popc(ties[j] & lower);
      if (key[j] > thr || (key[j] == thr && tie < left)) out[up + min(tie, left)] = index(base, j);
      x += __popc(ups[j]);
      y += __popc(ties[j]);
    }
    if (!one_round) {
      above0 += __reduce_add_sync(kFull, c.x);
      equal0 += __reduce_add_sync(kFull, c.y);
      __syncthreads();
    }
  });
  if (split > 1) cluster.barrier_wait();  // no CTA leaves while another reads its bins
}

pa_status launch_select(SelectParams& p, int64_t rows, cudaStream_t s) {
  if (p.k > kMostTokens) return PA_ERR_UNSUPPORTED;
  if (p.limit > kMostTokens) p.limit = (int)kMostTokens;  // (a longer row is flagged)
  // (16000 rows of 1000 candidates: 68 us by 128 threads, 109 by 256, 247 by 512)
  const int threads = p.limit <= 1024 ? 128 : p.limit <= 2048 ? 256 : 512, each = 8;
  p.split = 1;
  while (p.split < 8 && (int64_t)p.split * threads * each < p.limit) p.split *= 2;
  if (rows * p.split > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * p.split));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  auto kernel = threads == 128   ? select_kernel<128, 8>
                : threads == 256 ? select_kernel<256, 8>
                                 : select_kernel<512, 8>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
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
