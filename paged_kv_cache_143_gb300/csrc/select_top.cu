// select_top.cu — pa_select_blocks (the blocks that each query attends to) and
// pa_select_tokens (the tokens of a request that stay in the cache): of each
// row's candidates the first and last ones and the greatest others, listed in
// ascending order.
//
// Scores become 32-bit keys in the order of the numbers (NaN above all, forced
// candidates above NaN, -0 as 0). The k-th greatest key is found eight bits at a time
// from the top: of the keys that agree with what is found so far, a histogram in shared
// memory counts the next eight bits, and the digit is the one in which the k-th falls.
// Keys above the threshold are taken, and of those equal to it as many as are left,
// from the lowest index: one running count of both gives each candidate its place in
// the list. Counts are whole numbers, so nothing depends on the order of the atomics.
//  - A CTA of 128 threads (512 for more than 1024 candidates) holds eight candidates a
//    thread in registers; a row of more than 4096 is shared by a cluster of 2, 4 or 8
//    CTAs (histograms and counts joined through distributed shared memory), and one of
//    more than 32768 read again for every pass.
//  - What bounds it is latency (a few hundred kilobytes for a whole batch): a pass is
//    an atomic a candidate, and the digit, which one warp works out for all (every warp
//    for itself took more issue slots than the candidates). Replayed from a graph, 256
//    rows of up to 900, 2300 and 4063 candidates take 7.2, 8.3 and 9.9 us, 24 rows of
//    32000 14.1, one of 100000 50, rows that are taken whole 2.5 to 3. 256 threads of
//    sixteen candidates and 1024 of four: slower by 1 to 3 us.
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

template <int THREADS, int EACH>
struct SelectTail {
  alignas(16) int hist[4][kBins];         // of this CTA, pass by pass
  alignas(16) int total[kBins];           // of the cluster
  int2 counts[EACH * THREADS / 32];  // of a round, by place and warp: keys above the threshold
                                     // and equal to it; then the sums of those before
  int2 round;                        // a round's counts
  uint32_t digit;                    // a pass's digit, and which of its keys is wanted
  int rest;
  int row_state, row_n;              // what the row is: 0 nothing to do, 1 candidates
  const float* row_src;
  int cta_above, cta_equal;
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
// keys it is (from 1). The whole warp calls it; lane l has bins 255 - 8 l and below.
__device__ __forceinline__ void find_digit(const int* hist, int& left, uint32_t& digit) {
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
  int d = 0, rest = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (before < left && before + c[i] >= left) {
      d = kBins - 1 - 8 * lane - i;
      rest = left - before;
    }
    before += c[i];
  }
  digit = (uint32_t)__shfl_sync(kFull, d, who);
  left = __shfl_sync(kFull, rest, who);
}

template <int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS) select_kernel(SelectParams p) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = THREADS / 32, kRound = THREADS * EACH;
  __shared__ SelectTail<THREADS, EACH> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = p.split;
  const unsigned row = blockIdx.x / (unsigned)split;
  const int rank = (int)(blockIdx.x - row * split);
  for (int i = tid; i < 4 * kBins; i += THREADS) (&sm.hist[0][0])[i] = 0;
  if (warp == 0) {  // the row's candidates (every CTA of a cluster finds the same)
    int n = 0;
    const float* src = nullptr;
    bool ok = true;
    if (p.qsl) {
      const int t = (int)(row / (unsigned)p.H);
      const int r = request_of_row(p.qsl, p.R, t);
      ReqSpan s;
      ok = r >= 0 &&  // else a row behind the last sequence
           request_span(p.qsl, p.seq_lens, r, p.T, (int64_t)p.limit * p.unit, p.err, s);
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
  // this CTA's run of candidates; of each round a thread has every THREADS-th, in `held` places
  const int share = (n + split - 1) / split;
  const int begin = min(n, rank * share), end = min(n, begin + share);
  const int tail = n - p.last;
  const bool one_round = share <= kRound;
  const int held = min(EACH, (end - begin + THREADS - 1) / THREADS);
  uint32_t key[EACH];  // (0 where there is no candidate: the lowest key, of -inf, is greater)
  auto read = [&](int base) {
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int i = base + j * THREADS + tid;
      key[j] = i >= end ? 0u : i < p.first || i >= tail ? kForced : key_of(__ldg(src + i));
    }
  };
  read(begin);
  cg::cluster_group cluster = cg::this_cluster();
  uint32_t thr = 0;
  int left = p.k;  // of the k, those among the keys that agree with thr so far
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* hist = sm.hist[pass];
    for (int base = begin; base < end; base += kRound) {
      if (!one_round) read(base);
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        if (j % 4 == 0 && j >= held) break;
        const bool agrees = key[j] != 0u && (pass == 0 || ((key[j] ^ thr) >> (shift + 8)) == 0u);
        count_if(agrees, &hist[(key[j] >> shift) & (kBins - 1)]);
      }
    }
    if (split > 1) {
      cluster.sync();
      for (int i = tid; i < kBins; i += THREADS) {
        int c = 0;
        for (int o = 0; o < split; ++o) c += *cluster.map_shared_rank(&hist[i], o);
        sm.total[i] = c;
      }
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t digit;
      find_digit(split > 1 ? sm.total : hist, left, digit);
      if (lane == 0) {
        sm.digit = digit;
        sm.rest = left;
      }
    }
    __syncthreads();
    left = sm.rest;
    const uint32_t digit = sm.digit;
    thr |= digit << shift;
  }
  // left: how many of the keys equal to thr are taken. First, what the CTAs before have.
  int above0 = 0, equal0 = 0;
  if (split > 1) {
    int a = 0, e = 0;
    for (int base = begin; base < end; base += kRound) {
      if (!one_round) read(base);
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        a += key[j] > thr;
        e += key[j] == thr;
      }
    }
    a = __reduce_add_sync(kFull, a);
    e = __reduce_add_sync(kFull, e);
    if (tid == 0) sm.cta_above = sm.cta_equal = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&sm.cta_above, a);
      atomicAdd(&sm.cta_equal, e);
    }
    cluster.sync();
    for (int o = 0; o < rank; ++o) {
      above0 += *cluster.map_shared_rank(&sm.cta_above, o);
      equal0 += *cluster.map_shared_rank(&sm.cta_equal, o);
    }
    cluster.sync();  // no CTA leaves while another reads its counts
  }
  for (int base = begin; base < end; base += kRound) {
    if (!one_round) read(base);
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      if (j >= held) break;
      const unsigned up = __ballot_sync(kFull, key[j] > thr), tie = __ballot_sync(kFull, key[j] == thr);
      if (lane == 0) sm.counts[j * kWarps + warp] = make_int2(__popc(up), __popc(tie));
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sums over (place, warp)
      const int places = held * kWarps;
      int ca = 0, ce = 0;  // of the 32 before
      for (int i = lane; i < places + lane; i += 32) {
        const int2 c = i < places ? sm.counts[i] : make_int2(0, 0);
        int a = c.x, e = c.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, a, o), z = __shfl_up_sync(kFull, e, o);
          if (lane >= o) {
            a += y;
            e += z;
          }
        }
        if (i < places) sm.counts[i] = make_int2(ca + a - c.x, ce + e - c.y);
        ca += __shfl_sync(kFull, a, 31);
        ce += __shfl_sync(kFull, e, 31);
      }
      if (lane == 0) sm.round = make_int2(ca, ce);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      if (j >= held) break;
      const bool up = key[j] > thr, tie = key[j] == thr;
      const unsigned ups = __ballot_sync(kFull, up), ties = __ballot_sync(kFull, tie);
      if ((ups | ties) == 0u) continue;
      const int2 c = sm.counts[j * kWarps + warp];
      const unsigned lower = (1u << lane) - 1u;
      const int x = above0 + c.x + __popc(ups & lower), y = equal0 + c.y + __popc(ties & lower);
      if (up || (tie && y < left)) out[x + min(y, left)] = base + j * THREADS + tid;
    }
    if (!one_round) {
      above0 += sm.round.x;
      equal0 += sm.round.y;
      __syncthreads();
    }
  }
}

pa_status launch_select(SelectParams& p, int64_t rows, cudaStream_t s) {
  if (p.k > kMostTokens) return PA_ERR_UNSUPPORTED;
  if (p.limit > kMostTokens) p.limit = (int)kMostTokens;  // (a longer row is flagged)
  // 128 threads hold 1024 candidates: four such CTAs run where one of 512 does
  const bool small = p.limit <= 1024;
  const int threads = small ? 128 : 512, each = 8;
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
  if (cudaLaunchKernelEx(&cfg, small ? select_kernel<128, 8> : select_kernel<512, 8>, p) !=
      cudaSuccess) {
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
