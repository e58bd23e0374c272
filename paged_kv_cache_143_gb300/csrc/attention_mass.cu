// attention_mass.cu — pa_attention_mass: for each stored token the sum, over the
// last queries of its request and all heads, of the softmax weights that it
// received, added to what it had received before.
//
// The weights need each row's maximum and sum over all keys first, so the work
// has two passes over the scores. A request's rows for one kv head are its
// counted queries times the g heads that share the kv head; two forms:
//
//  - up to 16 rows (decodes, drafted tokens; up to 64, 16 at a time, in small calls
//    without longer requests): the keys are what costs. One pass
//    streams them once (warps with rings of 16-key cells, S^T = K Q^T by
//    warp-level MMAs with the keys as rows, as pa_sparse_forward), writes the
//    scores (4 g bytes a key against 2 D or D bytes of the key) to the
//    workspace and each split's row maxima and sums; the second joins those and
//    adds 2^(score - lse) over the rows, key by key, from L2.
//    40 decodes of 1k to 8k (8 kv heads, 4 rows, bf16): 72 us, 62 of them the first,
//    5.8 TB/s (0.86 of the copy rate).
//  - more rows (the last queries of a prompt): scores are made twice on tcgen05,
//    128 x 128 at a time, never leaving the SM. Pass 1 has query rows as the
//    accumulator's lanes, so that a thread owns a row and its running maximum
//    and sum; pass 2 has keys as lanes, S^T = K Q^T, so that the weights of a key
//    are added in the registers of four threads, over the rows of a tile, and over
//    tiles by a last kernel: no atomics,
//    and the order of every sum follows from the sizes alone.
//    The query rows are laid out once per call as shared-memory images of 128
//    rows, swizzled as the tensor cores read them, which one bulk copy fetches;
//    behind each image its rows' score factors.
//
// E4M3 pools: the codes are multiplied as they are. In the streaming form they widen to
// f16; on tcgen05 a query is the sum of two E4M3 numbers (8 significant bits, all
// that bf16 has) after a power-of-two scale that puts its row's largest magnitude
// into [2^7, 2^8): exact for elements down to 2^-8 of that one, off by 2^-17 of it
// at the most below. (Half a step of 2^-9, the smallest of E4M3, of 2^7.)
#include <cuda_fp8.h>

#include <algorithm>
#include <utility>

#include "batch_rows.cuh"
#include "cells.cuh"
#include "mbar_poll.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNarrowRows = 16;     // rows that a CTA of the streaming form takes
constexpr int kStreamRows = 64;     // rows of a request of that form, at the most
constexpr int kStreamUnits = 304;   // its CTAs, where they are to spare the tcgen05 form: one round
// Rows of all kv heads whose sums are at hand in shared memory: 48 KB but for the 1 KB that
// mass_sum_kernel has beside them.
constexpr int kSumRows = (49152 - 1024) / 4;
constexpr int kSplitKeys = 1024;    // keys of one of its CTAs
constexpr int kTile = 128;          // rows, and keys, of a tcgen05 tile
constexpr int kInfoBytes = 1024;    // behind an image: the score factors of its rows
// Of rows 2 i and 2 i + 1 four floats, (factor, factor, -lse, -lse), so that one load
// feeds one packed multiply-add: the row's factor is at info_at(row), -lse 2 further.
__device__ __forceinline__ int info_at(int row) { return (row >> 1) * 4 + (row & 1); }

constexpr int kFewReqs = 64;        // whose mirrors come with the launch

struct MassParams {
  const __nv_bfloat16* q;
  const float* mass_in;
  float* mass_out;
  int64_t mass_stride;
  const int32_t* idx;
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int2* mirrors;     // [R] the mirrors' new and stored tokens, of more than kFewReqs
  const int32_t* tables;
  int max_reqs, max_blocks, R, T, Hq, Hkv, g, B, num_blocks, window;
  float decay, qk_scale;   // softmax scale * log2(e) (* k_scale)
  // streaming form
  float* scores;           // request after request: [Hkv * rows][keys rounded up to 16]
  float2* split_stats;     // [R][Hkv][groups][16][splits] (maximum, sum)
  int splits;
  int groups;              // of 16 rows
  int sum_keys;            // keys of a CTA of the sums
  // tcgen05 form: a step is a row tile of a kv head and a key tile; request r's are the
  // flat steps first_step[r] + (kvh * tiles + row tile) * key tiles + key tile
  int4* tiled;             // [R]: first tile (-1: none), first row of q, new tokens, stored tokens
  int64_t* first_step;     // [R + 1]
  uint8_t* images;         // [n_tiles][Hkv][image]
  float2* tile_stats;      // [n_tiles][Hkv][pieces][4][128]
  float* sums;             // [steps][128]: a step's weights, key by key
  int64_t steps, per_cta;  // in all, and of a CTA
  int pieces;
  unsigned* err;
  int stream_rows;         // rows, by its mirror, up to which a request is streamed (-1: none is)
  int2 few[kFewReqs];      // the mirrors of up to as many requests
};

struct MassReq {
  int q0, q_len, seq, w, rows;  // w counted queries, rows = w * g
  bool wide;                    // of the tcgen05 form
};

// Request r as the device has it; without rows where an entry leaves the buffers, or its
// mirror, whose room is planned: what the requests before r take is then never more than
// planned either, so that every request finds its own. The form that it takes is the
// mirror's choice, so that a captured call whose lengths shrink finds it planned. (Mirrors
// that come with every launch need no launch of their own: a decode on 3000 tokens 16.4 us
// instead of 17.4.)
__device__ __forceinline__ MassReq rows_of(const MassParams& p, int r) {
  const int q0 = p.qsl[r], end = p.qsl[r + 1], seq = p.seq_lens[r];
  const int2 most = p.R <= kFewReqs ? p.few[r] : __ldcg(p.mirrors + r);
  MassReq m;
  m.q0 = q0;
  m.q_len = end - q0;
  m.seq = seq;
  m.wide = (int64_t)(p.window > 0 ? min(most.x, p.window) : most.x) * p.g > p.stream_rows;
  // (the mirrors' tokens fit the table, the mass and 32 bits)
  const bool fine = q0 >= 0 && end <= p.T && end >= q0 && seq >= m.q_len && m.q_len <= most.x && seq <= most.y;
  m.w = fine ? (p.window > 0 ? min(m.q_len, p.window) : m.q_len) : 0;
  m.rows = m.w * p.g;
  return m;
}
// The same of a request as mass_rows_kernel has held it against its mirror and put it down.
__device__ __forceinline__ MassReq tiled_rows_of(const MassParams& p, const int4& t) {
  MassReq m;
  m.q0 = t.y;
  m.q_len = t.z;
  m.seq = t.w;
  m.w = p.window > 0 ? min(m.q_len, p.window) : m.q_len;
  m.rows = m.w * p.g;
  m.wide = true;
  return m;
}
// Whether request r was left out for entries that leave the buffers.
__device__ __forceinline__ bool bad_request(const MassReq& m) { return m.rows == 0 && m.q_len != 0; }

__device__ __forceinline__ int padded_keys(int seq) { return (seq + 15) & ~15; }

// The sum of f over the requests before r; the whole warp calls it.
template <class F>
__device__ __forceinline__ int64_t before(const MassParams& p, int r, F f) {
  int64_t sum = 0;
  for (int i = threadIdx.x & 31; i < r; i += 32) sum += f(rows_of(p, i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum;
}

__device__ __forceinline__ int64_t score_floats_of(const MassParams& p, const MassReq& m) {
  return m.wide ? 0 : (int64_t)p.Hkv * m.rows * padded_keys(m.seq);
}

__device__ __forceinline__ int mass_row(const MassParams& p, int r) {
  const int at = p.idx ? p.idx[r] : r;
  return at >= 0 && at < p.max_reqs ? at : -1;
}

// (ref, sum) joined with another part's maximum and sum.
__device__ __forceinline__ void join_stats(float& ref, float& sum, float m, float l) {
  const float top = fmaxf(ref, m), base = top == -INFINITY ? 0.f : top;
  sum = sum * ex2_ftz(ref - base) + l * ex2_ftz(m - base);
  ref = top;
}

// The mirrors as the kernels after it read them: passed by value, so that a captured call
// keeps its own. 4 KB of parameters a launch.
constexpr int kMirrorsAtOnce = 480;
struct Mirrors {
  int2 v[kMirrorsAtOnce];
};
__global__ void mass_mirrors_kernel(int2* out, int n, const __grid_constant__ Mirrors m) {
  launch_dependents();
  if ((int)threadIdx.x < n) out[threadIdx.x] = m.v[threadIdx.x];
}

// ------------------------------------------------------------ streaming form

constexpr int kNarrowWarps = 4;
constexpr int kNarrowRing = 24576;  // of a warp: two CTAs on an SM

struct NarrowTail {
  uint64_t full[kNarrowWarps][8];
  float2 stats[kNarrowWarps][kNarrowRows];
};

template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kNarrowWarps * 32, 2)
    mass_scores_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ MassParams p) {
  using C = Cells<D, FP8>;
  constexpr int kStages = kNarrowRing / C::kBytes > 8 ? 8 : kNarrowRing / C::kBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  NarrowTail* tail = reinterpret_cast<NarrowTail*>(ring + kNarrowWarps * kNarrowRing);
  grid_dependency_wait();  // the mirrors are there (also for the kernel after this one)
  launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tig = lane & 3;
  const int split = blockIdx.x, kvh = blockIdx.y / p.groups, r = blockIdx.z;
  const int row0 = (blockIdx.y - kvh * p.groups) * kNarrowRows;  // the first of the CTA's 16 rows
  const MassReq m = rows_of(p, r);
  const bool reporter = tid == 0 && split == 0 && blockIdx.y == 0;
  if (m.wide) return;
  if (bad_request(m) || (m.rows > 0 && mass_row(p, r) < 0)) {
    if (reporter) raise_error(p.err, kErrBounds);
    return;
  }
  const int k0 = split * kSplitKeys;
  if (m.rows <= row0 || k0 >= m.seq) return;
  const int64_t at = before(p, r, [&](const MassReq& x) { return score_floats_of(p, x); });
  const int n_cells = (min(m.seq - k0, kSplitKeys) + kChunk - 1) / kChunk;
  const int stride = padded_keys(m.seq);
  const int n_rows = min(kNarrowRows, m.rows - row0);
  float* out = p.scores + at + ((int64_t)kvh * m.rows + row0) * stride;
  const int32_t* table = p.tables + (int64_t)r * p.max_blocks;
  uint8_t* my_ring = ring + warp * kNarrowRing;
  uint64_t* full = tail->full[warp];
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // the warp's cells are warp, warp + 4, ...; lane i fetches the block of the i-th (16 at most)
  static_assert(kSplitKeys / kChunk / kNarrowWarps <= 32, "a lane for each of a warp's cells");
  const int mine = (n_cells - warp + kNarrowWarps - 1) / kNarrowWarps;
  int id_lane = 0;
  if (lane < mine) {
    id_lane = __ldg(table + (k0 + (lane * kNarrowWarps + warp) * kChunk) / p.B);
    if (id_lane < 0 || id_lane >= p.num_blocks) {
      raise_error(p.err, kErrBounds);
      id_lane = p.num_blocks;  // past the tensor map: keys of zeros
    }
  }
  auto issue = [&](int i) {  // the warp's i-th cell
    const int id = __shfl_sync(kFull, id_lane, i & 31);
    if (lane == 0) {
      const int row = (k0 + (i * kNarrowWarps + warp) * kChunk) % p.B;
      mbar_arrive_expect_tx(&full[i % kStages], C::kBytes);
      C::load(my_ring + (i % kStages) * C::kBytes, &tmap_k, kvh * p.B + row, id,
              &full[i % kStages]);
    }
  };
  for (int i = 0; i < min(mine, kStages); ++i) issue(i);
  QueryCols<D, FP8, NH> q;
  q.load([&](int c) -> const __nv_bfloat16* {
    if (c >= n_rows) return nullptr;
    c += row0;
    return p.q + ((int64_t)(m.q0 + m.q_len - m.w + c / p.g) * p.Hq + kvh * p.g + c % p.g) * D;
  }, p.qk_scale, grp, tig);
  float mx[NH][2], l[NH][2];
  int lim[NH][2];  // keys that the query of column 2 tig + e sees
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[h][e] = -INFINITY;
      l[h][e] = 0.f;
      lim[h][e] = m.seq - m.w + (row0 + 8 * h + 2 * tig + e) / p.g + 1;
    }
  for (int i = 0; i < mine; ++i) {
    const int stage = i % kStages;
    if (!__all_sync(kFull, mbar_wait(&full[stage], (i / kStages) & 1, p.err))) {
      if (lane == 0)
        for (int x = i + 1; x < min(mine, i + kStages); ++x)
          mbar_wait(&full[x % kStages], (x / kStages) & 1, p.err);
      break;  // flagged
    }
    float s[NH][4];
    q.scores(my_ring + stage * C::kBytes, s, grp, tig);
    __syncwarp();
    if (i + kStages < mine) issue(i + kStages);
    const int key = k0 + (i * kNarrowWarps + warp) * kChunk + grp;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 8 * h + 2 * tig + e;
        float x0 = s[h][e] * q.sc[h][e];
        float x1 = s[h][2 + e] * q.sc[h][e];
        if (key >= lim[h][e]) x0 = -INFINITY;
        if (key + 8 >= lim[h][e]) x1 = -INFINITY;
        if (c < n_rows) {
          float* dst = out + (int64_t)c * stride + key;
          dst[0] = x0;
          dst[8] = x1;
        }
        // this lane's keys only: joined below
        const float ref = fmaxf(mx[h][e], fmaxf(x0, x1));
        const float base = ref == -INFINITY ? 0.f : ref;
        l[h][e] = l[h][e] * ex2_ftz(mx[h][e] - base) + (ex2_ftz(x0 - base) + ex2_ftz(x1 - base));
        mx[h][e] = ref;
      }
  }
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float m2 = __shfl_xor_sync(kFull, mx[h][e], o), l2 = __shfl_xor_sync(kFull, l[h][e], o);
        join_stats(mx[h][e], l[h][e], m2, l2);
      }
      if (grp == 0) tail->stats[warp][8 * h + 2 * tig + e] = make_float2(mx[h][e], l[h][e]);
    }
  __syncthreads();
  if (tid < n_rows) {
    float ref = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kNarrowWarps; ++w) ref = fmaxf(ref, tail->stats[w][tid].x);
    const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int w = 0; w < kNarrowWarps; ++w)
      sum += tail->stats[w][tid].y * ex2_ftz(tail->stats[w][tid].x - base);
    p.split_stats[(((int64_t)r * gridDim.y + blockIdx.y) * kNarrowRows + tid) * p.splits + split] =
        make_float2(ref, sum);
  }
}

// Log of the sum of 2^score of a row, from `n` parts (maximum, sum) `step` apart.
__device__ __forceinline__ float lse_of(const float2* s, int n, int64_t step) {
  float ref = -INFINITY, sum = 0.f;
  for (int i = 0; i < n; ++i) ref = fmaxf(ref, s[i * step].x);
  const float base = ref == -INFINITY ? 0.f : ref;
  for (int i = 0; i < n; ++i) sum += s[i * step].y * ex2_ftz(s[i * step].x - base);
  return ref + log2f(sum);  // (-inf for a row that scores -inf throughout: its weights are then NaN)
}

// A long sum of parts: what the roundings of the sum lost is put back at the end.
struct Total {
  float sum = 0.f, low = 0.f;
  __device__ __forceinline__ void add(float part) {
    const float x = part + low, next = sum + x;
    low = x - (next - sum);
    sum = next;
  }
  // (of a sum that is not finite nothing is put back)
  __device__ __forceinline__ float get() const { return isfinite(low) ? sum + low : sum; }
};

// *src, or 0: predicated, so that loads go out one after the other.
__device__ __forceinline__ float load_if(bool on, const float* src) {
  float x;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
      "@p ld.global.f32 %0, [%1];\n\t}"
      : "=f"(x)
      : "l"(src), "r"((uint32_t)on)
      : "memory");
  return x;
}

constexpr int kSumThreads = 256;

// A CTA takes p.sum_keys keys, all of whose rows a thread adds up, or a part of them.
__global__ void __launch_bounds__(kSumThreads, 5) mass_sum_kernel(const __grid_constant__ MassParams p) {
  extern __shared__ float lse[];  // [Hkv * rows]
  const int r = blockIdx.y;
  const MassReq m = rows_of(p, r);
  if (m.wide || m.rows == 0) return;
  const int key0 = blockIdx.x * p.sum_keys;
  if (key0 >= m.seq) return;
  const int slot = mass_row(p, r);
  if (slot < 0) return;  // (flagged)
  const int64_t at = before(p, r, [&](const MassReq& x) { return score_floats_of(p, x); });
  grid_dependency_wait();  // the scores and their statistics are complete
  const int rows = p.Hkv * m.rows, n_split = (m.seq + kSplitKeys - 1) / kSplitKeys;
  // eight lanes for each row, all rows of up to 32 at once
  for (int base = 0; base < rows; base += kSumThreads / 8) {
    const int x = base + ((int)threadIdx.x >> 3), lane = threadIdx.x & 7;
    float ref = -INFINITY, sum = 0.f;
    if (x < rows) {
      const int kvh = x / m.rows, row = x - kvh * m.rows;
      const float2* part = p.split_stats +
          (((int64_t)r * p.Hkv + kvh) * p.groups * kNarrowRows + row) * p.splits;
      for (int i = lane; i < n_split; i += 8) join_stats(ref, sum, part[i].x, part[i].y);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      join_stats(ref, sum, __shfl_xor_sync(kFull, ref, o), __shfl_xor_sync(kFull, sum, o));
    if (lane == 0 && x < rows) lse[x] = ref + log2f(sum);  // (as lse_of)
  }
  __syncthreads();
  const int part = (int)threadIdx.x / p.sum_keys, key = key0 + (int)threadIdx.x % p.sum_keys;
  const int per = (rows * p.sum_keys + kSumThreads - 1) / kSumThreads;  // rows of a thread
  const int x1 = key < m.seq ? min(rows, (part + 1) * per) : 0;
  const int stride = padded_keys(m.seq);
  const float* s = p.scores + at + (int64_t)part * per * stride + key;
  const int c0 = max(0, key - (m.seq - m.w)) * p.g;  // the first row that sees the key
  Total total;
  int x0 = part * per;
  if (c0 == 0)
    for (; x0 + 32 <= x1; x0 += 32, s += (int64_t)32 * stride) {
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 32; ++x) sum += ex2_ftz(s[x * (int64_t)stride] - lse[x0 + x]);
      total.add(sum);
    }
  for (; x0 < x1; x0 += 16) {  // (without a branch, which would make a load wait for the one before)
    float v[16];
#pragma unroll
    for (int x = 0; x < 16; ++x, s += stride) v[x] = load_if(x0 + x < x1, s);
    float sum = 0.f;
    int row = x0 % m.rows;  // of the kv head
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float y = ex2_ftz(v[x] - lse[min(x0 + x, rows - 1)]);
      sum += x0 + x < x1 && row >= c0 ? y : 0.f;
      if (++row == m.rows) row = 0;
    }
    total.add(sum);
  }
  float got = total.get();
  if (p.sum_keys < kSumThreads) {
    __shared__ float sums[kSumThreads];
    static_assert(4 * kSumRows + sizeof(sums) <= 49152, "what a kernel has without asking for more");
    sums[threadIdx.x] = got;
    __syncthreads();
    if (part > 0) return;
    Total all;
    for (int i = 0; i < kSumThreads; i += p.sum_keys) all.add(sums[i + threadIdx.x]);
    got = all.get();
  }
  if (key >= m.seq) return;
  const int64_t o = (int64_t)slot * p.mass_stride + key;
  p.mass_out[o] = (key < m.seq - m.q_len ? p.decay * p.mass_in[o] : 0.f) + got;
}

// -------------------------------------------------------------- tcgen05 form

template <int D, bool F8>
struct WideGeo {
  static constexpr int kTileBytes = kTile * D * 2;            // 128 query rows (E4M3: two numbers)
  static constexpr int kImage = kTileBytes + kInfoBytes;
  static constexpr int kRowSpan = F8 ? D : 128;               // bytes of a swizzled row
  static constexpr int kHalf = kTile * 128;                   // 64 bf16 columns of 128 rows
};

__device__ __forceinline__ int tiles_of(const MassReq& m) {
  return m.wide ? (m.rows + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ int64_t steps_of(const MassParams& p, const MassReq& m) {
  return (int64_t)tiles_of(m) * p.Hkv * ((m.seq + kTile - 1) / kTile);
}

// 16-byte piece c of row `row` in swizzled rows of SPAN (128 or 64) bytes.
template <int SPAN>
__device__ __forceinline__ int swizzled(int row, int c) {
  return row * SPAN + ((SPAN == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
}

// One CTA per (row tile, kv head, request): the image of its 128 query rows.
template <int D, bool F8>
__global__ void __launch_bounds__(kTile) mass_rows_kernel(const __grid_constant__ MassParams p) {
  using W = WideGeo<D, F8>;
  grid_dependency_wait();  // the mirrors are there
  launch_dependents();
  const int ti = blockIdx.x, kvh = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
  const MassReq m = rows_of(p, r);
  const bool reporter = tid == 0 && ti == 0 && kvh == 0;
  const int tiles = tiles_of(m);
  if (reporter && m.wide && bad_request(m)) raise_error(p.err, kErrBounds);
  const int64_t first = before(p, r, [](const MassReq& x) -> int64_t { return tiles_of(x); });
  if (ti == 0 && kvh == 0) {
    const int64_t step = before(p, r, [&](const MassReq& x) { return steps_of(p, x); });
    if (tid == 0) p.first_step[r] = step;
    if (tid == 0 && r == p.R - 1) p.first_step[p.R] = step + steps_of(p, m);
  }
  if (!tiles) {
    if (reporter) p.tiled[r] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (ti >= tiles) return;
  const bool has_row = mass_row(p, r) >= 0;
  if (reporter) {
    p.tiled[r] = make_int4(has_row ? (int)first : -1, m.q0, m.q_len, m.seq);
    if (!has_row) raise_error(p.err, kErrBounds);
  }
  if (!has_row) return;
  const int tile = (int)first + ti;
  uint8_t* image = p.images + ((int64_t)tile * p.Hkv + kvh) * W::kImage;
  const int c = ti * kTile + tid;
  uint4 v[D / 8];
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + ((int64_t)(m.q0 + m.q_len - m.w + c / p.g) * p.Hq + kvh * p.g + c % p.g) * D);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) v[i] = c < m.rows ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
  float sc = fabsf(p.qk_scale);  // its sign goes to the query: greater products are greater scores
  if (p.qk_scale < 0.f) {
    constexpr uint32_t kSigns = 0x80008000u;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      v[i] = make_uint4(v[i].x ^ kSigns, v[i].y ^ kSigns, v[i].z ^ kSigns, v[i].w ^ kSigns);
  }
  if constexpr (!F8) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      *reinterpret_cast<uint4*>(image + (i >> 3) * W::kHalf + swizzled<128>(tid, i & 7)) = v[i];
  } else {
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      float f[8];
      bf16x8_to_f32(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        amax = fmaxf(amax, fabsf(f[e]));
        finite &= fabsf(f[e]) < INFINITY;
      }
    }
    int e2 = 0;  // the power of two that puts amax into [2^7, 2^8)
    if (amax > 0.f && finite)
      e2 = min(120, max(-120, 7 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127)));
    const float up = __uint_as_float((uint32_t)(e2 + 127) << 23);
    sc *= __uint_as_float((uint32_t)(127 - e2) << 23);
    if (!finite) sc = NAN;  // E4M3 has no infinities: the whole row is NaN, as its softmax is
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4& x = v[2 * i + (w >> 1)];
        const uint32_t pair[2] = {w & 1 ? x.z : x.x, w & 1 ? x.w : x.y};
        hi[w] = lo[w] = 0u;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float a = bf16_lo(pair[u]) * up, b = bf16_hi(pair[u]) * up;
          const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
          float ha, hb;
          e4m3x2_to_f32((uint16_t)h, ha, hb);
          const uint32_t l =
              __nv_cvt_float2_to_fp8x2(make_float2(a - ha, b - hb), __NV_SATFINITE, __NV_E4M3);
          hi[w] |= h << (16 * u);
          lo[w] |= l << (16 * u);
        }
      }
      const int at = swizzled<W::kRowSpan>(tid, i);
      *reinterpret_cast<uint4*>(image + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(image + kTile * D + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  reinterpret_cast<float*>(image + W::kTileBytes)[tid] = sc;
}

// Warps 0-15: rows or keys, each group of four the accumulators of every fourth step;
// 16: copies; 17 and 18: MMAs, of every other step (what one waits for before it may
// issue passes while the other's run; one warp alone left the tensor cores idle for
// 0.2 us a step).
constexpr int kGroups = 4;
constexpr int kMmaWarps = 2;
constexpr int kCopyWarp = 4 * kGroups, kMmaWarp = kCopyWarp + 1;
constexpr int kWideThreads = 32 * (kMmaWarp + kMmaWarps);
constexpr uint32_t kWideCols = kGroups * kTile;  // all of tensor memory
constexpr int kMaxKeyStages = 10;

struct WideTail {
  uint64_t image_full[2], image_empty[2];
  uint64_t full[kMaxKeyStages], empty[kMaxKeyStages];
  uint64_t s_full[kGroups], s_empty[kGroups];
  uint32_t tmem;
  int abort;
  alignas(16) float factors[kGroups][2 * kTile];  // WEIGHTS: what a group turns scores with
};

// Shared memory of a CTA, one on an SM: two images, and as many stages of 128 keys as
// there is room for.
template <int D, bool F8>
struct WideSmem {
  using W = WideGeo<D, F8>;
  static constexpr int kStage = kTile * D * (F8 ? 1 : 2);
  static constexpr int kRoom = 232448 - 1024 - (int)sizeof(WideTail) - 2 * W::kImage;
  static constexpr int kStages = kRoom / kStage > kMaxKeyStages ? kMaxKeyStages : kRoom / kStage;
  static constexpr int kOffKeys = 2 * W::kImage;
  static constexpr int kOffTail = kOffKeys + kStages * kStage;
  static constexpr size_t kAlloc = 1024 + kOffTail + sizeof(WideTail);
  static_assert(kStages >= 3 && W::kImage % 1024 == 0 && kStage % 1024 == 0 && kAlloc <= 232448,
                "swizzled tiles start on 1024-byte boundaries");
};

// A swizzled K-major operand tile of rows of SPAN bytes.
template <int SPAN>
__device__ __forceinline__ uint64_t operand_desc(const void* smem) {
  uint64_t d = tc::smem_desc_sw128(smem, 16, SPAN == 128 ? 1024 : 512);
  if (SPAN == 64) d = (d & ~(7ull << 61)) | (4ull << 61);  // 64-byte swizzle
  return d;
}

__device__ __forceinline__ float max16(const uint32_t (&v)[16]) {
  auto f = [&](int i) { return __uint_as_float(v[i]); };
  const float a = fmax3(f(0), f(1), f(2)), b = fmax3(f(3), f(4), f(5)), c = fmax3(f(6), f(7), f(8));
  const float d = fmax3(f(9), f(10), f(11)), e = fmax3(f(12), f(13), f(14));
  return fmaxf(fmax3(a, b, c), fmax3(d, e, f(15)));
}

// The part of a CTA's steps that one row tile of a kv head has, from flat step f on.
struct Segment {
  bool on;         // (false: of a request that was left out; nothing to do up to `next`)
  int tile, ti, kvh;
  int key_tile, n;  // first key tile, and how many
  int piece, pieces;  // of the row tile's pieces, and how many it has
  int64_t next;
  MassReq m;
  int r;
};
__device__ __forceinline__ Segment segment_at(const MassParams& p, int64_t f, int64_t end) {
  Segment s;
  s.r = warp_last_le(p.R, f, [&](int x) { return p.first_step[x]; });
  const int64_t base = p.first_step[s.r], over = p.first_step[s.r + 1];
  const int4 t = p.tiled[s.r];
  s.m = tiled_rows_of(p, t);
  s.tile = t.x;
  const int tiles = tiles_of(s.m), keys = (s.m.seq + kTile - 1) / kTile;
  s.on = s.tile >= 0;
  s.next = min(end, over);
  if (s.next <= f) s.next = end;  // (cannot be: f lies within the request)
  if (!s.on) return s;
  const int64_t unit = (f - base) / keys, start = base + unit * keys;
  s.kvh = (int)(unit / tiles);
  s.ti = (int)(unit - (int64_t)s.kvh * tiles);
  s.tile += s.ti;
  s.key_tile = (int)(f - start);
  s.n = (int)min((int64_t)keys - s.key_tile, end - f);
  s.piece = (int)(f / p.per_cta - start / p.per_cta);
  s.pieces = (int)min((start + keys - 1) / p.per_cta - start / p.per_cta + 1, (int64_t)p.pieces);
  s.next = f + s.n;
  return s;
}

// One CTA per SM on an equal run of the call's steps. WEIGHTS false: each row tile's
// statistics over the keys of the run (A, the lanes: query rows; B, the columns: keys).
// WEIGHTS true: of each step the weights summed over the tile's rows, key by key (A: keys;
// B: rows). A row tile's image stays in shared memory while its key tiles stream; the
// next tile's arrives meanwhile, and nothing drains between them.
// 4 x the last 64 queries (32 heads) on 14k to 33k E4M3 tokens: 103 us in all, 46 and 49 of
// them here, where the products take 24 at the tensor cores' rate, and as long for the reads
// of their operands from shared memory. A step's chain (product, reads of its accumulator,
// exponentials, barriers) takes 4200 cycles, 2400 of them in the reading warps; four are
// under way at once, which is all of tensor memory.
template <int D, bool F8, bool WEIGHTS>
__global__ void __launch_bounds__(kWideThreads, 1)
    mass_tile_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ MassParams p) {
  using W = WideGeo<D, F8>;
  using S = WideSmem<D, F8>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* images = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* keys = images + S::kOffKeys;
  WideTail* t = reinterpret_cast<WideTail*>(images + S::kOffTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t->image_full[i], 1);
      mbar_init(&t->image_empty[i], kMmaWarps + 4 * kGroups);  // the MMAs, and who reads its factors
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&t->full[i], 1);
      mbar_init(&t->empty[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&t->s_full[i], 1);
      mbar_init(&t->s_empty[i], 4);
    }
    t->abort = 0;
    fence_mbar_init();
  }
  launch_dependents();
  grid_dependency_wait();  // the images (and, for WEIGHTS, the rows' lse) are complete
  const int64_t begin = (int64_t)blockIdx.x * p.per_cta;
  const int64_t end = min(min(begin + p.per_cta, p.first_step[p.R]), p.steps);
  if (begin >= end) return;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&t->tmem, kWideCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = t->tmem;
  auto wait = [&](uint64_t* bar, unsigned parity) {  // the whole warp
    const bool ok = __all_sync(kFull, mbar_wait_quiet(bar, parity, &t->abort, p.err));
    if (!ok) *static_cast<volatile int*>(&t->abort) = 1;
    return ok;
  };

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------- copies
    constexpr int kCols = F8 ? 1 : D / 64;  // boxes across a key row
    constexpr int kBoxRow = F8 ? D : 128;
    const int per_tile = kTile / p.B;
    const int my_blk = lane / kCols, my_col = lane % kCols;  // what this lane brings of a tile
    int st = 0, segments = 0;
    unsigned phase = 1;  // of a stage's empty barrier, once all have been filled
    int64_t issued = 0;
    bool ok = true;
    for (int64_t f = begin; f < end && ok;) {
      const Segment s = segment_at(p, f, end);
      f = s.next;
      if (!s.on) continue;
      const int32_t* table = p.tables + (int64_t)s.r * p.max_blocks;
      auto block_at = [&](int key_tile) {
        const int64_t lb = (int64_t)key_tile * per_tile + my_blk;
        return my_blk < per_tile && lb * p.B < s.m.seq ? __ldg(table + lb) : -1;
      };
      int id = block_at(s.key_tile);
      const int slot = segments & 1;
      if (segments > 1) ok = wait(&t->image_empty[slot], (segments / 2 - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&t->image_full[slot], W::kImage);
        bulk_g2s(images + slot * W::kImage, p.images + ((int64_t)s.tile * p.Hkv + s.kvh) * W::kImage,
                 W::kImage, &t->image_full[slot]);
      }
      ++segments;
      for (int k = 0; k < s.n; ++k) {
        const int next = k + 1 < s.n ? block_at(s.key_tile + k + 1) : -1;
        if (issued >= kStages) ok = wait(&t->empty[st], phase);
        if (!ok) break;
        const int64_t lb = (int64_t)(s.key_tile + k) * per_tile + my_blk;
        const bool on = my_blk < per_tile && lb * p.B < s.m.seq;
        if (on && (id < 0 || id >= p.num_blocks)) {
          raise_error(p.err, kErrBounds);
          id = p.num_blocks;  // past the tensor map: keys of zeros
        }
        const unsigned boxes = __popc(__ballot_sync(kFull, on));
        if (lane == 0) mbar_arrive_expect_tx(&t->full[st], boxes * (unsigned)(p.B * kBoxRow));
        __syncwarp();
        if (on)
          tc::tma_load_3d(keys + st * S::kStage + my_col * W::kHalf + my_blk * p.B * kBoxRow, &tmap_k,
                          my_col * 64, s.kvh * p.B, id, &t->full[st]);
        id = next;
        ++issued;
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // what is in flight lands before the CTA ends
      for (int x = max(0, segments - 2); x < segments; ++x)
        mbar_wait(&t->image_full[x & 1], (x / 2) & 1, nullptr);
      for (int64_t x = max((int64_t)0, issued - kStages); x < issued; ++x)
        mbar_wait(&t->full[x % kStages], (unsigned)(x / kStages) & 1, nullptr);
    }
  } else if (warp >= kMmaWarp) {
    // --------------------------------------------------------------- MMAs
    constexpr uint32_t idesc =
        F8 ? tc::idesc_e4m3_f32(kTile, kTile) : tc::idesc_16bit_f32(kTile, kTile, false, false, false);
    const int mine = warp - kMmaWarp;
    int st = mine, segments = 0;
    unsigned phase = 0;
    int64_t i0 = 0;  // steps before the segment
    bool ok = true;
    for (int64_t f = begin; f < end && ok;) {
      const Segment s = segment_at(p, f, end);
      f = s.next;
      if (!s.on) continue;
      const int slot = segments & 1;
      ok = wait(&t->image_full[slot], (segments / 2) & 1);
      ++segments;
      const uint64_t rows = operand_desc<W::kRowSpan>(images + slot * W::kImage);
      for (int k = (int)((mine - i0) & (kMmaWarps - 1)); k < s.n; k += kMmaWarps) {
        const int64_t i = i0 + k;
        const int buf = (int)i & (kGroups - 1);
        ok = wait(&t->full[st], phase);
        if (ok && i >= kGroups) ok = wait(&t->s_empty[buf], (unsigned)(i / kGroups - 1) & 1);
        if (!ok) break;
        if (tc::elect_one()) {
          tc::fence_after_sync();
          const uint64_t key = operand_desc<W::kRowSpan>(keys + st * S::kStage);
          const uint32_t d = tmem + buf * kTile;
          if constexpr (F8) {
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int x = 0; x < D / 32; ++x) {
                const uint64_t q = tc::desc_at(rows, part * kTile * D + x * 32);
                const uint64_t c = tc::desc_at(key, x * 32);
                tc::mma_e4m3_ss(d, WEIGHTS ? c : q, WEIGHTS ? q : c, idesc, part > 0 || x > 0);
              }
          } else {
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const uint64_t q = tc::desc_at(rows, (x >> 2) * W::kHalf + (x & 3) * 32);
              const uint64_t c = tc::desc_at(key, (x >> 2) * W::kHalf + (x & 3) * 32);
              tc::mma_bf16_ss(d, WEIGHTS ? c : q, WEIGHTS ? q : c, idesc, x > 0);
            }
          }
          tc::mma_commit(&t->empty[st]);
          tc::mma_commit(&t->s_full[buf]);
        }
        __syncwarp();
        st += kMmaWarps;
        if (st >= kStages) {
          st -= kStages;
          phase ^= 1;
        }
      }
      i0 += s.n;
      if (tc::elect_one()) tc::mma_commit(&t->image_empty[slot]);  // when its MMAs are done
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------ rows, or keys
    const int group = warp >> 2, me = tid & (kTile - 1);  // the row, or key, of the tile
    const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + group * kTile;
    // WEIGHTS: a thread reads four keys of its warp's 32, me4 + 8 j, and of every eight
    // columns two, so that what belongs to a column is loaded for four weights at once
    const int me4 = (warp & 3) * 32 + (lane >> 2), col2 = lane & 3;
    int segments = 0;
    int64_t i0 = 0;  // steps before the segment
    bool ok = true;
    for (int64_t f = begin; f < end && ok;) {
      const Segment s = segment_at(p, f, end);
      const int64_t f0 = f;
      f = s.next;
      if (!s.on) continue;
      // (WEIGHTS: the warps of a group stop together, and none is still at the last segment's
      // factors when they are overwritten)
      if (WEIGHTS && named_bar_or(1 + group, kTile, !ok)) break;
      const int slot = segments & 1;
      ok = wait(&t->image_full[slot], (segments / 2) & 1);
      ++segments;
      const int first_row = s.ti * kTile;
      const int seen_by_all = s.m.seq - s.m.w;  // the last key that all counted queries see
      const float sc = reinterpret_cast<const float*>(images + slot * W::kImage + W::kTileBytes)[me];
      const int64_t unit = (int64_t)s.tile * p.Hkv + s.kvh;
      float* factors = t->factors[group];
      if (WEIGHTS) {  // (score factor, -lse) of rows 2 i and 2 i + 1, from the pieces' statistics
        const float2* part = p.tile_stats + unit * p.pieces * kGroups * kTile + me;
        factors[info_at(me)] = sc;
        factors[info_at(me) + 2] = -lse_of(part, s.pieces * kGroups, kTile);
        named_bar_sync(1 + group, kTile);
      }
      const uint64_t sc2 = f2_pack(sc, sc);
      const int sees = seen_by_all + min(first_row + me, s.m.rows - 1) / p.g + 1;  // keys of the row
      float total = 0.f, ref = -INFINITY;
      for (int k = (int)((group - i0) & (kGroups - 1)); k < s.n; k += kGroups) {
        if (!ok) break;
        ok = wait(&t->s_full[group], (unsigned)((i0 + k) / kGroups) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const int k0 = (s.key_tile + k) * kTile;
        if constexpr (!WEIGHTS) {
          // 16 columns at a time, the next 16 on their way; (16 columns') maximum first
          uint32_t v[2][16];
          auto columns = [&](const uint32_t (&w)[16], float mx) {
            const float top = fmaxf(ref, mx * sc), base = top == -INFINITY ? 0.f : top;  // sc is not negative
            total *= ex2_ftz(ref - base);
            ref = top;
            const uint64_t base2 = f2_pack(-base, -base);
            uint64_t a[2] = {0ull, 0ull};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x, y;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), sc2, base2), x, y);
              a[(e >> 1) & 1] = f2_add(a[(e >> 1) & 1], f2_pack(ex2_ftz(x), ex2_ftz(y)));
            }
            float a0, a1;
            f2_unpack(f2_add(a[0], a[1]), a0, a1);
            total += a0 + a1;
          };
          if (__all_sync(kFull, k0 + kTile <= sees)) {
            tc::tmem_ld16(acc, v[0]);
            tc::tmem_wait_ld(v[0]);
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c) {
              const uint32_t (&w)[16] = v[c & 1];
              if (c + 1 < kTile / 16) tc::tmem_ld16(acc + 16 * (c + 1), v[(c + 1) & 1]);
              columns(w, max16(w));
              if (c + 1 < kTile / 16) tc::tmem_wait_ld(v[(c + 1) & 1]);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < kTile; c += 16) {
              tc::tmem_ld16(acc + c, v[0]);
              tc::tmem_wait_ld(v[0]);
              float mx = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (k0 + c + e < sees) mx = fmaxf(mx, __uint_as_float(v[0][e]));
              const float top = fmaxf(ref, mx * sc), base = top == -INFINITY ? 0.f : top;
              total *= ex2_ftz(ref - base);
              ref = top;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (k0 + c + e < sees) total += ex2_ftz(fmaf(__uint_as_float(v[0][e]), sc, -base));
            }
          }
        } else {
          const float4* info = reinterpret_cast<const float4*>(factors);
          const int rows = min(kTile, s.m.rows - first_row);
          // rows from which on the warp's last key is seen (0 and below: all keys by all rows)
          const int after = k0 + (warp & 3) * 32 + 31 - seen_by_all;
          const int64_t from = (int64_t)max(0, after) * p.g - first_row;
          uint64_t a[4] = {0ull, 0ull, 0ull, 0ull};
          uint32_t v[2][16];
          if (from <= 0 && rows == kTile) {
            tc::tmem_ld16x256_x2(acc, v[0]);
            tc::tmem_wait_ld(v[0]);
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c) {
              const uint32_t (&u)[16] = v[c & 1];
              if (c + 1 < kTile / 16) tc::tmem_ld16x256_x2(acc + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const float4 q = info[8 * c + 4 * n + col2];
                const uint64_t factor = f2_pack(q.x, q.y), lse = f2_pack(q.z, q.w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t* w = &u[8 * (j >> 1) + 4 * n + 2 * (j & 1)];
                  float x, y;
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(w[0]), __uint_as_float(w[1])), factor, lse), x, y);
                  a[j] = f2_add(a[j], f2_pack(ex2_ftz(x), ex2_ftz(y)));
                }
              }
              if (c + 1 < kTile / 16) tc::tmem_wait_ld(v[(c + 1) & 1]);
            }
          } else {
            // the tile's first row that sees key j of the thread's
            int first[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              first[j] = (int)min((int64_t)max(0, k0 + me4 + 8 * j - seen_by_all) * p.g - first_row,
                                  (int64_t)kTile);
#pragma unroll 1
            for (int c = 0; c < rows; c += 16) {
              tc::tmem_ld16x256_x2(acc + c, v[0]);
              tc::tmem_wait_ld(v[0]);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const float4 q = info[(c >> 1) + 4 * n + col2];
                const int row = c + 8 * n + 2 * col2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t* w = &v[0][8 * (j >> 1) + 4 * n + 2 * (j & 1)];
                  const float x = ex2_ftz(fmaf(__uint_as_float(w[0]), q.x, q.z));
                  const float y = ex2_ftz(fmaf(__uint_as_float(w[1]), q.y, q.w));
                  a[j] = f2_add(a[j], f2_pack(row >= first[j] && row < rows ? x : 0.f,
                                              row + 1 >= first[j] && row + 1 < rows ? y : 0.f));
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            f2_unpack(a[j], x, y);
            x += y;
            x += __shfl_xor_sync(kFull, x, 1);
            x += __shfl_xor_sync(kFull, x, 2);
            if (col2 == 0) p.sums[(f0 + k) * kTile + me4 + 8 * j] = x;
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t->s_empty[group]);
      }
      i0 += s.n;
      if (!WEIGHTS)
        p.tile_stats[((unit * p.pieces + s.piece) * kGroups + group) * kTile + me] = make_float2(ref, total);
      __syncwarp();
      if (lane == 0) mbar_arrive(&t->image_empty[slot]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kWideCols);
}

// The steps' sums of each key, over the row tiles of all heads, into the mass.
__global__ void __launch_bounds__(kSumThreads) mass_add_kernel(const __grid_constant__ MassParams p) {
  grid_dependency_wait();
  const int r = blockIdx.y;
  const int4 t = p.tiled[r];
  if (t.x < 0) return;
  const MassReq m = tiled_rows_of(p, t);
  const int key = blockIdx.x * kSumThreads + (int)threadIdx.x;
  if (key >= m.seq) return;
  const int key_tiles = (m.seq + kTile - 1) / kTile, units = tiles_of(m) * p.Hkv;
  const float* s = p.sums + (p.first_step[r] + key / kTile) * kTile + key % kTile;
  const int64_t step = (int64_t)key_tiles * kTile;
  Total total;
  for (int u = 0; u < units; u += 16) {
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (u + i < units) part += s[(u + i) * step];
    total.add(part);
  }
  const int64_t o = (int64_t)mass_row(p, r) * p.mass_stride + key;
  p.mass_out[o] = (key < m.seq - m.q_len ? p.decay * p.mass_in[o] : 0.f) + total.get();
}

// ------------------------------------------------------------------- planning

struct MassPlan {
  int64_t score_floats, narrow, n_tiles, max_tiles, max_narrow_rows, steps, per_cta, ctas;
  int64_t narrow_keys, wide_keys;
  int splits, pieces, key_tiles, groups, stream_rows;
  size_t off_mirrors, off_stats, off_tiled, off_steps, off_images, off_tile_stats, off_sums, total;
};

// What a batch needs, from its mirrors alone (head_dim 128's images serve 64 too).
pa_status plan_mass(const int32_t* qsl, const int32_t* seq, int R, int Hq, int Hkv, int window,
                    MassPlan& pl) {
  pl = MassPlan{};
  const int64_t g = Hq / Hkv;
  int64_t narrow_keys = 0, wide_keys = 0;
  // The rows up to which keys are streamed, 16 rows at a time: 16, or 64 where no request
  // has more and what has more than 16 makes no more than a round of CTAs, so that the four
  // launches of the tcgen05 form do not run: 3 x 2 to 7 tokens of 40 heads on 130 tokens 14 us
  // instead of 46, 13 x 6 of 32 heads on 210 13 instead of 37. (Up to 128 rows and two rounds:
  // 2 x 16 tokens of 16 heads on 16 tokens 12 instead of 16, but 5 x 64 of 16 heads on 551 to
  // 1802, where the scores are written and read again, 60 instead of 26.)
  // (Of more kv heads than kSumRows / 16, fewer.)
  int64_t stream_rows = std::min((int64_t)kNarrowRows, kSumRows / (int64_t)Hkv), units = 0, most = 0;
  for (int r = 0; r < R; ++r) {
    const int64_t q_len = (int64_t)qsl[r + 1] - qsl[r];
    const int64_t rows = (window > 0 && q_len > window ? window : q_len) * g;
    if (rows > most) most = rows;
    if (rows > kNarrowRows)
      units += (rows + kNarrowRows - 1) / kNarrowRows * Hkv * ((seq[r] + (int64_t)kSplitKeys - 1) / kSplitKeys);
  }
  if (most <= kStreamRows && units <= kStreamUnits && Hkv * (int64_t)kStreamRows <= kSumRows)
    stream_rows = kStreamRows;
  int64_t wide_reqs = 0, with_rows = 0;
  for (int r = 0; r < R; ++r) {
    const int64_t q_len = (int64_t)qsl[r + 1] - qsl[r];
    if (q_len > 0) ++with_rows;
    if ((window > 0 && q_len > window ? window : q_len) * g > stream_rows) ++wide_reqs;
  }
  // (with them the requests without new tokens, so that one form flags what the device has of them)
  if (wide_reqs == with_rows) stream_rows = -1;
  pl.stream_rows = (int)stream_rows;
  for (int r = 0; r < R; ++r) {
    const int64_t q_len = (int64_t)qsl[r + 1] - qsl[r];
    if (q_len < 0 || (q_len > 0 && seq[r] < q_len)) return PA_ERR_INVALID;
    if (q_len == 0) continue;
    const int64_t rows = (window > 0 && q_len > window ? window : q_len) * g;
    if (rows > 0x3fffffff || seq[r] > kMostTokens) return PA_ERR_UNSUPPORTED;
    if (rows <= stream_rows) {
      ++pl.narrow;
      pl.score_floats += (int64_t)Hkv * rows * (((int64_t)seq[r] + 15) & ~15ll);
      if (seq[r] > narrow_keys) narrow_keys = seq[r];
      if (rows > pl.max_narrow_rows) pl.max_narrow_rows = rows;
    } else {
      const int64_t tiles = (rows + kTile - 1) / kTile;
      pl.n_tiles += tiles;
      if (tiles > pl.max_tiles) pl.max_tiles = tiles;
      if (seq[r] > wide_keys) wide_keys = seq[r];
      pl.steps += tiles * Hkv * (((int64_t)seq[r] + kTile - 1) / kTile);
    }
  }
  pl.narrow_keys = narrow_keys;
  pl.wide_keys = wide_keys;
  pl.splits = (int)((narrow_keys + kSplitKeys - 1) / kSplitKeys);
  pl.key_tiles = (int)((wide_keys + kTile - 1) / kTile);
  // An equal run of steps for each of 152 SMs (whatever the device has: the workspace's size
  // is asked for without one), but four at the least where that keeps the
  // pieces of a row tile, whose statistics are joined, below ten.
  const int64_t least = (pl.key_tiles + 7) / 8 < 4 ? (pl.key_tiles + 7) / 8 : 4;
  pl.per_cta = std::max((pl.steps + 151) / 152, std::max(least, (int64_t)1));
  pl.groups = (int)((pl.max_narrow_rows + kNarrowRows - 1) / kNarrowRows);
  pl.ctas = (pl.steps + pl.per_cta - 1) / pl.per_cta;
  pl.pieces = (int)((pl.key_tiles + pl.per_cta - 1) / pl.per_cta) + 1;
  if (pl.n_tiles > 0x7fffffff / (int64_t)Hkv || pl.max_tiles > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  auto up = [](size_t x) { return (x + 1023) & ~(size_t)1023; };
  size_t at = up((size_t)pl.score_floats * 4);
  pl.off_mirrors = at;
  if (with_rows && R > kFewReqs) at = up(at + (size_t)R * sizeof(int2));
  pl.off_stats = at;
  if (pl.narrow) at = up(at + (size_t)R * Hkv * pl.groups * kNarrowRows * pl.splits * sizeof(float2));
  pl.off_tiled = at;
  if (pl.n_tiles) at = up(at + (size_t)R * sizeof(int4));
  pl.off_steps = at;
  if (pl.n_tiles) at = up(at + ((size_t)R + 1) * sizeof(int64_t));
  pl.off_images = at;
  at = up(at + (size_t)pl.n_tiles * Hkv * WideGeo<128, false>::kImage);
  pl.off_tile_stats = at;
  at = up(at + (size_t)pl.n_tiles * Hkv * pl.pieces * kGroups * kTile * sizeof(float2));
  pl.off_sums = at;
  at = up(at + (size_t)pl.steps * kTile * sizeof(float));
  pl.total = at;
  return PA_OK;
}

// A pool's keys as [block][kv head * B + offset][dims], boxes of `rows` keys across
// 128 bytes (64 for E4M3 at head_dim 64), swizzled over as many.
bool key_map(CUtensorMap* m, const pa_kv_pool* pool, int rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const bool f8 = pool->dtype == PA_KV_FP8_E4M3;
  const cuuint64_t elt = f8 ? 1 : 2, D = (cuuint64_t)pool->head_dim;
  const cuuint64_t lines = (cuuint64_t)pool->num_kv_heads * pool->block_size;
  cuuint64_t dims[3] = {D, lines, (cuuint64_t)pool->num_blocks};
  cuuint64_t strides[2] = {D * elt, lines * D * elt};
  cuuint32_t box[3] = {(cuuint32_t)(f8 ? D : 64), (cuuint32_t)rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return encode(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                pool->k_pool, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                f8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dependent: the kernel may be scheduled before the one ahead of it has ended, and waits
// for that itself.
template <class... KArgs, class... Args>
pa_status launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem,
                       cudaStream_t s, bool dependent, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return launch_status();
}

pa_status set_mirrors(int2* out, const int32_t* qsl, const int32_t* seq, int R, cudaStream_t s) {
  for (int r0 = 0; r0 < R; r0 += kMirrorsAtOnce) {
    Mirrors m;
    const int n = std::min(R - r0, kMirrorsAtOnce);
    for (int i = 0; i < n; ++i) m.v[i] = make_int2(qsl[r0 + i + 1] - qsl[r0 + i], seq[r0 + i]);
    mass_mirrors_kernel<<<1, (n + 31) & ~31, 0, s>>>(out + r0, n, m);
    if (launch_status() != PA_OK) return PA_ERR_CUDA;
  }
  return PA_OK;
}

template <int D, bool F8>
pa_status run_mass(const MassParams& p, const MassPlan& pl, const pa_kv_pool* pool,
                   const int32_t* qsl_host, const int32_t* seq_host, cudaStream_t s) {
  static OncePerDevice once;
  constexpr size_t narrow_smem = 1024 + (size_t)kNarrowWarps * kNarrowRing + sizeof(NarrowTail);
  constexpr size_t wide_smem = WideSmem<D, F8>::kAlloc;
  if (!once.done([] {
        auto set = [](const void* f, size_t n) {
          return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)n) ==
                 cudaSuccess;
        };
        return set((const void*)mass_scores_kernel<D, F8, 1>, narrow_smem) &&
               set((const void*)mass_scores_kernel<D, F8, 2>, narrow_smem) &&
               set((const void*)mass_tile_kernel<D, F8, false>, wide_smem) &&
               set((const void*)mass_tile_kernel<D, F8, true>, wide_smem);
      }))
    return PA_ERR_CUDA;
  CUtensorMap tmap{}, tmap_tile{};
  if ((pl.narrow && !cell_map<D, F8>(&tmap, pool->k_pool, pool->num_blocks, p.Hkv * p.B)) ||
      (pl.n_tiles && !key_map(&tmap_tile, pool, p.B)))
    return PA_ERR_CUDA;
  const bool many = p.R > kFewReqs;
  pa_status st = many ? set_mirrors(const_cast<int2*>(p.mirrors), qsl_host, seq_host, p.R, s) : PA_OK;
  if (st != PA_OK) return st;
  if (pl.narrow) {
    const dim3 grid((unsigned)pl.splits, (unsigned)(p.Hkv * pl.groups), (unsigned)p.R);
    st = launch_after(pl.max_narrow_rows <= 8 ? mass_scores_kernel<D, F8, 1> : mass_scores_kernel<D, F8, 2>,
                      grid, kNarrowWarps * 32, narrow_smem, s, many, tmap, p);
    if (st != PA_OK) return st;
    st = launch_after(mass_sum_kernel, dim3((unsigned)((pl.narrow_keys + p.sum_keys - 1) / p.sum_keys), (unsigned)p.R),
                      kSumThreads, (size_t)p.Hkv * pl.max_narrow_rows * 4, s, true, p);
    if (st != PA_OK) return st;
  }
  if (!pl.n_tiles) return PA_OK;
  st = launch_after(mass_rows_kernel<D, F8>, dim3((unsigned)pl.max_tiles, (unsigned)p.Hkv, (unsigned)p.R),
                    kTile, 0, s, many && !pl.narrow, p);
  if (st != PA_OK) return st;
  const dim3 ctas((unsigned)pl.ctas);
  st = launch_after(mass_tile_kernel<D, F8, false>, ctas, kWideThreads, wide_smem, s, true, tmap_tile, p);
  if (st != PA_OK) return st;
  st = launch_after(mass_tile_kernel<D, F8, true>, ctas, kWideThreads, wide_smem, s, true, tmap_tile, p);
  if (st != PA_OK) return st;
  return launch_after(mass_add_kernel, dim3((unsigned)((pl.wide_keys + kSumThreads - 1) / kSumThreads), (unsigned)p.R),
                      kSumThreads, 0, s, true, p);
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_attention_mass_workspace_size(const int32_t* qsl_host,
                                                   const int32_t* seq_lens_host, int32_t num_reqs,
                                                   int32_t num_q_heads, int32_t num_kv_heads,
                                                   int32_t window) {
  if (num_reqs <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      window < 0 || !qsl_host || !seq_lens_host)
    return 0;
  pa::MassPlan pl;
  return pa::plan_mass(qsl_host, seq_lens_host, num_reqs, num_q_heads, num_kv_heads, window, pl) ==
                 PA_OK
             ? pl.total
             : 0;
}

extern "C" pa_status pa_attention_mass(
    const void* q, const float* mass_in, float* mass_out, int64_t mass_stride, int32_t max_reqs,
    const int32_t* idx_mapping, const int32_t* query_start_loc, const int32_t* seq_lens,
    const int32_t* qsl_host, const int32_t* seq_lens_host, const int32_t* block_tables,
    int32_t max_blocks, int32_t num_reqs, int32_t num_tokens, int32_t num_q_heads,
    const pa_kv_pool* pool, float scale, float decay, int32_t window, void* workspace,
    size_t workspace_bytes, pa_stream_t stream) {
  using namespace pa;
  pa_status st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks < 0 || max_reqs < 0 || mass_stride < 0 ||
      window < 0 || num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0)
    return PA_ERR_INVALID;
  if (num_reqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !aligned16(q) || !mass_in || !mass_out || (reinterpret_cast<uintptr_t>(mass_in) & 3u) ||
      (reinterpret_cast<uintptr_t>(mass_out) & 3u) || !query_start_loc || !seq_lens || !qsl_host ||
      !seq_lens_host || !block_tables || pool->num_blocks < 1)
    return PA_ERR_INVALID;
  if (qsl_host[0] != 0 || qsl_host[num_reqs] != num_tokens) return PA_ERR_INVALID;
  MassPlan pl;
  MassParams p{};
  st = plan_mass(qsl_host, seq_lens_host, num_reqs, num_q_heads, pool->num_kv_heads, window, pl);
  if (st != PA_OK) return st;
  for (int r = 0; r < num_reqs; ++r)
    if (qsl_host[r + 1] > qsl_host[r] && (seq_lens_host[r] > (int64_t)max_blocks * pool->block_size ||
                                          seq_lens_host[r] > mass_stride))
      return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < pl.total || !aligned16(workspace)) return PA_ERR_INVALID;
  if (num_reqs > 65535 || pool->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.mass_stride = mass_stride;
  p.idx = idx_mapping;
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.tables = block_tables;
  p.max_reqs = max_reqs;
  p.max_blocks = max_blocks;
  p.R = num_reqs;
  p.T = num_tokens;
  p.Hq = num_q_heads;
  p.Hkv = pool->num_kv_heads;
  p.g = num_q_heads / p.Hkv;
  p.B = pool->block_size;
  p.num_blocks = pool->num_blocks;
  p.window = window;
  p.decay = decay;
  const bool f8 = pool->dtype == PA_KV_FP8_E4M3;
  p.qk_scale = scale * 1.44269504088896340736f * (f8 ? pool->k_scale : 1.f);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.scores = pl.narrow ? reinterpret_cast<float*>(ws) : nullptr;
  p.mirrors = reinterpret_cast<const int2*>(ws + pl.off_mirrors);
  p.split_stats = reinterpret_cast<float2*>(ws + pl.off_stats);
  p.splits = pl.splits;
  p.groups = pl.groups;
  p.stream_rows = pl.stream_rows;
  for (int r = 0; r < num_reqs && num_reqs <= kFewReqs; ++r)
    p.few[r] = make_int2(qsl_host[r + 1] - qsl_host[r], seq_lens_host[r]);
  // Eight threads a key where a thread a key would leave SMs idle (3 decodes of 128 heads on
  // 200 tokens 9.6 us instead of 12.2, 13 x 4 to 6 tokens of 32 heads on 210 13 instead of
  // 28); else one, which joins the rows' statistics for more keys.
  p.sum_keys = (pl.narrow_keys + kSumThreads - 1) / kSumThreads * num_reqs <= num_sms() ? kSumThreads / 8 : kSumThreads;
  p.tiled = reinterpret_cast<int4*>(ws + pl.off_tiled);
  p.images = ws + pl.off_images;
  p.tile_stats = reinterpret_cast<float2*>(ws + pl.off_tile_stats);
  p.first_step = reinterpret_cast<int64_t*>(ws + pl.off_steps);
  p.sums = reinterpret_cast<float*>(ws + pl.off_sums);
  p.steps = pl.steps;
  p.per_cta = pl.per_cta;
  p.pieces = pl.pieces;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  auto run = [&](auto kernels) { return kernels(p, pl, pool, qsl_host, seq_lens_host, s); };
  if (pool->head_dim == 128) return f8 ? run(run_mass<128, true>) : run(run_mass<128, false>);
  return f8 ? run(run_mass<64, true>) : run(run_mass<64, false>);
}
