// attention_mass.cu — pa_attention_mass: for each stored token the sum, over the
// last queries of its request and all heads, of the softmax weights that it
// received, added to what it had received before.
//
// The weights need each row's maximum and sum over all keys first, so the work
// has two passes over the scores. A request's rows for one kv head are its
// counted queries times the g heads that share the kv head; two forms:
//
//  - up to 16 rows (decodes, drafted tokens): the keys are what costs. One pass
//    streams them once (warps with rings of 16-key cells, S^T = K Q^T by
//    warp-level MMAs with the keys as rows, as pa_sparse_forward), writes the
//    scores (4 g bytes a key against 2 D or D bytes of the key) to the
//    workspace and each split's row maxima and sums; the second joins those and
//    adds 2^(score - lse) over the rows, key by key, from L2.
//  - more rows (the last queries of a prompt): scores are made twice on tcgen05,
//    128 x 128 at a time, never leaving the SM. Pass 1 has query rows as the
//    accumulator's lanes, so that a thread owns a row and its running maximum
//    and sum; pass 2 has keys as lanes, S^T = K Q^T, so that a thread owns a key
//    and adds its weights in registers, over all rows of all heads: no atomics,
//    and the order of every sum follows from the sizes alone.
//    The query rows are laid out once per call as shared-memory images of 128
//    rows, swizzled as the tensor cores read them, which one bulk copy fetches;
//    behind each image its rows' score factors and, after pass 1, their lse.
//
// E4M3 pools: the codes are multiplied as they are. Up to 16 rows they widen to
// f16; on tcgen05 a query is the sum of two E4M3 numbers (8 significant bits, all
// that bf16 has) after a power-of-two scale that puts its row's largest magnitude
// into [2^7, 2^8): exact for elements down to 2^-8 of that one, off by 2^-18 of it
// below.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <utility>

#include "batch_rows.cuh"
#include "cells.cuh"
#include "mbar_poll.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNarrowRows = 16;     // rows of the streaming form, at the most
constexpr int kSplitKeys = 1024;    // keys of one of its CTAs
constexpr int kTile = 128;          // rows, and keys, of a tcgen05 tile
constexpr int kInfoBytes = 1024;    // behind an image: what its rows' scores are turned with
// Of rows 2 i and 2 i + 1 four floats, (factor, factor, -lse, -lse), so that one load
// feeds one packed multiply-add: the row's factor is at info_at(row), -lse 2 further.
__device__ __forceinline__ int info_at(int row) { return (row >> 1) * 4 + (row & 1); }

struct MassParams {
  const __nv_bfloat16* q;
  const float* mass_in;
  float* mass_out;
  int64_t mass_stride;
  const int32_t* idx;
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int32_t* tables;
  int max_reqs, max_blocks, R, T, Hq, Hkv, g, B, num_blocks, window;
  float decay, qk_scale;   // softmax scale * log2(e) (* k_scale)
  // streaming form
  float* scores;           // request after request: [Hkv * rows][keys rounded up to 16]
  int64_t score_floats;
  float2* split_stats;     // [R][Hkv][16][splits] (maximum, sum)
  int splits;
  int narrow_rows;         // rows of a request of this form, at the most
  // tcgen05 form
  int4* tile_of;           // [n_tiles] (request or -1, row tile, keys, counted queries)
  int* first_tile;         // [R], -1: not of this form
  uint8_t* images;         // [n_tiles][Hkv][image]
  float2* tile_stats;      // [n_tiles][Hkv][parts][128]
  int n_tiles, parts, part_keys;
  int key_tiles;           // key tiles of the longest request
  unsigned* err;
};

struct MassReq {
  int q0, q_len, seq, w, rows;  // w counted queries, rows = w * g
};

__device__ __forceinline__ MassReq rows_of(const MassParams& p, int q0, int end, int seq) {
  MassReq m;
  m.q0 = q0;
  m.q_len = end - q0;
  m.seq = seq;
  const bool fine = q0 >= 0 && end <= p.T && end >= q0 && seq >= m.q_len &&
                    seq <= (int64_t)p.max_blocks * p.B && seq <= p.mass_stride;
  m.w = fine ? (p.window > 0 ? min(m.q_len, p.window) : m.q_len) : 0;
  const int64_t rows = (int64_t)m.w * p.g;
  m.rows = rows > 0x3fffffff ? 0 : (int)rows;
  return m;
}
__device__ __forceinline__ MassReq rows_of(const MassParams& p, int r) {
  return rows_of(p, p.qsl[r], p.qsl[r + 1], p.seq_lens[r]);
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
  return m.rows > 0 && m.rows <= kNarrowRows ? (int64_t)p.Hkv * m.rows * padded_keys(m.seq) : 0;
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

// ------------------------------------------------------------ streaming form

constexpr int kNarrowWarps = 4;
constexpr int kNarrowRing = 24576;  // of a warp: two CTAs on an SM

struct NarrowTail {
  uint64_t full[kNarrowWarps][8];
  float2 stats[kNarrowWarps][kNarrowRows];
};

template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kNarrowWarps * 32, 2)
    mass_scores_kernel(const __grid_constant__ CUtensorMap tmap_k, MassParams p) {
  using C = Cells<D, FP8>;
  constexpr int kStages = kNarrowRing / C::kBytes > 8 ? 8 : kNarrowRing / C::kBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  NarrowTail* tail = reinterpret_cast<NarrowTail*>(ring + kNarrowWarps * kNarrowRing);
  launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tig = lane & 3;
  const int split = blockIdx.x, kvh = blockIdx.y, r = blockIdx.z;
  const MassReq m = rows_of(p, r);
  const bool reporter = tid == 0 && split == 0 && kvh == 0;
  if (bad_request(m) || (m.rows > kNarrowRows && p.n_tiles == 0) ||
      (m.rows > 0 && mass_row(p, r) < 0)) {
    if (reporter) raise_error(p.err, kErrBounds);
    return;
  }
  if (m.rows == 0 || m.rows > kNarrowRows) return;
  const int64_t at = before(p, r, [&](const MassReq& x) { return score_floats_of(p, x); });
  if (at + score_floats_of(p, m) > p.score_floats || m.seq > (int64_t)p.splits * kSplitKeys ||
      m.rows > p.narrow_rows) {
    if (reporter) raise_error(p.err, kErrBounds);  // more than the mirrors said
    return;
  }
  const int k0 = split * kSplitKeys;
  if (k0 >= m.seq) return;
  const int n_cells = (min(m.seq - k0, kSplitKeys) + kChunk - 1) / kChunk;
  const int stride = padded_keys(m.seq);
  float* out = p.scores + at + (int64_t)kvh * m.rows * stride;
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
      id_lane = 0;  // a valid block; the request's mass is then unspecified
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
    return c < m.rows ? p.q + ((int64_t)(m.q0 + m.q_len - m.w + c / p.g) * p.Hq + kvh * p.g + c % p.g) * D
                      : nullptr;
  }, p.qk_scale, grp, tig);
  float mx[NH][2], l[NH][2];
  int lim[NH][2];  // keys that the query of column 2 tig + e sees
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[h][e] = -INFINITY;
      l[h][e] = 0.f;
      lim[h][e] = m.seq - m.w + (8 * h + 2 * tig + e) / p.g + 1;
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
        if (c < m.rows) {
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
  if (tid < m.rows) {
    float ref = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kNarrowWarps; ++w) ref = fmaxf(ref, tail->stats[w][tid].x);
    const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int w = 0; w < kNarrowWarps; ++w)
      sum += tail->stats[w][tid].y * ex2_ftz(tail->stats[w][tid].x - base);
    p.split_stats[(((int64_t)r * p.Hkv + kvh) * kNarrowRows + tid) * p.splits + split] =
        make_float2(ref, sum);
  }
}

// Log of the sum of 2^score of a row, from `n` parts (maximum, sum) `step` apart.
__device__ __forceinline__ float lse_of(const float2* s, int n, int64_t step) {
  float ref = -INFINITY, sum = 0.f;
  for (int i = 0; i < n; ++i) ref = fmaxf(ref, s[i * step].x);
  const float base = ref == -INFINITY ? 0.f : ref;
  for (int i = 0; i < n; ++i) sum += s[i * step].y * ex2_ftz(s[i * step].x - base);
  return ref + log2f(sum);  // NaN for a row that scores -inf throughout
}

constexpr int kSumThreads = 256;

__global__ void __launch_bounds__(kSumThreads) mass_sum_kernel(MassParams p) {
  extern __shared__ float lse[];  // [Hkv * rows]
  const int r = blockIdx.y;
  const MassReq m = rows_of(p, r);
  if (m.rows == 0 || m.rows > p.narrow_rows || m.seq > (int64_t)p.splits * kSplitKeys) return;
  const int key0 = blockIdx.x * kSumThreads;
  if (key0 >= m.seq) return;
  const int64_t at = before(p, r, [&](const MassReq& x) { return score_floats_of(p, x); });
  if (at + score_floats_of(p, m) > p.score_floats) return;
  const int slot = mass_row(p, r);
  if (slot < 0) {
    if (threadIdx.x == 0) raise_error(p.err, kErrBounds);
    return;
  }
  grid_dependency_wait();  // the scores and their statistics are complete
  const int rows = p.Hkv * m.rows, n_split = (m.seq + kSplitKeys - 1) / kSplitKeys;
  for (int x = threadIdx.x >> 5; x < rows; x += kSumThreads / 32) {  // a warp for each row
    const float2* part = p.split_stats +
        ((int64_t)(r * (int64_t)p.Hkv + x / m.rows) * kNarrowRows + x % m.rows) * p.splits;
    const int lane = threadIdx.x & 31;
    float ref = -INFINITY, sum = 0.f;
    for (int i = lane; i < n_split; i += 32) join_stats(ref, sum, part[i].x, part[i].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      join_stats(ref, sum, __shfl_xor_sync(kFull, ref, o), __shfl_xor_sync(kFull, sum, o));
    if (lane == 0) lse[x] = ref + log2f(sum);  // NaN for a row that scores -inf throughout
  }
  __syncthreads();
  const int key = key0 + (int)threadIdx.x;
  if (key >= m.seq) return;
  const int stride = padded_keys(m.seq);
  const float* s = p.scores + at + key;
  float sum = 0.f;
  if (key <= m.seq - m.w) {  // seen by all counted queries
#pragma unroll 16
    for (int x = 0; x < rows; ++x) sum += ex2_ftz(s[(int64_t)x * stride] - lse[x]);
  } else {
    const int c0 = (key - (m.seq - m.w)) * p.g;  // the first row that sees the key
    for (int x = 0; x < rows; ++x)
      if (x % m.rows >= c0) sum += ex2_ftz(s[(int64_t)x * stride] - lse[x]);
  }
  const int64_t o = (int64_t)slot * p.mass_stride + key;
  p.mass_out[o] = (key < m.seq - m.q_len ? p.decay * p.mass_in[o] : 0.f) + sum;
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
  return m.rows > kNarrowRows ? (m.rows + kTile - 1) / kTile : 0;
}

// 16-byte piece c of row `row` in swizzled rows of SPAN (128 or 64) bytes.
template <int SPAN>
__device__ __forceinline__ int swizzled(int row, int c) {
  return row * SPAN + ((SPAN == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
}

// One CTA per (row tile, kv head, request): the image of its 128 query rows.
template <int D, bool F8>
__global__ void __launch_bounds__(kTile) mass_rows_kernel(MassParams p) {
  using W = WideGeo<D, F8>;
  launch_dependents();
  const int ti = blockIdx.x, kvh = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
  const MassReq m = rows_of(p, r);
  const bool reporter = tid == 0 && ti == 0 && kvh == 0;
  const int tiles = tiles_of(m);
  if (reporter && (bad_request(m) || (m.rows > 0 && !tiles && !p.scores))) raise_error(p.err, kErrBounds);
  if (r == p.R - 1 && ti == 0 && kvh == 0) {  // entries past the device's rows
    const int64_t end = before(p, r, [](const MassReq& x) -> int64_t { return tiles_of(x); }) + tiles;
    for (int64_t x = end + tid; x < p.n_tiles; x += kTile) p.tile_of[x] = make_int4(-1, 0, 0, 0);
  }
  if (!tiles) {
    if (reporter) p.first_tile[r] = -1;
    return;
  }
  if (ti >= tiles) return;
  const int64_t first = before(p, r, [](const MassReq& x) -> int64_t { return tiles_of(x); });
  const bool fits = first + tiles <= p.n_tiles && tiles <= (int)gridDim.x &&
                    (m.seq + kTile - 1) / kTile <= p.key_tiles &&
                    m.seq <= (int64_t)p.parts * p.part_keys && mass_row(p, r) >= 0;
  if (reporter) {
    p.first_tile[r] = fits ? (int)first : -1;
    if (!fits) raise_error(p.err, kErrBounds);
  }
  if (tid == 0 && kvh == 0) {
    if (first + ti < p.n_tiles) p.tile_of[first + ti] = make_int4(fits ? r : -1, ti, m.seq, m.w);
    // (no CTA comes to tiles past the grid's)
    if (ti == 0)
      for (int64_t x = first + gridDim.x; x < first + tiles && x < p.n_tiles; ++x)
        p.tile_of[x] = make_int4(-1, 0, 0, 0);
  }
  if (!fits) return;
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
  reinterpret_cast<float*>(image + W::kTileBytes)[info_at(tid)] = sc;
}

struct WideTail {
  uint64_t fixed_full[2], fixed_empty[2];
  uint64_t full[4], empty[4];      // stages of the streamed operand
  uint64_t info_full[8];           // WEIGHTS: what is behind a step's image
  uint64_t s_full[2], s_empty[2];  // accumulators
  uint32_t tmem;
  int abort;
  float part[2][kTile];            // results of the warpgroups, for each other and the cluster
};

// Warps 0-3 and 4-7: rows or keys, each group of four the accumulators of one stage
// (every other step); 8: copies; 9: MMAs.
constexpr int kWideThreads = 320;
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr uint32_t kWideCols = 2 * kTile;

// Shared memory of a CTA, two of which run on an SM: the tile that stays (WEIGHTS: two
// slots, the next kv head's keys arrive while this one's are multiplied), as many stages
// of the stream as there is room for (a stage is free again as soon as its MMAs are
// done), and a ring of eight steps' row factors. Two slots of 128 bf16 keys of 128 dims
// leave room for 64 query rows a stage.
template <int D, bool F8, bool WEIGHTS>
struct WideSmem {
  using W = WideGeo<D, F8>;
  static constexpr int kRows = WEIGHTS && !F8 && D == 128 ? 64 : kTile;  // columns of a step
  static constexpr int kKeys = kTile * D * (F8 ? 1 : 2);
  static constexpr int kSlots = WEIGHTS ? 2 : 1;
  static constexpr int kFixed = WEIGHTS ? kKeys : W::kImage;
  static constexpr int kStage = WEIGHTS ? kRows * D * 2 : kKeys;
  static constexpr int kRoom = (108 << 10) - kSlots * kFixed - 8 * kInfoBytes;
  static constexpr int kStages = kRoom / kStage > 4 ? 4 : kRoom / kStage;
  static constexpr int kOffStream = kSlots * kFixed;
  static constexpr int kOffInfo = kOffStream + kStages * kStage;
  static constexpr int kOffTail = kOffInfo + 8 * kInfoBytes;
  static constexpr size_t kAlloc = 1024 + kOffTail + sizeof(WideTail);
  static_assert(kStages >= 2 && kFixed % 1024 == 0 && kStage % 1024 == 0,
                "swizzled tiles start on 1024-byte boundaries");
};

// A swizzled K-major operand tile of rows of SPAN bytes.
template <int SPAN>
__device__ __forceinline__ uint64_t operand_desc(const void* smem) {
  uint64_t d = tc::smem_desc_sw128(smem, 16, SPAN == 128 ? 1024 : 512);
  if (SPAN == 64) d = (d & ~(7ull << 61)) | (4ull << 61);  // 64-byte swizzle
  return d;
}

// WEIGHTS false: the statistics of a row tile over one part of the keys (the row
// tile stays in shared memory, the key tiles stream). WEIGHTS true: the mass of a
// key tile (a kv head's keys stay, its row tiles stream), the kv heads shared by
// the CTAs of a cluster. Both multiply the tile that stays (A, the lanes) with
// each tile of the stream (B, the columns).
template <int D, bool F8, bool WEIGHTS>
__global__ void __launch_bounds__(kWideThreads, 2)
    mass_tile_kernel(const __grid_constant__ CUtensorMap tmap_k, MassParams p) {
  using W = WideGeo<D, F8>;
  using S = WideSmem<D, F8, WEIGHTS>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* fixed = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* stream = fixed + S::kOffStream;
  uint8_t* infos = fixed + S::kOffInfo;
  WideTail* t = reinterpret_cast<WideTail*>(fixed + S::kOffTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  launch_dependents();
  grid_dependency_wait();  // the images (and, for WEIGHTS, the rows' lse) are complete
  int r, tile0, n_steps, key0, n_tiles = 1, ti0 = 0, kvh0, kvh_step = 1;
  MassReq m;
  if (!WEIGHTS) {
    const int tile = blockIdx.x / p.Hkv;
    kvh0 = blockIdx.x - tile * p.Hkv;
    const int4 who = p.tile_of[tile];
    if (who.x < 0) return;
    r = who.x;
    m.q0 = m.q_len = 0;  // (not needed here)
    m.seq = who.z;
    m.w = who.w;
    m.rows = m.w * p.g;
    tile0 = tile;
    ti0 = who.y;
    key0 = blockIdx.y * p.part_keys;
    // the keys that the tile's last row sees
    const int last = min(m.rows - 1, ti0 * kTile + kTile - 1) / p.g;
    const int end = min(m.seq - m.w + last + 1, key0 + p.part_keys);
    n_steps = max(0, (end - key0 + kTile - 1) / kTile);
    if (n_steps == 0) {
      if (tid < kTile)
        p.tile_stats[(((int64_t)tile0 * p.Hkv + kvh0) * p.parts + blockIdx.y) * kTile + tid] =
            make_float2(-INFINITY, 0.f);
      return;
    }
  } else {
    r = blockIdx.y;
    tile0 = p.first_tile[r];
    if (tile0 < 0) return;
    m = rows_of(p, r);
    key0 = blockIdx.x * kTile;
    if (key0 >= m.seq) return;
    // row tiles whose last query comes before the tile's first key add nothing
    ti0 = (int)((int64_t)max(0, key0 - (m.seq - m.w)) * p.g / S::kRows);
    n_tiles = (m.rows + S::kRows - 1) / S::kRows - ti0;
    kvh0 = blockIdx.z;
    kvh_step = gridDim.z;
    n_steps = kvh0 < p.Hkv ? ((p.Hkv - kvh0 + kvh_step - 1) / kvh_step) * n_tiles : 0;
  }

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t->fixed_full[i], 1);
      mbar_init(&t->fixed_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&t->full[i], 1);
      mbar_init(&t->empty[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&t->info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t->s_full[i], 1);
      mbar_init(&t->s_empty[i], 4);
    }
    t->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&t->tmem, kWideCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = t->tmem;
  auto wait = [&](uint64_t* bar, unsigned parity) {
    const bool ok = mbar_wait_quiet(bar, parity, &t->abort, p.err);
    if (!ok) *static_cast<volatile int*>(&t->abort) = 1;
    return ok;
  };
  float total = 0.f, ref = -INFINITY;
  if (warp == kCopyWarp) {
    // ------------------------------------------------------------- copies
    constexpr int kCols = F8 ? 1 : D / 64;  // boxes across a key row
    const int32_t* table = p.tables + (int64_t)r * p.max_blocks;
    const int per_tile = kTile / p.B;
    constexpr int kBoxRow = F8 ? D : 128;
    // the block that this lane brings of the tile at key k0, -1 past the keys
    const int my_blk = lane / kCols, my_col = lane % kCols;
    auto block_at = [&](int64_t k0) {
      const int64_t lb = k0 / p.B + my_blk;
      return my_blk < per_tile && lb * p.B < m.seq ? __ldg(table + lb) : -1;
    };
    auto load_keys = [&](uint8_t* dst, int64_t k0, int id, int kvh, uint64_t* bar) {
      bool on = my_blk < per_tile && (k0 / p.B + my_blk) * p.B < m.seq;
      if (on && (id < 0 || id >= p.num_blocks)) {
        raise_error(p.err, kErrBounds);
        on = false;
      }
      const unsigned boxes = __popc(__ballot_sync(kFull, on));
      if (lane == 0) mbar_arrive_expect_tx(bar, boxes * (unsigned)(p.B * kBoxRow));
      __syncwarp();
      if (on)
        tc::tma_load_3d(dst + my_col * W::kHalf + my_blk * p.B * kBoxRow, &tmap_k, my_col * 64,
                        kvh * p.B, id, bar);
    };
    auto image_of = [&](int tile, int kvh) {
      return p.images + ((int64_t)tile * p.Hkv + kvh) * W::kImage;
    };
    auto copy = [&](void* dst, const uint8_t* src, unsigned bytes, uint64_t* bar) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(dst, src, bytes, bar);
      }
    };
    int i = 0, fixed_loads = 0;
    bool ok = true;
    int id = block_at(key0);  // of the next key tile (WEIGHTS: the only one)
    int kvh = kvh0, ti = ti0, st = 0;
    unsigned st_phase = 1;  // of the stage's empty barrier, once all have been filled
    if (!WEIGHTS) {
      copy(fixed, image_of(tile0, kvh0), W::kImage, &t->fixed_full[0]);
      fixed_loads = 1;
    }
    for (; i < n_steps && ok; ++i) {
      if (WEIGHTS && ti == ti0) {
        const int slot = fixed_loads & 1;
        if (fixed_loads > 1) ok = __all_sync(kFull, wait(&t->fixed_empty[slot], (fixed_loads / 2 - 1) & 1));
        if (!ok) break;
        load_keys(fixed + slot * S::kFixed, key0, id, kvh, &t->fixed_full[slot]);
        ++fixed_loads;
      }
      if (i >= kStages) ok = __all_sync(kFull, wait(&t->empty[st], st_phase));
      if (!ok) break;
      uint8_t* dst = stream + st * S::kStage;
      if (WEIGHTS) {
        constexpr int kParts = kTile / S::kRows;  // steps of an image
        const uint8_t* image = image_of(tile0 + ti / kParts, kvh);
        if constexpr (kParts == 1) {
          copy(dst, image, W::kTileBytes, &t->full[st]);
        } else if (lane == 0) {  // its rows of both halves
          constexpr int kPiece = S::kRows * 128;
          mbar_arrive_expect_tx(&t->full[st], 2 * kPiece);
          for (int h = 0; h < 2; ++h)
            bulk_g2s(dst + h * kPiece, image + h * W::kHalf + ti % kParts * kPiece, kPiece, &t->full[st]);
        }
        // Slot i mod 8 has been read: the stage is free since step i - kStages' MMAs are done,
        // and those waited until step i - kStages - 2, of the same accumulator, had been read.
        static_assert(kStages + 2 <= 8, "the ring of row factors");
        copy(infos + (i & 7) * kInfoBytes, image + W::kTileBytes + ti % kParts * S::kRows * 8,
             S::kRows * 8, &t->info_full[i & 7]);
        if (++ti == ti0 + n_tiles) {
          ti = ti0;
          kvh += kvh_step;
        }
      } else {
        const int64_t k0 = (int64_t)key0 + i * kTile;
        const int next = i + 1 < n_steps ? block_at(k0 + kTile) : -1;
        load_keys(dst, k0, id, kvh0, &t->full[st]);
        id = next;
      }
      if (++st == kStages) {
        st = 0;
        st_phase ^= 1;
      }
    }
    if (!ok) {  // what is in flight lands before the CTA ends
      for (int x = max(0, fixed_loads - 2); x < fixed_loads; ++x)
        mbar_wait(&t->fixed_full[x & 1], (x / 2) & 1, nullptr);
      for (int x = max(0, i - kStages); x < i; ++x)
        mbar_wait(&t->full[x % kStages], (x / kStages) & 1, nullptr);
      if (WEIGHTS)
        for (int x = max(0, i - 8); x < i; ++x) mbar_wait(&t->info_full[x & 7], (x >> 3) & 1, nullptr);
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------------- MMAs
    if (tc::elect_one()) {
      constexpr uint32_t idesc =
          F8 ? tc::idesc_e4m3_f32(kTile, S::kRows)
             : tc::idesc_16bit_f32(kTile, S::kRows, false, false, false);
      int heads = 0, left = 0, st = -1;  // left: steps with the tile that stays
      unsigned st_phase = 1;
      for (int i = 0; i < n_steps; ++i) {
        const int buf = i & 1;
        st = st + 1 == kStages ? 0 : st + 1;
        if (st == 0) st_phase ^= 1;
        if (left == 0) {
          left = WEIGHTS ? n_tiles : n_steps;
          if (!wait(&t->fixed_full[heads & 1], (heads / 2) & 1)) break;
          ++heads;
        }
        const int slot = (heads - 1) & 1;
        if (!wait(&t->full[st], st_phase)) break;
        if (i >= 2 && !wait(&t->s_empty[buf], ((i >> 1) - 1) & 1)) break;
        tc::fence_after_sync();
        const uint64_t a0 = operand_desc<W::kRowSpan>(fixed + slot * S::kFixed);
        const uint64_t b0 = operand_desc<W::kRowSpan>(stream + st * S::kStage);
        const uint32_t d = tmem + buf * kTile;
        if constexpr (F8) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              tc::mma_e4m3_ss(d, tc::desc_at(a0, (WEIGHTS ? 0 : part * kTile * D) + k * 32),
                              tc::desc_at(b0, (WEIGHTS ? part * kTile * D : 0) + k * 32), idesc,
                              part > 0 || k > 0);
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_bf16_ss(d, tc::desc_at(a0, (k >> 2) * W::kHalf + (k & 3) * 32),
                            tc::desc_at(b0, (k >> 2) * (WEIGHTS ? S::kRows * 128 : W::kHalf) + (k & 3) * 32), idesc,
                            k > 0);
        }
        tc::mma_commit(&t->empty[st]);
        tc::mma_commit(&t->s_full[buf]);
        if (--left == 0 && WEIGHTS) tc::mma_commit(&t->fixed_empty[slot]);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ rows, or keys
    const int me = tid & (kTile - 1);  // the thread's row, or key, of the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    float sc = 0.f;
    int sees = 0;  // !WEIGHTS: keys that the thread's row sees
    if (!WEIGHTS && n_steps > 0) {
      if (wait(&t->fixed_full[0], 0))
        sc = reinterpret_cast<const float*>(fixed + W::kTileBytes)[info_at(me)];
      sees = m.seq - m.w + min(ti0 * kTile + me, m.rows - 1) / p.g + 1;
    }
    // WEIGHTS: a thread reads four keys of its warp's 32, me4 + 8 j, and of every eight
    // columns two, so that what belongs to a column is loaded for four weights at once;
    // their sums, and what the roundings of those lost
    const int me4 = (warp & 3) * 32 + (lane >> 2), col2 = lane & 3;
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
    const int buf = warp >> 2;
    int ti = ti0 + buf;  // WEIGHTS: the step's row tile
    while (WEIGHTS && ti >= ti0 + n_tiles) ti -= n_tiles;
    for (int i = buf; i < n_steps; i += 2) {
      if (!__all_sync(kFull, (!WEIGHTS || wait(&t->info_full[i & 7], (i >> 3) & 1)) &&
                                 wait(&t->s_full[buf], (i >> 1) & 1)))
        break;
      tc::fence_after_sync();
      const uint32_t s = tmem + lane_base + buf * kTile;
      if (!WEIGHTS) {
        const int k0 = key0 + i * kTile;
        const bool whole = __all_sync(kFull, k0 + kTile <= sees);
        const uint64_t sc2 = f2_pack(sc, sc);
#pragma unroll
        for (int c = 0; c < kTile; c += 32) {
          uint32_t v[32];
          tc::tmem_ld32(s + c, v);
          tc::tmem_wait_ld();
          if (!whole)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k0 + c + e >= sees) v[e] = 0xff800000u;  // -inf
          float mx = __uint_as_float(v[0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            mx = fmax3(mx, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          mx = fmaxf(mx, __uint_as_float(v[31])) * sc;  // sc is not negative
          if (mx > ref) {
            total *= ex2_ftz(ref - mx);
            ref = mx;
          }
          const float base = ref == -INFINITY ? 0.f : ref;
          const uint64_t base2 = f2_pack(-base, -base);
          uint64_t a[2] = {0ull, 0ull};
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x, y;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, base2), x, y);
              a[(e >> 1) & 1] = f2_add(a[(e >> 1) & 1], f2_pack(ex2_ftz(x), ex2_ftz(y)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x, y;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, base2), x, y);
              x = k0 + c + e < sees ? ex2_ftz(x) : 0.f;  // (a factor of 0 times -inf is NaN)
              y = k0 + c + e + 1 < sees ? ex2_ftz(y) : 0.f;
              a[(e >> 1) & 1] = f2_add(a[(e >> 1) & 1], f2_pack(x, y));
            }
          }
          float a0, a1;
          f2_unpack(f2_add(a[0], a[1]), a0, a1);
          total += a0 + a1;
        }
      } else {
        const float4* info = reinterpret_cast<const float4*>(infos + (i & 7) * kInfoBytes);
        const int row0 = ti * S::kRows;
        ti += 2;
        while (ti >= ti0 + n_tiles) ti -= n_tiles;
        const int rows = min(S::kRows, m.rows - row0);
        // rows from which on the warp's last key is seen (0 and below: all keys by all rows)
        const int after = key0 + (warp & 3) * 32 + 31 - (m.seq - m.w);
        const int64_t from = (int64_t)max(0, after) * p.g - row0;
        uint64_t a[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < S::kRows; c += 32) {
          uint32_t v[2][16];
          tc::tmem_ld16x256_x4(s + c, v[0]);
          tc::tmem_ld16x256_x4(s + (16u << 16) + c, v[1]);
          tc::tmem_wait_ld();
          if (from <= c && c + 32 <= rows) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float4 f = info[(c >> 1) + 4 * n + col2];
              const uint64_t factor = f2_pack(f.x, f.y), lse = f2_pack(f.z, f.w);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* w = &v[j >> 1][4 * n + 2 * (j & 1)];
                float x, y;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(w[0]), __uint_as_float(w[1])), factor, lse), x, y);
                a[j] = f2_add(a[j], f2_pack(ex2_ftz(x), ex2_ftz(y)));
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // the tile's first row that sees the key
              const int64_t first64 = (int64_t)max(0, key0 + me4 + 8 * j - (m.seq - m.w)) * p.g - row0;
              const int first = (int)min(first64, (int64_t)kTile);
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                const float4 f = info[(c >> 1) + 4 * n + col2];
                const uint32_t* w = &v[j >> 1][4 * n + 2 * (j & 1)];
                const int row = c + 8 * n + 2 * col2;
                const float x = ex2_ftz(fmaf(__uint_as_float(w[0]), f.x, f.z));
                const float y = ex2_ftz(fmaf(__uint_as_float(w[1]), f.y, f.w));
                a[j] = f2_add(a[j], f2_pack(row >= first && row < rows ? x : 0.f,
                                            row + 1 >= first && row + 1 < rows ? y : 0.f));
              }
            }
          }
        }
        // one sum of up to millions of weights: the rounding of each addition is kept
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a0, a1;
          f2_unpack(a[j], a0, a1);
          const float add = (a0 + a1) + low[j];
          const float next = sum[j] + add;
          low[j] = add - (next - sum[j]);
          sum[j] = next;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&t->s_empty[buf]);
    }
    if (!WEIGHTS) {
      if (buf == 1) t->part[0][me] = ref, t->part[1][me] = total;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = sum[j] + (isnan(low[j]) ? 0.f : low[j]);  // (a NaN sum has lost no rounding)
        x += __shfl_xor_sync(kFull, x, 1);
        x += __shfl_xor_sync(kFull, x, 2);
        if (col2 == 0) t->part[buf][me4 + 8 * j] = x;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kWideCols);
  if (!WEIGHTS) {
    if (warp < 4) {
      join_stats(ref, total, t->part[0][tid], t->part[1][tid]);
      p.tile_stats[(((int64_t)tile0 * p.Hkv + kvh0) * p.parts + blockIdx.y) * kTile + tid] =
          make_float2(ref, total);
    }
    return;
  }
  if (warp < 4) total = t->part[0][tid] + t->part[1][tid];
  if (gridDim.z > 1) {
    if (warp < 4) t->part[0][tid] = total;  // (read by this thread alone)
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (blockIdx.z == 0 && warp < 4) {
      total = 0.f;
      for (unsigned c = 0; c < gridDim.z; ++c) total += *cluster.map_shared_rank(&t->part[0][tid], c);
    }
    cluster.sync();
  }
  if (blockIdx.z == 0 && warp < 4 && key0 + tid < m.seq) {
    const int64_t o = (int64_t)mass_row(p, r) * p.mass_stride + key0 + tid;
    p.mass_out[o] = (key0 + tid < m.seq - m.q_len ? p.decay * p.mass_in[o] : 0.f) + total;
  }
}

// The rows' lse into the images, from the parts' statistics.
template <int D, bool F8>
__global__ void __launch_bounds__(kTile) mass_join_kernel(MassParams p) {
  using W = WideGeo<D, F8>;
  launch_dependents();
  grid_dependency_wait();
  const int tile = blockIdx.x / p.Hkv;
  const int4 who = p.tile_of[tile];
  if (who.x < 0) return;
  const int n = min(p.parts, (who.z + p.part_keys - 1) / p.part_keys);
  float* info =
      reinterpret_cast<float*>(p.images + (int64_t)blockIdx.x * W::kImage + W::kTileBytes);
  info[info_at(threadIdx.x) + 2] =
      -lse_of(p.tile_stats + (int64_t)blockIdx.x * p.parts * kTile + threadIdx.x, n, kTile);
}

// ------------------------------------------------------------------- planning

struct MassPlan {
  int64_t score_floats, narrow, n_tiles, max_tiles, max_narrow_rows, sum_key_tiles;
  int splits, parts, part_keys, key_tiles, narrow_keys;
  size_t off_stats, off_tile_of, off_first, off_images, off_tile_stats, total;
};

// What a batch needs, from its mirrors alone (head_dim 128's images serve 64 too).
pa_status plan_mass(const int32_t* qsl, const int32_t* seq, int R, int Hq, int Hkv, int window,
                    MassPlan& pl) {
  pl = MassPlan{};
  const int64_t g = Hq / Hkv;
  int64_t steps = 0;  // of pass 1: row tiles x kv heads x key tiles
  int narrow_keys = 0, wide_keys = 0;
  for (int r = 0; r < R; ++r) {
    const int64_t q_len = (int64_t)qsl[r + 1] - qsl[r];
    if (q_len < 0 || (q_len > 0 && seq[r] < q_len)) return PA_ERR_INVALID;
    if (q_len == 0) continue;
    const int64_t rows = (window > 0 && q_len > window ? window : q_len) * g;
    if (rows > 0x3fffffff) return PA_ERR_UNSUPPORTED;
    if (rows <= kNarrowRows) {
      ++pl.narrow;
      pl.score_floats += (int64_t)Hkv * rows * (((int64_t)seq[r] + 15) & ~15ll);
      if (seq[r] > narrow_keys) narrow_keys = seq[r];
      if (rows > pl.max_narrow_rows) pl.max_narrow_rows = rows;
    } else {
      const int64_t tiles = (rows + kTile - 1) / kTile;
      pl.n_tiles += tiles;
      if (tiles > pl.max_tiles) pl.max_tiles = tiles;
      if (seq[r] > wide_keys) wide_keys = seq[r];
      steps += tiles * Hkv * ((seq[r] + kTile - 1) / kTile);
      pl.sum_key_tiles += (seq[r] + kTile - 1) / kTile;
    }
  }
  pl.narrow_keys = narrow_keys;
  pl.splits = (narrow_keys + kSplitKeys - 1) / kSplitKeys;
  pl.key_tiles = (wide_keys + kTile - 1) / kTile;
  // Parts of the keys in pass 1, of 4 to 32 key tiles: 1216 CTAs and more, of which 304 run
  // at once on 152 SMs.
  int64_t per = (steps + 1215) / 1216;
  per = per < 4 ? 4 : per > 32 ? 32 : per;
  pl.part_keys = (int)per * kTile;
  pl.parts = (wide_keys + pl.part_keys - 1) / pl.part_keys;
  if (pl.n_tiles > 0x7fffffff / (int64_t)Hkv || pl.max_tiles > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  auto up = [](size_t x) { return (x + 1023) & ~(size_t)1023; };
  size_t at = up((size_t)pl.score_floats * 4);
  pl.off_stats = at;
  if (pl.narrow) at = up(at + (size_t)R * Hkv * kNarrowRows * pl.splits * sizeof(float2));
  pl.off_tile_of = at;
  at = up(at + (size_t)pl.n_tiles * sizeof(int4));
  pl.off_first = at;
  if (pl.n_tiles) at = up(at + (size_t)R * sizeof(int));
  pl.off_images = at;
  at = up(at + (size_t)pl.n_tiles * Hkv * WideGeo<128, false>::kImage);
  pl.off_tile_stats = at;
  at = up(at + (size_t)pl.n_tiles * Hkv * pl.parts * kTile * sizeof(float2));
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

template <class... KArgs, class... Args>
pa_status launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem,
                       cudaStream_t s, bool dependent, unsigned cluster_z, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  unsigned n = 0;
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster_z > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = cluster_z;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return launch_status();
}

template <int D, bool F8>
pa_status run_mass(const MassParams& p, const MassPlan& pl, const pa_kv_pool* pool,
                   cudaStream_t s) {
  static OncePerDevice once;
  constexpr size_t narrow_smem = 1024 + (size_t)kNarrowWarps * kNarrowRing + sizeof(NarrowTail);
  constexpr size_t stats_smem = WideSmem<D, F8, false>::kAlloc, sum_smem = WideSmem<D, F8, true>::kAlloc;
  if (!once.done([] {
        auto set = [](const void* f, size_t n) {
          return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)n) ==
                 cudaSuccess;
        };
        return set((const void*)mass_scores_kernel<D, F8, 1>, narrow_smem) &&
               set((const void*)mass_scores_kernel<D, F8, 2>, narrow_smem) &&
               set((const void*)mass_tile_kernel<D, F8, false>, stats_smem) &&
               set((const void*)mass_tile_kernel<D, F8, true>, sum_smem);
      }))
    return PA_ERR_CUDA;
  CUtensorMap tmap{};
  pa_status st = PA_OK;
  if (pl.narrow) {
    if (!cell_map<D, F8>(&tmap, pool->k_pool, pool->num_blocks, p.Hkv * p.B)) return PA_ERR_CUDA;
    const dim3 grid((unsigned)pl.splits, (unsigned)p.Hkv, (unsigned)p.R);
    st = launch_after(pl.max_narrow_rows <= 8 ? mass_scores_kernel<D, F8, 1> : mass_scores_kernel<D, F8, 2>,
                      grid, kNarrowWarps * 32, narrow_smem, s, false, 1, tmap, p);
    if (st != PA_OK) return st;
    st = launch_after(mass_sum_kernel, dim3((unsigned)((pl.narrow_keys + kSumThreads - 1) / kSumThreads), (unsigned)p.R),
                      kSumThreads, (size_t)p.Hkv * pl.max_narrow_rows * 4, s, true, 1, p);
    if (st != PA_OK) return st;
  }
  if (!pl.n_tiles) return PA_OK;
  if (!key_map(&tmap, pool, p.B)) return PA_ERR_CUDA;
  st = launch_after(mass_rows_kernel<D, F8>, dim3((unsigned)pl.max_tiles, (unsigned)p.Hkv, (unsigned)p.R),
                    kTile, 0, s, false, 1, p);
  if (st != PA_OK) return st;
  st = launch_after(mass_tile_kernel<D, F8, false>, dim3((unsigned)(pl.n_tiles * p.Hkv), (unsigned)p.parts),
                    kWideThreads, stats_smem, s, true, 1, tmap, p);
  if (st != PA_OK) return st;
  st = launch_after(mass_join_kernel<D, F8>, dim3((unsigned)(pl.n_tiles * p.Hkv)), kTile, 0, s, true, 1, p);
  if (st != PA_OK) return st;
  // a cluster shares the kv heads of a key tile while there are less than four rounds of CTAs
  unsigned share = 1;
  while (share < 8 && (int)share * 2 <= p.Hkv && pl.sum_key_tiles * share < 8 * num_sms()) share *= 2;
  return launch_after(mass_tile_kernel<D, F8, true>, dim3((unsigned)pl.key_tiles, (unsigned)p.R, share),
                      kWideThreads, sum_smem, s, true, share, tmap, p);
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
  st = plan_mass(qsl_host, seq_lens_host, num_reqs, num_q_heads, pool->num_kv_heads, window, pl);
  if (st != PA_OK) return st;
  for (int r = 0; r < num_reqs; ++r)
    if (qsl_host[r + 1] > qsl_host[r] && (seq_lens_host[r] > (int64_t)max_blocks * pool->block_size ||
                                          seq_lens_host[r] > mass_stride))
      return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < pl.total || !aligned16(workspace)) return PA_ERR_INVALID;
  if (num_reqs > 65535 || pool->num_kv_heads > 65535 || pl.parts > 65535 ||
      pool->num_kv_heads * pl.max_narrow_rows > 12288)
    return PA_ERR_UNSUPPORTED;
  MassParams p{};
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
  p.score_floats = pl.score_floats;
  p.split_stats = reinterpret_cast<float2*>(ws + pl.off_stats);
  p.splits = pl.splits;
  p.narrow_rows = (int)pl.max_narrow_rows;
  p.tile_of = reinterpret_cast<int4*>(ws + pl.off_tile_of);
  p.first_tile = reinterpret_cast<int*>(ws + pl.off_first);
  p.images = ws + pl.off_images;
  p.tile_stats = reinterpret_cast<float2*>(ws + pl.off_tile_stats);
  p.n_tiles = (int)pl.n_tiles;
  p.parts = pl.parts;
  p.part_keys = pl.part_keys;
  p.key_tiles = pl.key_tiles;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  if (pool->head_dim == 128)
    return f8 ? run_mass<128, true>(p, pl, pool, s) : run_mass<128, false>(p, pl, pool, s);
  return f8 ? run_mass<64, true>(p, pl, pool, s) : run_mass<64, false>(p, pl, pool, s);
}
