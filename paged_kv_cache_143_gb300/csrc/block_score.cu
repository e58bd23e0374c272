// block_score.cu — pa_update_block_bounds (the least and greatest key of each
// block) and pa_score_blocks (from them, the most that any key of a block can
// score with a query).
//
// For a block whose keys lie in the box [lo, hi],
//   max over the box of q . k = sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// so with q+ = max(q, 0) and q- = min(q, 0) the scores of many blocks are the
// product of [hi lo] (blocks x 2D) with [q+ q-] (2D x heads): a matrix product
// that reads 4 D bytes of a (block, kv head) where its keys and values take
// 4 D B (bf16).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "batch_rows.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------ bounds
//
// One warp per (block, kv head): its lanes read the block's key rows in
// 16-byte pieces (a row in D * size / 16 lanes), eight loads in flight, keep
// the least and greatest of their dims in packed 16-bit arithmetic (exact:
// E4M3 codes widen to f16) and join by shuffles. HBM traffic is the keys once.
// The blocks that a step touched are found from slots: request r owns the
// slots from qsl[r] / B + 2 r on, which leaves room for the
// (q_len - 1) / B + 2 blocks at most that q_len tokens reach.
constexpr int kBoundWarps = 8;

template <bool FP8>
struct Pack;  // two elements in 32 bits
template <>
struct Pack<false> {
  using T = __nv_bfloat162;
  static __device__ __forceinline__ T least(T a, T b) { return __hmin2_nan(a, b); }
  static __device__ __forceinline__ T most(T a, T b) { return __hmax2_nan(a, b); }
};
template <>
struct Pack<true> {
  using T = __half2;
  static __device__ __forceinline__ T least(T a, T b) { return __hmin2_nan(a, b); }
  static __device__ __forceinline__ T most(T a, T b) { return __hmax2_nan(a, b); }
};

__device__ __forceinline__ __half2 e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(h)
      : "r"(codes));
  return *reinterpret_cast<__half2*>(&h);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundWarps * 32)
    block_bounds_kernel(const uint8_t* __restrict__ k_pool, __nv_bfloat16* __restrict__ bounds,
                        const int32_t* __restrict__ qsl, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ tables, int max_blocks, int R, int T, int Hkv,
                        int B, int num_blocks, int64_t n_items, unsigned* err) {
  using P = Pack<FP8>;
  using V = typename P::T;
  constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  constexpr int kRowLanes = kRowBytes / 16;  // lanes that read one key row
  constexpr int kRows = 32 / kRowLanes;      // key rows that a warp reads at once
  constexpr int kPairs = FP8 ? 8 : 4;        // element pairs of a lane's 16 bytes
  constexpr int kDeep = 8;                   // loads in flight
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  if (item >= n_items) return;
  const int64_t slot = item / Hkv;
  const int kvh = (int)(item - slot * Hkv);
  int r, i, n;  // request, logical block, the request's stored tokens
  if (qsl) {
    r = warp_last_le(R, slot, [&](int x) { return (int64_t)(__ldg(qsl + x) / B) + 2 * (int64_t)x; });
    ReqSpan s;
    if (!request_span(qsl, seq_lens, r, T, (int64_t)max_blocks * B, err, s) || s.q_len == 0) return;
    n = s.seq;
    const int64_t at = slot - ((int64_t)(s.q0 / B) + 2 * (int64_t)r) + (n - s.q_len) / B;
    if (at < 0 || at * B >= n) return;
    i = (int)at;
  } else {
    r = (int)(slot / max_blocks);
    i = (int)(slot - (int64_t)r * max_blocks);
    n = seq_lens[r];
    if (n < 0 || n > (int64_t)max_blocks * B) {
      raise_error(err, kErrBounds);
      return;
    }
    if ((int64_t)i * B >= n) return;
  }
  const int id = tables[(int64_t)r * max_blocks + i];
  if (id < 0 || id >= num_blocks) {
    raise_error(err, kErrBounds);
    return;
  }
  const int rows = min(B, n - i * B);
  const uint8_t* src = k_pool + (((int64_t)id * Hkv + kvh) * B) * kRowBytes +
                       (lane % kRowLanes) * 16;
  V lo[kPairs] = {}, hi[kPairs] = {};
  bool any = false;
  for (int row0 = lane / kRowLanes; row0 < rows; row0 += kRows * kDeep) {
    uint4 x[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (row0 + u * kRows < rows)
        x[u] = *reinterpret_cast<const uint4*>(src + (int64_t)(row0 + u * kRows) * kRowBytes);
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (row0 + u * kRows >= rows) break;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        V v;
        if constexpr (FP8)
          v = e4m3x2(w[p >> 1] >> (16 * (p & 1)));
        else
          v = *reinterpret_cast<const V*>(&w[p]);
        lo[p] = any ? P::least(lo[p], v) : v;
        hi[p] = any ? P::most(hi[p], v) : v;
      }
      any = true;
    }
  }
#pragma unroll
  for (int m = kRowLanes; m < 32; m <<= 1) {
    const bool other = __shfl_xor_sync(kFull, any, m);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      uint32_t a = *reinterpret_cast<uint32_t*>(&lo[p]), b = *reinterpret_cast<uint32_t*>(&hi[p]);
      a = __shfl_xor_sync(kFull, a, m);
      b = __shfl_xor_sync(kFull, b, m);
      const V va = *reinterpret_cast<V*>(&a), vb = *reinterpret_cast<V*>(&b);
      if (other) {
        lo[p] = any ? P::least(lo[p], va) : va;
        hi[p] = any ? P::most(hi[p], vb) : vb;
      }
    }
    any |= other;
  }
  if (lane >= kRowLanes) return;
  // infinite keys become the largest finite bounds, so that a query's zero still makes zero of them
  const __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0x7F7F), __ushort_as_bfloat16(0x7F7F));
  __nv_bfloat16* out = bounds + ((int64_t)id * Hkv + kvh) * 2 * D + lane * 2 * kPairs;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const V v = h ? hi[p] : lo[p];
      __nv_bfloat162 o;
      if constexpr (FP8) {
        const float2 f = __half22float2(v);
        o = __floats2bfloat162_rn(f.x, f.y);  // exact
      } else {
        o = __hmax2_nan(__hmin2_nan(v, top), __hneg2(top));
      }
      w[p] = *reinterpret_cast<uint32_t*>(&o);
    }
#pragma unroll
    for (int p = 0; p < kPairs; p += 4)
      *reinterpret_cast<uint4*>(out + h * D + 2 * p) = make_uint4(w[p], w[p + 1], w[p + 2], w[p + 3]);
  }
}

// ------------------------------------------------------------------ scores
//
// A warp takes 16 blocks as the rows of m16n8k16 MMAs and the (token, head)
// pairs of a row tile as the columns, eight at a time. The blocks' bounds go
// straight from memory to registers as A fragments (lane (grp, tig) holds dims
// 32 j + 8 tig .. + 7 of rows grp and grp + 8, the same dims for both operands,
// so that a fragment is a 16-byte load) and stay there for all columns; q+ and
// q- are cut once by the CTA into B fragments in shared memory. The maximum
// over the heads of a kv head is taken in registers.
constexpr int kScoreWarps = 4;
constexpr int kMaxColTiles = 8;  // n-tiles of a CTA's row tile

struct ScoreParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  float* scores;
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int32_t* tables;
  int max_blocks, R, T, Hq, Hkv, g, B, num_blocks;
  int gp;         // columns that a token takes: g padded to 1, 2, 4 or a multiple of 8
  int tile;       // tokens of a row tile
  int tiles;      // 16-block tiles that a warp goes through
  float k_scale;
  unsigned* err;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(x, 0) and min(x, 0) of two bf16; NaN stays NaN in both
__device__ __forceinline__ uint32_t positive(uint32_t x) {
  const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
  __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), z);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t negative(uint32_t x) {
  const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
  __nv_bfloat162 v = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&x), z);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) block_score_kernel(ScoreParams p) {
  constexpr int KJ = D / 32;
  extern __shared__ uint4 qfrag[];  // [n-tile][j][q+, q-][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, tig = lane & 3;
  const int kvh = blockIdx.x % p.Hkv;
  const int slot = blockIdx.x / p.Hkv;
  const int r = warp_last_le(p.R, slot, [&](int x) { return __ldg(p.qsl + x) / p.tile + x; });
  ReqSpan s;
  if (!request_span(p.qsl, p.seq_lens, r, p.T, (int64_t)p.max_blocks * p.B, p.err, s)) return;
  const int j0 = (slot - (s.q0 / p.tile + r)) * p.tile;
  if (j0 < 0 || j0 >= s.q_len) return;
  const int nt = min(p.tile, s.q_len - j0);             // tokens of this tile
  const int pos0 = s.seq - s.q_len + j0;                // position of its first token
  const int n_blocks = (pos0 + nt - 1) / p.B + 1;       // blocks that its last token sees
  const int first = (int)blockIdx.y * kScoreWarps * p.tiles * 16;
  if (first >= n_blocks) return;
  const int n_col = (nt * p.gp + 7) / 8;                // n-tiles in use
  for (int x = threadIdx.x; x < n_col * KJ * 32; x += kScoreWarps * 32) {
    const int l = x & 31, j = (x >> 5) % KJ, c = x / (32 * KJ);
    const int col = c * 8 + (l >> 2);
    const int t = min(col / p.gp, nt - 1), h = min(col % p.gp, p.g - 1);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(
        p.q + ((int64_t)(s.q0 + j0 + t) * p.Hq + kvh * p.g + h) * D + 32 * j + 8 * (l & 3)));
    uint4* dst = qfrag + ((c * KJ + j) * 2) * 32 + l;
    dst[0] = make_uint4(positive(v.x), positive(v.y), positive(v.z), positive(v.w));
    dst[32] = make_uint4(negative(v.x), negative(v.y), negative(v.z), negative(v.w));
  }
  __syncthreads();
  const int32_t* table = p.tables + (int64_t)r * p.max_blocks;
  for (int it = 0; it < p.tiles; ++it) {
    const int b0 = first + (it * kScoreWarps + warp) * 16;
    if (b0 >= n_blocks) break;
    uint4 a[2][2][KJ];  // [lo, hi][row grp, row grp + 8]
#pragma unroll
    for (int ri = 0; ri < 2; ++ri) {
      const int i = b0 + grp + 8 * ri;
      int id = i < n_blocks ? __ldg(table + i) : -1;
      if (i < n_blocks && (id < 0 || id >= p.num_blocks)) {
        raise_error(p.err, kErrBounds);
        id = -1;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.bounds + (((int64_t)max(id, 0) * p.Hkv + kvh) * 2 + h) * D + 8 * tig);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          a[h][ri][j] = id >= 0 ? __ldg(src + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    float run[2] = {-INFINITY, -INFINITY};  // over the n-tiles of one token (gp > 8)
    for (int c = 0; c < n_col; ++c) {
      float acc[2][4] = {};
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const uint4 qp = qfrag[((c * KJ + j) * 2) * 32 + lane];
        const uint4 qn = qfrag[((c * KJ + j) * 2 + 1) * 32 + lane];
        mma_bf16(acc[1], a[1][0][j].x, a[1][1][j].x, a[1][0][j].y, a[1][1][j].y, qp.x, qp.y);
        mma_bf16(acc[0], a[0][0][j].x, a[0][1][j].x, a[0][0][j].y, a[0][1][j].y, qn.x, qn.y);
        mma_bf16(acc[1], a[1][0][j].z, a[1][1][j].z, a[1][0][j].w, a[1][1][j].w, qp.z, qp.w);
        mma_bf16(acc[0], a[0][0][j].z, a[0][1][j].z, a[0][0][j].w, a[0][1][j].w, qn.z, qn.w);
      }
      // columns 2 tig, 2 tig + 1 of rows grp (e = 0, 1) and grp + 8 (e = 2, 3)
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (acc[0][e] + acc[1][e]) * p.k_scale;
      if (p.gp == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = c * 8 + 2 * tig + (e & 1), i = b0 + grp + 8 * (e >> 1);
          if (t < nt && i * p.B <= pos0 + t)
            p.scores[((int64_t)(s.q0 + j0 + t) * p.Hkv + kvh) * p.max_blocks + i] = v[e];
        }
        continue;
      }
      float m[2] = {max_nan(v[0], v[1]), max_nan(v[2], v[3])};
#pragma unroll
      for (int ri = 0; ri < 2; ++ri) {
        if (p.gp >= 4) m[ri] = max_nan(m[ri], __shfl_xor_sync(kFull, m[ri], 1));
        if (p.gp >= 8) m[ri] = max_nan(m[ri], __shfl_xor_sync(kFull, m[ri], 2));
      }
      int t, writer;  // the token of this lane's columns, and the lane of its group that writes
      if (p.gp > 8) {
        const int part = c % (p.gp / 8);
        run[0] = part ? max_nan(run[0], m[0]) : m[0];
        run[1] = part ? max_nan(run[1], m[1]) : m[1];
        if (part + 1 < p.gp / 8) continue;
        m[0] = run[0];
        m[1] = run[1];
        t = c / (p.gp / 8);
        writer = 0;
      } else {
        t = (c * 8 + 2 * tig) / p.gp;
        writer = tig & ~(p.gp / 2 - 1);
      }
#pragma unroll
      for (int ri = 0; ri < 2; ++ri) {
        const int i = b0 + grp + 8 * ri;
        if (tig == writer && t < nt && (int64_t)i * p.B <= pos0 + t)
          p.scores[((int64_t)(s.q0 + j0 + t) * p.Hkv + kvh) * p.max_blocks + i] = m[ri];
      }
    }
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_update_block_bounds(const pa_kv_pool* pool, void* bounds,
                                            const int32_t* query_start_loc,
                                            const int32_t* seq_lens, const int32_t* block_tables,
                                            int32_t max_blocks, int32_t num_reqs,
                                            int32_t num_tokens, pa_stream_t stream) {
  using namespace pa;
  pa_status st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || max_blocks < 0 || num_tokens < 0) return PA_ERR_INVALID;
  if (num_reqs == 0 || max_blocks == 0 || (query_start_loc && num_tokens == 0)) return PA_OK;
  if (!bounds || !aligned16(bounds) || !seq_lens || !block_tables) return PA_ERR_INVALID;
  const int B = pool->block_size, D = pool->head_dim, Hkv = pool->num_kv_heads;
  const int64_t slots = query_start_loc ? num_tokens / B + 2 * (int64_t)num_reqs
                                        : (int64_t)num_reqs * max_blocks;
  const int64_t items = slots * Hkv, ctas = (items + kBoundWarps - 1) / kBoundWarps;
  if (ctas > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  unsigned* err = error_word();
  if (!err) return PA_ERR_CUDA;
  auto launch = [&](auto kernel) {
    kernel<<<(unsigned)ctas, kBoundWarps * 32, 0, as_stream(stream)>>>(
        static_cast<const uint8_t*>(pool->k_pool), static_cast<__nv_bfloat16*>(bounds),
        query_start_loc, seq_lens, block_tables, max_blocks, num_reqs, num_tokens, Hkv, B,
        pool->num_blocks, items, err);
  };
  const bool fp8 = pool->dtype == PA_KV_FP8_E4M3;
  if (D == 128)
    fp8 ? launch(block_bounds_kernel<128, true>) : launch(block_bounds_kernel<128, false>);
  else
    fp8 ? launch(block_bounds_kernel<64, true>) : launch(block_bounds_kernel<64, false>);
  return launch_status();
}

extern "C" pa_status pa_score_blocks(const void* q, const void* bounds, float* scores,
                                     const int32_t* query_start_loc, const int32_t* seq_lens,
                                     const int32_t* block_tables, int32_t max_blocks,
                                     int32_t num_reqs, int32_t num_tokens, int32_t num_q_heads,
                                     const pa_kv_pool* pool, pa_stream_t stream) {
  using namespace pa;
  pa_status st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || max_blocks < 0 || num_tokens < 0 || num_q_heads <= 0 ||
      num_q_heads % pool->num_kv_heads != 0)
    return PA_ERR_INVALID;
  if (num_reqs == 0 || num_tokens == 0 || max_blocks == 0) return PA_OK;
  if (!q || !aligned16(q) || !bounds || !aligned16(bounds) || !scores ||
      (reinterpret_cast<uintptr_t>(scores) & 3u) || !query_start_loc || !seq_lens || !block_tables)
    return PA_ERR_INVALID;
  ScoreParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.bounds = static_cast<const __nv_bfloat16*>(bounds);
  p.scores = scores;
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.tables = block_tables;
  p.max_blocks = max_blocks;
  p.R = num_reqs;
  p.T = num_tokens;
  p.Hq = num_q_heads;
  p.Hkv = pool->num_kv_heads;
  p.g = num_q_heads / p.Hkv;
  p.B = pool->block_size;
  p.num_blocks = pool->num_blocks;
  p.gp = p.g <= 1 ? 1 : p.g <= 2 ? 2 : p.g <= 4 ? 4 : (p.g + 7) / 8 * 8;
  if (p.gp > 8 * kMaxColTiles) return PA_ERR_UNSUPPORTED;
  p.tile = 8 * kMaxColTiles / p.gp;
  p.tiles = 2;
  p.k_scale = pool->dtype == PA_KV_FP8_E4M3 ? pool->k_scale : 1.f;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  const int64_t slots = num_tokens / p.tile + (int64_t)num_reqs;
  const int per_cta = kScoreWarps * p.tiles * 16;
  const int64_t chunks = ((int64_t)max_blocks + per_cta - 1) / per_cta;
  if (slots * p.Hkv > 0x7fffffff || chunks > 65535) return PA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(slots * p.Hkv), (unsigned)chunks);
  const size_t smem = (size_t)kMaxColTiles * (pool->head_dim / 32) * 2 * 32 * sizeof(uint4);
  if (pool->head_dim == 128)
    block_score_kernel<128><<<grid, kScoreWarps * 32, smem, as_stream(stream)>>>(p);
  else
    block_score_kernel<64><<<grid, kScoreWarps * 32, smem, as_stream(stream)>>>(p);
  return launch_status();
}
