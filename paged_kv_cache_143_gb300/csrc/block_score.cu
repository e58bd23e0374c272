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

#include <algorithm>

#include "batch_rows.cuh"
#include "mbar_poll.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------ bounds
//
// A warp takes a kv head of a block, or a few one after the other: its lanes read the key
// rows in 16-byte pieces (a row in D * size / 16 lanes), eight loads in flight, and keep
// the least and greatest of their dims in packed 16-bit arithmetic (exact: E4M3 codes
// widen to f16). The lanes that hold the same dims join by halves: at each step a lane
// hands the half of its dims to its partner that the partner keeps, so that in the end
// every lane has, and writes, dims of its own (all dims to all lanes took two and a half
// times the shuffles, and half of the time for blocks of 16 E4M3 keys). HBM traffic is
// the keys once.
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

// Of 2 KEEP pairs the lane keeps KEEP, joined with the partner M lanes away; then on to M / 2,
// down to LAST.
template <bool FP8, int M, int KEEP, int LAST, class V, int N>
__device__ __forceinline__ void join_halves(V (&lo)[N], V (&hi)[N], int& pair, int lane) {
  using P = Pack<FP8>;
  const bool upper = lane & M;
  pair += upper ? KEEP : 0;
#pragma unroll
  for (int p = 0; p < KEEP; ++p) {
    auto share = [&](V& near, const V& far, auto join) {  // (by value: a choice of lvalues goes to memory)
      const uint32_t x = *reinterpret_cast<const uint32_t*>(&near), y = *reinterpret_cast<const uint32_t*>(&far);
      const uint32_t got = __shfl_xor_sync(kFull, upper ? x : y, M), own = upper ? y : x;
      near = join(*reinterpret_cast<const V*>(&own), *reinterpret_cast<const V*>(&got));
    };
    share(lo[p], lo[p + KEEP], [](V a, V b) { return P::least(a, b); });
    share(hi[p], hi[p + KEEP], [](V a, V b) { return P::most(a, b); });
  }
  if constexpr (M > LAST) join_halves<FP8, M / 2, KEEP / 2, LAST>(lo, hi, pair, lane);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kBoundWarps * 32)
    block_bounds_kernel(const uint8_t* __restrict__ k_pool, __nv_bfloat16* __restrict__ bounds,
                        const int32_t* __restrict__ qsl, const int32_t* __restrict__ seq_lens,
                        const int32_t* __restrict__ tables, int max_blocks, int R, int T, int Hkv,
                        int B, int num_blocks, int per_warp, int64_t n_items, unsigned* err) {
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
  const int shares = (Hkv + per_warp - 1) / per_warp;
  const int64_t slot = item / shares;
  const int head0 = (int)(item - slot * shares) * per_warp, head1 = min(head0 + per_warp, Hkv);
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
  // infinite keys become the largest finite bounds, so that a query's zero still makes zero of them
  const __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0x7F7F), __ushort_as_bfloat16(0x7F7F));
  // (a lane without a row of its own takes the first, which changes nothing)
  const int mine = lane / kRowLanes < rows ? lane / kRowLanes : 0;
  const uint8_t* src = k_pool + (((int64_t)id * Hkv + head0) * B + mine) * kRowBytes + (lane % kRowLanes) * 16;
  __nv_bfloat16* out = bounds + ((int64_t)id * Hkv + head0) * 2 * D;
  for (int h = head0; h < head1; ++h, src += B * kRowBytes, out += 2 * D) {
    V lo[kPairs], hi[kPairs];
    for (int row0 = 0; row0 + mine < rows; row0 += kRows * kDeep) {
      uint4 x[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (row0 + mine + u * kRows < rows)
          x[u] = *reinterpret_cast<const uint4*>(src + (row0 + u * kRows) * kRowBytes);
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (row0 + mine + u * kRows >= rows) break;
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
          V v;
          if constexpr (FP8)
            v = e4m3x2(w[p >> 1] >> (16 * (p & 1)));
          else
            v = *reinterpret_cast<const V*>(&w[p]);
          const bool first = row0 == 0 && u == 0;
          lo[p] = first ? v : P::least(lo[p], v);
          hi[p] = first ? v : P::most(hi[p], v);
        }
      }
    }
    __syncwarp();
    int pair = 0;  // the first of the pairs that the lane keeps
    join_halves<FP8, 16, kPairs / 2, kRowLanes>(lo, hi, pair, lane);
    constexpr int kKept = kPairs * kRowLanes / 32;  // 1 or 2
    uint32_t w[2][kKept];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int p = 0; p < kKept; ++p) {
        const V v = e ? hi[p] : lo[p];
        __nv_bfloat162 o;
        if constexpr (FP8) {
          const float2 f = __half22float2(v);
          o = __floats2bfloat162_rn(f.x, f.y);  // exact
        } else {
          o = __hmax2_nan(__hmin2_nan(v, top), __hneg2(top));
        }
        w[e][p] = *reinterpret_cast<uint32_t*>(&o);
      }
    uint32_t* dst = reinterpret_cast<uint32_t*>(out) + (lane % kRowLanes) * kPairs + pair;
    if constexpr (kKept == 2) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0][0], w[0][1]);
      *reinterpret_cast<uint2*>(dst + D / 2) = make_uint2(w[1][0], w[1][1]);
    } else {
      dst[0] = w[0][0];
      dst[D / 2] = w[1][0];
    }
  }
}

// ------------------------------------------------------------------ scores

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// (a block id outside the pool: bounds of zeros)
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16u : 0u)
               : "memory");
}

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
  float k_scale;
  unsigned* err;
};

// A unit of work is UNIT blocks of a row tile (p.tile tokens of a request) of a kv head.
// A request's are numbered by kv head, row tile and blocks, of which each row tile has as
// many as the last; every worker has an equal run of the batch's (batch_run), whatever the
// lengths. (A CTA for each row tile and 512 blocks: 64 decodes of up to 16k tokens 35 us
// instead of 31, 32 of 9k to 65k 59 instead of 55.)
struct ScoreReq {
  int q0, q_len, seq;
  int tiles, run;  // row tiles; units of one
};
template <int UNIT>
__device__ __forceinline__ ScoreReq score_request(const ScoreParams& p, int r, bool& bad) {
  ScoreReq s;
  s.q0 = __ldg(p.qsl + r);
  const int end = __ldg(p.qsl + r + 1);
  s.seq = __ldg(p.seq_lens + r);
  s.q_len = end - s.q0;
  const bool fine = s.q0 >= 0 && end <= p.T && s.q0 <= end &&
                    (s.q_len == 0 || (s.seq >= s.q_len && s.seq <= (int64_t)p.max_blocks * p.B));
  bad |= !fine;
  if (!fine) s.q_len = 0;
  s.tiles = (s.q_len + p.tile - 1) / p.tile;
  s.run = s.q_len > 0 ? ((s.seq - 1) / p.B + UNIT) / UNIT : 0;
  return s;
}
__device__ __forceinline__ int64_t score_units(const ScoreParams& p, const ScoreReq& s) {
  return (int64_t)p.Hkv * s.tiles * s.run;
}

// The part of a worker's run that one row tile of a kv head has.
struct ScoreTile {
  int r, kvh, t0, nt;   // request, kv head, first row of q, tokens
  int pos0;             // position of the first token
  int first, n_blocks;  // first block, and where the part's blocks end
};
template <int UNIT>
struct ScoreRun {
  ScoreReq req;
  int64_t left;               // units
  int r, kvh, tile, blocks;   // request, kv head, row tile and block unit of the next one

  // The whole warp calls it; false if there is nothing to do.
  __device__ __forceinline__ bool start(const ScoreParams& p, int64_t workers, int64_t worker) {
    bool bad = false;
    const BatchRun run = batch_run(p.R, workers, worker, [&](int x) {
      return score_units(p, score_request<UNIT>(p, x, bad));
    });
    if (bad) raise_error(p.err, kErrBounds);
    left = run.end - run.begin;
    if (left <= 0) return false;
    r = run.r;
    req = score_request<UNIT>(p, r, bad);
    const int64_t at = run.begin - run.base, unit = at / req.run;
    blocks = (int)(at - unit * req.run);
    kvh = (int)(unit / req.tiles);
    tile = (int)(unit - (int64_t)kvh * req.tiles);
    return true;
  }
  // The next part, false at the end.
  __device__ __forceinline__ bool next(const ScoreParams& p, ScoreTile& s) {
    while (left > 0) {
      if (kvh == p.Hkv || req.run == 0) {  // (without units: between the run's first and last request)
        kvh = 0;
        if (++r >= p.R) return false;  // (cannot be: a request has the unit)
        bool bad = false;
        req = score_request<UNIT>(p, r, bad);
        if (req.run == 0) continue;
      }
      const int j0 = tile * p.tile, n = (int)min((int64_t)(req.run - blocks), left);
      s.r = r;
      s.kvh = kvh;
      s.t0 = req.q0 + j0;
      s.nt = min(p.tile, req.q_len - j0);
      s.pos0 = req.seq - req.q_len + j0;
      s.first = blocks * UNIT;
      s.n_blocks = (int)min((int64_t)((s.pos0 + s.nt - 1) / p.B + 1), (int64_t)s.first + (int64_t)n * UNIT);
      left -= n;
      blocks = 0;
      if (++tile == req.tiles) {
        tile = 0;
        ++kvh;
      }
      if (s.first < s.n_blocks) return true;
    }
    return false;
  }
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
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Of N values, N 1, 2, 4 or 8.
template <int N>
__device__ __forceinline__ float max_nan(const uint32_t* v) {
  float x = __uint_as_float(v[0]);
  if constexpr (N == 2) x = max_nan(x, __uint_as_float(v[1]));
#pragma unroll
  for (int i = 1; i + 1 < N; i += 2) x = max_nan(x, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
  if constexpr (N > 2) x = max_nan(x, __uint_as_float(v[N - 1]));
  return x;
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
__device__ __forceinline__ uint4 positive(uint4 v) {
  return make_uint4(positive(v.x), positive(v.y), positive(v.z), positive(v.w));
}
__device__ __forceinline__ uint4 negative(uint4 v) {
  return make_uint4(negative(v.x), negative(v.y), negative(v.z), negative(v.w));
}

// Decodes (a row tile of at most 8 NH columns): the bounds are what costs, 4 D bytes
// a (block, kv head) read once. The workers are warps, none of which waits for another:
// a warp takes 16 blocks as the rows of m16n8k16 MMAs and the (token, head) pairs as
// columns; q+ and q- stay in registers. The bounds of a block come with one cp.async of
// the warp (16 bytes a lane) into its ring of two 16-block stages (records 64 bytes apart
// in banks, so that the 16-byte fragment loads of a quarter-warp do not collide). Three
// CTAs of four warps run on an SM (two with three stages: 69 us where three took 59).
// The maximum over the heads is taken in registers. 32 decodes of 9k to 65k tokens (8 kv
// heads, blocks of 16): 55 us, 5.7 TB/s, 0.84 of the copy rate; 2 to 3 us are the
// workers' start.
constexpr int kScoreWarps = 4;
constexpr int kScoreStages = 2;

template <int D>
struct ScoreRing {
  static constexpr int kRecord = 4 * D;          // least and greatest key
  static constexpr int kPitch = kRecord + 64;
  static constexpr int kStage = 16 * kPitch;
  static constexpr int kWarp = kScoreStages * kStage;
  static constexpr size_t kAlloc = kScoreWarps * kWarp;
};

template <int D, int NH>
__global__ void __launch_bounds__(kScoreWarps * 32, 3) block_score_kernel(ScoreParams p) {
  using Rg = ScoreRing<D>;
  constexpr int KJ = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * Rg::kWarp;
  ScoreRun<16> work;
  if (!work.start(p, (int64_t)gridDim.x * kScoreWarps, (int64_t)blockIdx.x * kScoreWarps + warp)) return;
  for (ScoreTile s; work.next(p, s);) {
    const int kvh = s.kvh, first = s.first, end = s.n_blocks;
    const int32_t* table = p.tables + (int64_t)s.r * p.max_blocks;
    const int mine = (end - first + 15) / 16;
    auto block_of = [&](int i) { return first + 16 * i + (lane & 15); };
    auto fetch = [&](int i) { return i < mine && lane < 16 && block_of(i) < end ? __ldg(table + block_of(i)) : 0; };
    constexpr int kAtOnce = 512 / Rg::kRecord;  // records that the warp's lanes bring with one load
    auto issue = [&](int i, int id) {  // (a group of copies for each tile, be there one or not)
      if (i < mine) {
        bool on = lane < 16 && block_of(i) < end;
        if (on && (id < 0 || id >= p.num_blocks)) {
          raise_error(p.err, kErrBounds);
          on = false;
        }
        const int use = on ? id : -1, piece = lane % (32 / kAtOnce);
        uint8_t* dst = ring + (i % kScoreStages) * Rg::kStage + piece * 16;
#pragma unroll
        for (int b = 0; b < 16; b += kAtOnce) {
          const int rec = b + lane / (32 / kAtOnce);
          const int from = __shfl_sync(kFull, use, rec);
          cp_async16_or_zero(dst + rec * Rg::kPitch,
                             p.bounds + ((int64_t)max(from, 0) * p.Hkv + kvh) * 2 * D + piece * 8, from >= 0);
        }
      }
      cp_async_commit();
    };
    for (int i = 0; i < kScoreStages; ++i) issue(i, fetch(i));
    int next_id = fetch(kScoreStages);
    uint4 qp[NH][KJ], qn[NH][KJ];  // lane (grp, tig): dims 32 j + 8 tig .. + 7 of column 8 h + grp
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int col = 8 * h + grp;
      const int t = min(col / p.gp, s.nt - 1), head = min(col % p.gp, p.g - 1);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((int64_t)(s.t0 + t) * p.Hq + kvh * p.g + head) * D + 8 * tig);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const uint4 v = __ldg(src + 4 * j);
        qp[h][j] = positive(v);
        qn[h][j] = negative(v);
      }
    }
    for (int i = 0; i < mine; ++i) {
      const int st = i % kScoreStages;
      cp_async_wait<kScoreStages - 1>();
      __syncwarp();
      float acc[NH][2][4] = {};
      const uint8_t* rec = ring + st * Rg::kStage + grp * Rg::kPitch + 16 * tig;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const uint4 l0 = *reinterpret_cast<const uint4*>(rec + 64 * j);
        const uint4 l1 = *reinterpret_cast<const uint4*>(rec + 8 * Rg::kPitch + 64 * j);
        const uint4 h0 = *reinterpret_cast<const uint4*>(rec + 2 * D + 64 * j);
        const uint4 h1 = *reinterpret_cast<const uint4*>(rec + 8 * Rg::kPitch + 2 * D + 64 * j);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          mma_bf16(acc[h][1], h0.x, h1.x, h0.y, h1.y, qp[h][j].x, qp[h][j].y);
          mma_bf16(acc[h][0], l0.x, l1.x, l0.y, l1.y, qn[h][j].x, qn[h][j].y);
          mma_bf16(acc[h][1], h0.z, h1.z, h0.w, h1.w, qp[h][j].z, qp[h][j].w);
          mma_bf16(acc[h][0], l0.z, l1.z, l0.w, l1.w, qn[h][j].z, qn[h][j].w);
        }
      }
      __syncwarp();
      issue(i + kScoreStages, next_id);
      next_id = fetch(i + kScoreStages + 1);
      const int b0 = first + 16 * i;
      float* out = p.scores + ((int64_t)s.t0 * p.Hkv + kvh) * p.max_blocks + b0 + grp;
      const int64_t token = (int64_t)p.Hkv * p.max_blocks;
      // columns 2 tig, 2 tig + 1 of rows grp (e = 0, 1) and grp + 8 (e = 2, 3)
      if (p.gp == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 2 * tig + (e & 1), blk = b0 + grp + 8 * (e >> 1);
          if (t < s.nt && (int64_t)blk * p.B <= s.pos0 + t)
            out[t * token + 8 * (e >> 1)] = (acc[0][0][e] + acc[0][1][e]) * p.k_scale;
        }
        continue;
      }
      float m[NH][2];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int ri = 0; ri < 2; ++ri) {
          float x = max_nan(acc[h][0][2 * ri] + acc[h][1][2 * ri],
                            acc[h][0][2 * ri + 1] + acc[h][1][2 * ri + 1]);
          if (p.gp >= 4) x = max_nan(x, __shfl_xor_sync(kFull, x, 1));
          if (p.gp >= 8) x = max_nan(x, __shfl_xor_sync(kFull, x, 2));
          m[h][ri] = x;
        }
      const int t = NH == 1 ? 2 * tig / p.gp : 0;             // the token of this lane's columns
      const int writer = NH == 1 ? tig & ~(p.gp / 2 - 1) : 0;  // and the lane that writes for it
#pragma unroll
      for (int ri = 0; ri < 2; ++ri) {
        const int blk = b0 + grp + 8 * ri;
        const float x = NH == 1 ? m[0][ri] : max_nan(m[0][ri], m[NH - 1][ri]);
        if (tig == writer && t < s.nt && (int64_t)blk * p.B <= s.pos0 + t)
          out[t * token + 8 * ri] = x * p.k_scale;
      }
    }
  }
}

// Chunks: a matrix product of full size, [lo hi] (128 blocks) x [q- q+] (224 columns)
// on tcgen05; the workers are CTAs, one on an SM. Seven warps keep q- and q+ of a row
// tile in shared memory as the operand of up to 224 columns and have the next one's in
// registers when its products begin; four bring the bounds of 128 blocks, 64 dims a
// stage, as the operand of 128 rows: 16 bytes a thread by cp.async, straight to their
// swizzled place. Four warps read the two accumulators in turn (a thread owns a block
// and takes the maximum over the heads in registers), so that neighbouring threads
// write neighbouring blocks' scores. What bounds it is shared memory: for a unit of 128
// blocks the products read 114 KB of columns and 64 KB of bounds, which were written
// there before, 1900 cycles of its 128 bytes (the products alone: 1800 at the rate that
// is reached elsewhere); and 2 us a row tile until the next columns are written. 3 chunks
// on up to 33k tokens (8 kv heads, blocks of 32): 31 us, 8 of them the ends of the launch;
// 4 on up to 64k (blocks of 64): 75. Two CTAs an SM of 112 columns: 33 and 86. Eight
// warps for the scores, or for the copies, or fewer fences for the copies: level.
constexpr int kChunkThreads = 512;  // warps 0-3: scores; 4-7: copies; 8: MMAs; 9-15: columns
constexpr int kChunkCopy = 4, kChunkMma = 8, kChunkColumn = 9;
constexpr int kChunkCols = 224;
constexpr int kChunkStages = 7;
constexpr int kChunkBuf = 256;  // tensor memory columns of an accumulator

template <int D>
struct ChunkSmem {
  static constexpr int kStage = 128 * 128;                // 64 dims of 128 blocks
  static constexpr int kSteps = 2 * D / 64;               // of a tile: least keys, then greatest
  static constexpr int kColHalf = kChunkCols * 128;       // 64 dims of the columns
  static constexpr int kOffRing = 2 * (D / 64) * kColHalf;  // q- (with the least keys), q+
  static constexpr int kOffTail = kOffRing + kChunkStages * kStage;
};
struct ChunkTail {
  uint64_t full[kChunkStages], empty[kChunkStages];
  uint64_t q_ready, q_empty, s_full[2], s_empty[2];
  uint32_t tmem;
  int abort;
};
template <int D>
constexpr size_t chunk_alloc() {
  return 1024 + ChunkSmem<D>::kOffTail + sizeof(ChunkTail);
}

// Scores of one block (a thread's TMEM lane) for the tokens of a row tile whose tokens
// take GP columns (a power of two up to 8; 0: a multiple of 8 that is known at run time).
template <int GP>
struct BlockScores {
  float* out;         // the next token's score
  int64_t token;      // to the one after it
  int from, nt, gp;   // first token that sees the block, tokens, columns of one
  bool seen;          // the warp's blocks are seen by all tokens
  float k_scale;
  float run = 0.f;    // (GP 0) of the columns of token t that were gone through
  int in_token = 0, t = 0;

  __device__ __forceinline__ void columns(const uint32_t (&v)[32], int c) {  // c .. c + 31
    if constexpr (GP > 0) {
      const int tok0 = c / GP;
      if (seen && tok0 + 32 / GP <= nt) {
#pragma unroll
        for (int e = 0; e < 32; e += GP) {
          *out = max_nan<GP>(v + e) * k_scale;
          out += token;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += GP) {
          const int tok = tok0 + e / GP;
          if (tok >= from && tok < nt) *out = max_nan<GP>(v + e) * k_scale;
          out += token;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        const float x = max_nan<8>(v + e);
        run = in_token ? max_nan(run, x) : x;
        in_token += 8;
        if (in_token == gp) {
          if (t >= from && t < nt) *out = run * k_scale;
          out += token;
          ++t;
          in_token = 0;
        }
      }
    }
  }
};

template <int GP>
__device__ __forceinline__ void write_scores(const ScoreParams& p, const ScoreTile& s, uint32_t tm,
                                             float* out, int64_t token, int blk, int n_cols) {
  BlockScores<GP> b;
  b.out = out;
  b.token = token;
  b.from = max(0, (int)min((int64_t)blk * p.B - s.pos0, (int64_t)s.nt));
  b.nt = s.nt;
  b.gp = p.gp;
  b.seen = __all_sync(kFull, b.from == 0);
  b.k_scale = p.k_scale;
#pragma unroll 1
  for (int c = 0; c < n_cols; c += 64) {
    uint32_t va[32], vb[32];
    tc::tmem_ld32(tm + c, va);
    tc::tmem_ld32(tm + c + 32, vb);  // (columns past n_cols hold anything and belong to no token)
    tc::tmem_wait_ld();
    b.columns(va, c);
    b.columns(vb, c + 32);
  }
}

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_score_kernel(ScoreParams p) {
  using S = ChunkSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* cols = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* ring = cols + S::kOffRing;
  ChunkTail* t = reinterpret_cast<ChunkTail*>(cols + S::kOffTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ScoreRun<128> work;
  if (!work.start(p, gridDim.x, blockIdx.x)) return;  // (the same for all warps)
  if (tid == 0) {
    for (int i = 0; i < kChunkStages; ++i) {
      mbar_init(&t->full[i], 128);
      mbar_init(&t->empty[i], 1);
    }
    mbar_init(&t->q_ready, kChunkCols);
    mbar_init(&t->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t->s_full[i], 1);
      mbar_init(&t->s_empty[i], 4);
    }
    t->abort = 0;
    fence_mbar_init();
  }
  if (warp == kChunkMma) {
    tc::tmem_alloc(&t->tmem, 2 * kChunkBuf);
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
  constexpr int kPieces = D / 8;  // 16-byte pieces of a row of dims
  if (warp >= kChunkCopy && warp < kChunkMma) {
    // ------------------------------------------------------------- copies
    // a warp's lanes bring 64 dims of four blocks at once; lane l knows block 32 w + l's id
    const int w = warp - kChunkCopy, piece = lane & 7;
    unsigned step = 0;
    bool ok = true;
    for (ScoreTile s; ok && work.next(p, s);) {
      const int32_t* table = p.tables + (int64_t)s.r * p.max_blocks;
      auto fetch = [&](int blk) { return blk < s.n_blocks ? __ldg(table + blk) : -1; };
      int blk = s.first + w * 32 + lane;
      int id = fetch(blk);
      for (int b0 = s.first; b0 < s.n_blocks && ok; b0 += 128, blk += 128) {
        const int next = fetch(blk + 128);
        const bool good = id >= 0 && id < p.num_blocks;
        if (!good && blk < s.n_blocks) raise_error(p.err, kErrBounds);
        const int use = good ? id : -1;
        const __nv_bfloat16* src[8];
        unsigned there = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int from = __shfl_sync(kFull, use, 4 * b + lane / 8);  // of the warp's 32 blocks
          src[b] = p.bounds + ((int64_t)max(from, 0) * p.Hkv + s.kvh) * 2 * D + piece * 8;
          there |= (unsigned)(from >= 0) << b;
        }
#pragma unroll
        for (int h = 0; h < S::kSteps; ++h, ++step) {
          const unsigned st = step % kChunkStages, round = step / kChunkStages;
          if (round > 0) ok = __all_sync(kFull, wait(&t->empty[st], (round - 1) & 1));
          if (!ok) break;
          uint8_t* dst = ring + st * S::kStage;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const int row = w * 32 + 4 * b + lane / 8;
            cp_async16_or_zero(dst + row * 128 + ((piece ^ (row & 7)) << 4), src[b] + h * 64,
                               (there >> b) & 1);
          }
          // an arrival of this thread once its copies have landed
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           smem_u32(&t->full[st]))
                       : "memory");
        }
        id = next;
      }
    }
    cp_async_wait_all();  // what is in flight lands before the CTA ends
  } else if (warp >= kChunkColumn) {
    // ------------------------------------------------------------ columns
    const int c = tid - kChunkColumn * 32;  // a column a thread, its loads all at once
    bool ok = true;
    unsigned part = 0;
    for (ScoreTile s; ok && work.next(p, s); ++part) {
      const bool mine = c < ((s.nt * p.gp + 15) & ~15);
      const int tok = min(c / p.gp, s.nt - 1), head = min(c % p.gp, p.g - 1);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((int64_t)(s.t0 + tok) * p.Hq + s.kvh * p.g + head) * D);
      uint4 v[kPieces];
#pragma unroll
      for (int x = 0; x < kPieces; ++x)
        if (mine) v[x] = __ldg(src + x);
      if (part > 0) ok = __all_sync(kFull, wait(&t->q_empty, (part - 1) & 1));
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < kPieces; ++x) {
        uint8_t* dst = cols + (x >> 3) * S::kColHalf + c * 128 + (((x & 7) ^ (c & 7)) << 4);
        if (mine) {
          *reinterpret_cast<uint4*>(dst) = negative(v[x]);
          *reinterpret_cast<uint4*>(dst + (D / 64) * S::kColHalf) = positive(v[x]);
        }
      }
      tc::fence_proxy_async_smem();
      mbar_arrive(&t->q_ready);
    }
  } else if (warp == kChunkMma) {
    // --------------------------------------------------------------- MMAs
    bool ok = true;
    unsigned step = 0, part = 0, i = 0;
    auto all_wait = [&](uint64_t* bar, unsigned parity) { return __all_sync(kFull, wait(bar, parity)); };
    for (ScoreTile s; ok && work.next(p, s); ++part) {
      const int n_cols = (s.nt * p.gp + 15) & ~15;
      const uint32_t idesc = tc::idesc_16bit_f32(128, 16, false, false, false) - (2u << 17) +
                             ((uint32_t)(n_cols >> 3) << 17);
      ok = all_wait(&t->q_ready, part & 1);
      for (int b0 = s.first; b0 < s.n_blocks && ok; b0 += 128, ++i) {
        const unsigned buf = i & 1;
        if (i >= 2) ok = all_wait(&t->s_empty[buf], ((i >> 1) - 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < S::kSteps; ++h, ++step) {
          const unsigned st = step % kChunkStages;
          ok = all_wait(&t->full[st], step / kChunkStages & 1);
          if (!ok) break;
          if (tc::elect_one()) {
            tc::fence_proxy_async_smem();  // cp.async writes as threads do, the MMAs read as copies do
            tc::fence_after_sync();
            const uint64_t a = tc::smem_desc_sw128(ring + st * S::kStage, 16, 1024);
            const uint64_t b = tc::smem_desc_sw128(cols + h * S::kColHalf, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_bf16_ss(tmem + buf * kChunkBuf, tc::desc_at(a, k * 32), tc::desc_at(b, k * 32), idesc,
                              h > 0 || k > 0);
            tc::mma_commit(&t->empty[st]);
            if (h == S::kSteps - 1) {
              if (b0 + 128 >= s.n_blocks) tc::mma_commit(&t->q_empty);
              tc::mma_commit(&t->s_full[buf]);
            }
          }
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- scores
    const int64_t token = (int64_t)p.Hkv * p.max_blocks;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    unsigned i = 0;
    bool ok = true;
    for (ScoreTile s; ok && work.next(p, s);) {
      const int n_cols = (s.nt * p.gp + 15) & ~15;
      for (int b0 = s.first; b0 < s.n_blocks; b0 += 128, ++i) {
        const unsigned buf = i & 1;
        const int blk = b0 + tid;
        ok = __all_sync(kFull, wait(&t->s_full[buf], (i >> 1) & 1));
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t tm = tmem + lanes + buf * kChunkBuf;
        float* out = p.scores + ((int64_t)s.t0 * p.Hkv + s.kvh) * p.max_blocks + blk;
        switch (p.gp) {
          case 1: write_scores<1>(p, s, tm, out, token, blk, n_cols); break;
          case 2: write_scores<2>(p, s, tm, out, token, blk, n_cols); break;
          case 4: write_scores<4>(p, s, tm, out, token, blk, n_cols); break;
          case 8: write_scores<8>(p, s, tm, out, token, blk, n_cols); break;
          default: write_scores<0>(p, s, tm, out, token, blk, n_cols);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&t->s_empty[buf]);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kChunkMma) tc::tmem_dealloc(tmem, 2 * kChunkBuf);
}

template <int D, int NH>
bool score_attributes() {
  static OncePerDevice once;
  return once.done([] {
    return cudaFuncSetAttribute(block_score_kernel<D, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)ScoreRing<D>::kAlloc) == cudaSuccess;
  });
}
template <int D>
bool chunk_attributes() {
  static OncePerDevice once;
  return once.done([] {
    return cudaFuncSetAttribute(chunk_score_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)chunk_alloc<D>()) == cudaSuccess;
  });
}

template <int D>
pa_status launch_scores(ScoreParams& p, cudaStream_t stream) {
  // At most one token a request on average and 16 columns a token: the streaming form, else
  // the chunks' (which takes any batch: a single token costs it one small MMA more).
  const bool decodes = p.T <= p.R && p.gp <= 16;
  const int cols = decodes ? (p.gp <= 8 ? 8 : 16) : kChunkCols;
  p.tile = cols / p.gp;
  // As many CTAs as run at once, or as there can be units (per) for.
  const int64_t slots = p.T / p.tile + (int64_t)p.R;
  const int per = decodes ? kScoreWarps * 16 : 128;
  const int64_t chunks = ((int64_t)p.max_blocks + per - 1) / per;
  const int64_t at_once = (decodes ? 3 : 1) * (int64_t)num_sms();
  const unsigned grid =
      (unsigned)(slots >= at_once || chunks >= at_once ? at_once : std::min(at_once, slots * chunks * p.Hkv));
  if (!decodes) {
    if (!chunk_attributes<D>()) return PA_ERR_CUDA;
    chunk_score_kernel<D><<<grid, kChunkThreads, chunk_alloc<D>(), stream>>>(p);
  } else if (p.gp <= 8) {
    if (!score_attributes<D, 1>()) return PA_ERR_CUDA;
    block_score_kernel<D, 1><<<grid, kScoreWarps * 32, ScoreRing<D>::kAlloc, stream>>>(p);
  } else {
    if (!score_attributes<D, 2>()) return PA_ERR_CUDA;
    block_score_kernel<D, 2><<<grid, kScoreWarps * 32, ScoreRing<D>::kAlloc, stream>>>(p);
  }
  return launch_status();
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
  // A warp takes heads of up to 128 keys in all, as long as every SM has 32 warps: finding
  // its place costs a warp more than a head of 16 keys. (24 prompts of 15k to 20k tokens,
  // E4M3, blocks of 16: 160 us one by one, 107 by 4, 100 by 8; blocks of 64: 84, 80, 78.)
  const int64_t want = slots * Hkv / (32 * (int64_t)num_sms());
  const int per_warp = (int)(want < 1 ? 1 : want > 128 / B ? 128 / B : want);
  const int64_t items = slots * ((Hkv + per_warp - 1) / per_warp);
  const int64_t ctas = (items + kBoundWarps - 1) / kBoundWarps;
  if (ctas > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  unsigned* err = error_word();
  if (!err) return PA_ERR_CUDA;
  auto launch = [&](auto kernel) {
    kernel<<<(unsigned)ctas, kBoundWarps * 32, 0, as_stream(stream)>>>(
        static_cast<const uint8_t*>(pool->k_pool), static_cast<__nv_bfloat16*>(bounds),
        query_start_loc, seq_lens, block_tables, max_blocks, num_reqs, num_tokens, Hkv, B,
        pool->num_blocks, per_warp, items, err);
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
  if (p.g > 64) return PA_ERR_UNSUPPORTED;
  p.k_scale = pool->dtype == PA_KV_FP8_E4M3 ? pool->k_scale : 1.f;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  return pool->head_dim == 128 ? launch_scores<128>(p, as_stream(stream))
                               : launch_scores<64>(p, as_stream(stream));
}
