// sparse_attn.cu — pa_sparse_forward: attention of every query token over the
// cache blocks that its (token, kv head) list names.
//
// Per (token, kv head) the work is a decode of the heads that share the kv head
// over the keys of at most k blocks, so the kernel is a stream of 16-key cells
// (a cell's keys, and its values, are each one contiguous run of the pool), read
// once and bound by HBM, or by L2 where neighbouring tokens list the same blocks.
//  - A CTA of four warps serves one (token, kv head, up to 16 heads). Each warp
//    takes every fourth listed block and has a ring of cells of its own in shared
//    memory that its first lane fills with tensor copies:
//    no warp waits for another until the end. The list is read 32 entries at a
//    time, one a lane, and turned into the cells that hold visible keys.
//  - S^T = K Q^T and O^T += V^T P^T are warp-level m16n8k16 MMAs with the 16 keys
//    of a cell as rows and the heads as columns (cells.cuh; g heads are far below
//    the smallest tcgen05 tile), the running maximum and sum of the softmax per
//    head in registers, in fp32. The second product takes each weight as the sum of
//    two 16-bit numbers (bf16 alone is off by 2^-9 of each weight, as much as the output's
//    own rounding; with the second, decodes take what they took, 300 tokens of a chunk
//    96 us instead of 90).
//  - The warps join by log-sum-exp in shared memory. Where there are too few
//    (token, kv head) pairs for the GPU, a cluster of 2, 4 or 8 CTAs shares each
//    list and joins through distributed shared memory: no workspace, one launch.
//    48 decodes on 256 blocks of 16 E4M3 keys (8 kv heads of 128): 74 us, 5.4 TB/s, 0.80
//    of the copy rate; 64 decodes on 128 blocks of 16 bf16 keys: 92 us, 5.8 TB/s. What
//    is left is the start and the end of a CTA's list and uneven CTAs at the end.
#include <cooperative_groups.h>

#include "batch_rows.cuh"
#include "cells.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSparseWarps = 4;
constexpr int kSparseThreads = kSparseWarps * 32;

struct SparseParams {
  const __nv_bfloat16* q;   // [T][Hq][D]
  __nv_bfloat16* out;       // [T][Hq][D]
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int32_t* tables;    // [R][max_blocks]
  const int32_t* selected;  // [T][Hkv][k]
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  int max_blocks, R, T, Hq, Hkv, g, parts, k, B, num_blocks;
  int split;                // CTAs (a cluster) per (token, kv head, part)
  float q_scale, v_scale;
  unsigned* err;
};

// One warp's heads (NH groups of eight) against 16-key cells: the softmax's running
// maxima and sums and the unnormalised output in registers. The reference of a row
// moves only when its maximum grows by more than 2^8 (MmaRows::rebase), and may stay
// at -inf: a cell that scores -inf throughout weighs 0.
template <int D, bool FP8, int NH>
struct CellHeads {
  using C = Cells<D, FP8>;
  static constexpr int MT = C::MT;
  QueryCols<D, FP8, NH> q;
  float o[NH][MT][4];  // [mt]: (dim d, column 2 tig), (d, 2 tig + 1), (d + 1, ..), d = value_dim(mt, grp)
  float m[NH][2], l[NH][2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) o[h][mt][0] = o[h][mt][1] = o[h][mt][2] = o[h][mt][3] = 0.f;
      m[h][0] = m[h][1] = -INFINITY;
      l[h][0] = l[h][1] = 0.f;
    }
  }

  // 2^x, x a score less its reference (up to 8); for f16 parts, exact to 2^-25 at the best,
  // times 2^7, which makes that 2^-32 of the reference's weight.
  static __device__ __forceinline__ float weight(float x) { return ex2_ftz(FP8 ? x + 7.f : x); }

  // Two weights as sums of two 16-bit numbers, hi + lo. f16 (E4M3 pools): both rounded, off by
  // 2^-23. bf16: hi is cut off below the weight, so that lo is positive like hi and an
  // infinite value keeps its sign; off by (2^-7 + 2^-10) 2^-9, just above 2^-16.
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    if constexpr (FP8) {
      const __half2 a = __floats2half2_rn(x, y);
      const float2 f = __half22float2(a);
      const __half2 b = __floats2half2_rn(x - f.x, y - f.y);
      hi = *reinterpret_cast<const uint32_t*>(&a);
      lo = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      constexpr float kBelow = 1.f - 0x1p-10f;
      const uint32_t a = __float_as_uint(x * kBelow) & 0xffff0000u;
      const uint32_t b = __float_as_uint(y * kBelow) & 0xffff0000u;
      const __nv_bfloat162 rest = __floats2bfloat162_rn(x - __uint_as_float(a), y - __uint_as_float(b));
      hi = (a >> 16) | b;
      lo = *reinterpret_cast<const uint32_t*>(&rest);
    }
  }

  // The cell's keys Ks and values Vs, of which the first n are visible (1..16).
  __device__ __forceinline__ void cell(const uint8_t* Ks, const uint8_t* Vs, int n, int grp,
                                       int tig) {
    float s[NH][4];
    q.scores(Ks, s, grp, tig);
    const bool whole = n >= 16;
    uint32_t pb[NH][2], pl[NH][2];  // the weights, and what their rounding left
    bool rescale = false;
    float alpha[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& x0 = s[h][e];
        float& x1 = s[h][2 + e];
        x0 = whole || grp < n ? x0 * q.sc[h][e] : -INFINITY;
        x1 = whole || grp + 8 < n ? x1 * q.sc[h][e] : -INFINITY;
        float mx = fmaxf(x0, x1);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float ref = MmaRows<D, FP8>::rebase(m[h][e], mx, alpha[h][e]);
        const float base = ref == -INFINITY ? 0.f : ref;  // (-inf minus -inf would be NaN)
        x0 = weight(x0 - base);
        x1 = weight(x1 - base);
        l[h][e] = l[h][e] * alpha[h][e] + (x0 + x1);
        m[h][e] = ref;
        rescale |= alpha[h][e] != 1.f;
      }
      split(s[h][0], s[h][1], pb[h][0], pl[h][0]);
      split(s[h][2], s[h][3], pb[h][1], pl[h][1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        MmaKeys<D, FP8>::movtrans(pb[h][i]);
        MmaKeys<D, FP8>::movtrans(pl[h][i]);
      }
    }
    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          o[h][mt][0] *= alpha[h][0];
          o[h][mt][1] *= alpha[h][1];
          o[h][mt][2] *= alpha[h][0];
          o[h][mt][3] *= alpha[h][1];
        }
    }
    uint32_t vw[4][C::kWords];  // rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kr = 2 * tig + (i & 1) + 8 * (i >> 1);
      C::value_words(Vs, kr, grp, vw[i]);
      if (!whole && kr >= n)  // a hidden cell may hold NaN, which a weight of 0 must not meet
#pragma unroll
        for (int w = 0; w < C::kWords; ++w) vw[i][w] = 0u;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t a0, a1, a2, a3;
      asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(a0) : "r"(vw[0][mt]), "r"(vw[1][mt]));
      asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(a1) : "r"(vw[0][mt]), "r"(vw[1][mt]));
      asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(a2) : "r"(vw[2][mt]), "r"(vw[3][mt]));
      asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(a3) : "r"(vw[2][mt]), "r"(vw[3][mt]));
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        MmaRows<D, FP8>::mma(o[h][mt], a0, a1, a2, a3, pb[h][0], pb[h][1]);
        MmaRows<D, FP8>::mma(o[h][mt], a0, a1, a2, a3, pl[h][0], pl[h][1]);
      }
    }
  }

  // This warp's heads into its part of the join: o [8 NH][D], then m and l.
  __device__ __forceinline__ void store(float* comb, int grp, int tig) {
    float* cm = comb + 8 * NH * D;
    float* cl = cm + 8 * NH;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[h][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * h + 2 * tig + e;
        if (grp == 0) {
          cm[row] = m[h][e];
          cl[row] = sum;
        }
#pragma unroll
        for (int w = 0; w < MT; w += 2)
          *reinterpret_cast<float4*>(comb + row * D + C::value_dim(w, grp)) =
              make_float4(o[h][w][e], o[h][w][2 + e], o[h][w + 1][e], o[h][w + 1][2 + e]);
      }
  }
};

template <int D, bool FP8>
struct SparseGeo {
  static constexpr int kCell = 2 * Cells<D, FP8>::kBytes;  // keys, then values
  // cells of a warp's ring: 16 KB a warp, 64 KB a CTA, three CTAs on an SM
  static constexpr int kWarpBytes = 16384;  // ring, later the warp's part of the join
  static constexpr int kStages = kWarpBytes / kCell > 8 ? 8 : kWarpBytes / kCell;
  static_assert(kStages >= 2, "ring");
  static_assert((16 * D + 32) * 4 <= kWarpBytes, "join");
};

struct SparseTail {
  uint64_t full[kSparseWarps][8];
  uint2 cells[kSparseWarps][128];  // (block id, key offset in the block | visible keys << 8)
  float stat_m[16], stat_l[16];    // the CTA's heads, for the other CTAs of its cluster
  int seen[kSparseWarps];          // whether a warp met a visible key
  int any;
};

template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kSparseThreads, NH == 1 ? 3 : 2)
    sparse_attn_kernel(const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, SparseParams p) {
  using CH = CellHeads<D, FP8, NH>;
  using SG = SparseGeo<D, FP8>;
  using C = Cells<D, FP8>;
  constexpr int kStages = SG::kStages;
  constexpr int kRows = 8 * NH;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  SparseTail* tail = reinterpret_cast<SparseTail*>(ring + kSparseWarps * SG::kWarpBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tig = lane & 3;
  const int64_t unit = blockIdx.x / p.split;
  const int rank = (int)(blockIdx.x - unit * p.split);
  const int part = (int)(unit % p.parts);
  const int kvh = (int)(unit / p.parts % p.Hkv);
  const int t = (int)(unit / p.parts / p.Hkv);
  const int hq0 = kvh * p.g + part * kRows;
  const int heads = min(kRows, p.g - part * kRows);
  const int32_t* list = p.selected + ((int64_t)t * p.Hkv + kvh) * p.k;
  const int lanes_of = kSparseWarps * p.split;  // warps that share the list
  const int first = rank * kSparseWarps + warp;
  // the list's entries of a round, one a lane; the first ones come with the row's lengths
  auto entry = [&](int64_t base) {
    const int64_t e = base + (int64_t)lane * lanes_of + first;
    return e < p.k ? __ldg(list + e) : -1;
  };
  int b = entry(0);
  // every CTA of a cluster takes the same way out here
  ReqSpan sp;
  const int r = span_of_row(p.qsl, p.seq_lens, p.R, t, sp);
  if (r < 0) return;  // a row behind the last sequence
  if (!span_fits(sp, p.T, (int64_t)p.max_blocks * p.B, p.err)) return;
  const int sees = sp.seq - sp.q_len + (t - sp.q0) + 1;  // keys that the token may see

  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&tail->full[warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  CH st;
  st.reset();

  uint8_t* my_ring = ring + warp * SG::kWarpBytes;
  uint64_t* full = tail->full[warp];
  uint2* cells = tail->cells[warp];
  const int32_t* table = p.tables + (int64_t)r * p.max_blocks;
  uint32_t pos = 0;  // cells gone through: stage pos mod kStages, phase pos / kStages
  bool ok = true;
  int seen = 0;
  auto issue = [&](uint32_t at, uint2 c) {  // one lane
    const uint32_t stage = at % kStages;
    uint8_t* dst = my_ring + stage * SG::kCell;
    mbar_arrive_expect_tx(&full[stage], SG::kCell);
    const int line = kvh * p.B + (int)(c.y & 0xffu);
    C::load(dst, &tmap_k, line, (int)c.x, &full[stage]);
    C::load(dst + C::kBytes, &tmap_v, line, (int)c.x, &full[stage]);
  };
  for (int64_t base = 0; base < p.k && ok; base += 32 * lanes_of) {
    int n_cells = 0, id = 0, keys = 0;
    if (b < -1 || b >= p.max_blocks) {
      raise_error(p.err, kErrBounds);
    } else if (b >= 0 && (int64_t)b * p.B < sees) {
      id = __ldg(table + b);
      keys = min(p.B, sees - b * p.B);
      if (id < 0 || id >= p.num_blocks)
        raise_error(p.err, kErrBounds);
      else
        n_cells = (keys + kChunk - 1) / kChunk;
    }
    b = entry(base + 32 * lanes_of);
    int end = n_cells;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const int total = __shfl_sync(0xffffffffu, end, 31);
    __syncwarp();  // the cells of the round before have been read
    for (int c = 0; c < n_cells; ++c)
      cells[end - n_cells + c] =
          make_uint2((uint32_t)id, (uint32_t)(c * kChunk) |
                                       ((uint32_t)min(kChunk, keys - c * kChunk) << 8));
    __syncwarp();
    seen |= total > 0;
    if (lane == 0)
      for (int c = 0; c < min(total, kStages); ++c) issue(pos + c, cells[c]);
    if (base == 0)  // (while the first cells are on their way)
      st.q.load([&](int c) { return c < heads ? p.q + ((int64_t)t * p.Hq + hq0 + c) * D : nullptr; },
                p.q_scale, grp, tig);
    for (int c = 0; c < total; ++c) {
      const uint32_t at = pos + c, stage = at % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], (at / kStages) & 1, p.err))) {
        ok = false;  // flagged; the copies still in flight land before the ring is used again
        if (lane == 0)
          for (int x = c + 1; x < min(total, c + kStages); ++x)
            mbar_wait(&full[(pos + x) % kStages], ((pos + x) / kStages) & 1, p.err);
        __syncwarp();
        break;
      }
      const uint8_t* Ks = my_ring + stage * SG::kCell;
      st.cell(Ks, Ks + C::kBytes, (int)(cells[c].y >> 8), grp, tig);
      __syncwarp();
      if (lane == 0 && c + kStages < total) issue(at + kStages, cells[c + kStages]);
    }
    pos += total;
  }
  // the join: each warp's heads in its own (now idle) part of the ring
  float* comb = reinterpret_cast<float*>(my_ring);
  if (lane == 0) tail->seen[warp] = seen;
  __syncwarp();
  st.store(comb, grp, tig);
  __syncthreads();
  constexpr int kCombFloats = SG::kWarpBytes / 4;
  float* all = reinterpret_cast<float*>(ring);  // warp w's part at w * kCombFloats
  const int any = tail->seen[0] | tail->seen[1] | tail->seen[2] | tail->seen[3];
  auto ref_of = [](float m) { return m == -INFINITY ? 0.f : m; };
  if (p.split == 1) {
    for (int x = tid; x < heads * (D / 2); x += kSparseThreads) {
      const int row = x / (D / 2), d = 2 * (x % (D / 2));
      float mw[kSparseWarps], M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSparseWarps; ++w) {
        mw[w] = all[w * kCombFloats + kRows * D + row];
        M = fmaxf(M, mw[w]);
      }
      float L = 0.f, a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < kSparseWarps; ++w) {
        const float f = ex2_ftz(mw[w] - ref_of(M));
        const float2 v = *reinterpret_cast<const float2*>(all + w * kCombFloats + row * D + d);
        L += f * all[w * kCombFloats + kRows * D + kRows + row];
        a += f * v.x;
        b += f * v.y;
      }
      __nv_bfloat162 y = __floats2bfloat162_rn(a / L * p.v_scale, b / L * p.v_scale);
      if (!any) y = __floats2bfloat162_rn(0.f, 0.f);  // no visible key
      *reinterpret_cast<__nv_bfloat162*>(p.out + ((int64_t)t * p.Hq + hq0 + row) * D + d) = y;
    }
    return;
  }
  // the CTA's warps into warp 0's part, its statistics beside it
  for (int x = tid; x < heads * (D / 2); x += kSparseThreads) {
    const int row = x / (D / 2), d = 2 * (x % (D / 2));
    float mw[kSparseWarps], M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
      mw[w] = all[w * kCombFloats + kRows * D + row];
      M = fmaxf(M, mw[w]);
    }
    float L = 0.f, a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
      const float f = ex2_ftz(mw[w] - ref_of(M));
      const float2 v = *reinterpret_cast<const float2*>(all + w * kCombFloats + row * D + d);
      L += f * all[w * kCombFloats + kRows * D + kRows + row];
      a += f * v.x;
      b += f * v.y;
    }
    *reinterpret_cast<float2*>(all + row * D + d) = make_float2(a, b);  // (read by this thread alone)
    if (d == 0) {
      tail->stat_m[row] = M;
      tail->stat_l[row] = L;
    }
  }
  if (tid == 0) tail->any = any;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  int any_at_all = 0;
  for (int c = 0; c < p.split; ++c) any_at_all |= *cluster.map_shared_rank(&tail->any, c);
  for (int x = rank * kSparseThreads + tid; x < heads * (D / 2); x += kSparseThreads * p.split) {
    const int row = x / (D / 2), d = 2 * (x % (D / 2));
    float M = -INFINITY;
    for (int c = 0; c < p.split; ++c) M = fmaxf(M, *cluster.map_shared_rank(&tail->stat_m[row], c));
    float L = 0.f, a = 0.f, b = 0.f;
    for (int c = 0; c < p.split; ++c) {
      const float f = ex2_ftz(*cluster.map_shared_rank(&tail->stat_m[row], c) - ref_of(M));
      const float2 v = *reinterpret_cast<const float2*>(cluster.map_shared_rank(all + row * D + d, c));
      L += f * *cluster.map_shared_rank(&tail->stat_l[row], c);
      a += f * v.x;
      b += f * v.y;
    }
    __nv_bfloat162 y = __floats2bfloat162_rn(a / L * p.v_scale, b / L * p.v_scale);
    if (!any_at_all) y = __floats2bfloat162_rn(0.f, 0.f);
    *reinterpret_cast<__nv_bfloat162*>(p.out + ((int64_t)t * p.Hq + hq0 + row) * D + d) = y;
  }
  cluster.sync();  // no CTA leaves while another reads its part
}

template <int D, bool FP8, int NH>
pa_status launch_sparse(const SparseParams& p, int64_t ctas, cudaStream_t s) {
  constexpr size_t smem =
      1024 + (size_t)kSparseWarps * SparseGeo<D, FP8>::kWarpBytes + sizeof(SparseTail);
  static OncePerDevice once;
  if (!once.done([] {
        return cudaFuncSetAttribute(sparse_attn_kernel<D, FP8, NH>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem) == cudaSuccess;
      }))
    return PA_ERR_CUDA;
  CUtensorMap tk, tv;
  if (!cell_map<D, FP8>(&tk, p.k_pool, p.num_blocks, p.Hkv * p.B) ||
      !cell_map<D, FP8>(&tv, p.v_pool, p.num_blocks, p.Hkv * p.B))
    return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kSparseThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, sparse_attn_kernel<D, FP8, NH>, tk, tv, p) != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_sparse_forward(const void* q, void* out, const int32_t* query_start_loc,
                                       const int32_t* seq_lens, const int32_t* block_tables,
                                       int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                                       int32_t num_q_heads, const int32_t* selected, int32_t k,
                                       const pa_kv_pool* pool, float scale, pa_stream_t stream) {
  using namespace pa;
  pa_status st = check_pool(pool);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks < 0 || k < 1 || num_q_heads <= 0 ||
      num_q_heads % pool->num_kv_heads != 0)
    return PA_ERR_INVALID;
  if (num_reqs == 0 || num_tokens == 0) return PA_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) || !query_start_loc || !seq_lens ||
      !block_tables || !selected || max_blocks == 0 || pool->num_blocks < 1)
    return PA_ERR_INVALID;
  SparseParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.tables = block_tables;
  p.selected = selected;
  p.k_pool = static_cast<const uint8_t*>(pool->k_pool);
  p.v_pool = static_cast<const uint8_t*>(pool->v_pool);
  p.max_blocks = max_blocks;
  p.R = num_reqs;
  p.T = num_tokens;
  p.Hq = num_q_heads;
  p.Hkv = pool->num_kv_heads;
  p.g = num_q_heads / p.Hkv;
  p.k = k;
  p.B = pool->block_size;
  p.num_blocks = pool->num_blocks;
  const bool fp8 = pool->dtype == PA_KV_FP8_E4M3, wide = p.g > 8;
  p.parts = (p.g + 15) / 16;
  p.q_scale = scale * 1.44269504088896340736f * (fp8 ? pool->k_scale : 1.f);
  p.v_scale = fp8 ? pool->v_scale : 1.f;
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  // A cluster shares a list where that many CTAs still run at once (three on an SM, two
  // for more than 8 heads), each warp keeping two blocks; and two CTAs share one of 128
  // blocks or more where the lists are up to a third more than run at once, so that the
  // second round is half as long. Lists of 128 blocks of 16 keys (bf16, 8 kv heads), us by
  // 1, 2, 4 and 8 CTAs: 8 decodes 27, 22, 20, 27; 16: 31, 31, 37, 39; 40: 57, 61, 65, 78. Up
  // to a third more than at once, by 1 and 2: 64 decodes on 128 blocks 96 and 94, on 256 184
  // and 166, E4M3 117 and 111, on 32 blocks 33 and 39; 46 of 16 heads a kv head on 256 160
  // and 143. Beyond: 80 decodes on 128 104 and 111, 100 E4M3 76 and 86, 300 tokens of a chunk
  // (64 blocks) 96 and 133.
  const int64_t units = (int64_t)num_tokens * p.Hkv * p.parts;
  const int64_t at_once = (int64_t)(wide ? 2 : 3) * num_sms();
  p.split = 1;
  while (p.split < 8 && k >= 4 * kSparseWarps * p.split && units * 2 * p.split <= at_once) p.split *= 2;
  if (k >= 128 && units > at_once && 3 * units <= 4 * at_once) p.split = 2;
  if (units * p.split > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  const int64_t ctas = units * p.split;
  cudaStream_t s = as_stream(stream);
  if (pool->head_dim == 128)
    return fp8 ? (wide ? launch_sparse<128, true, 2>(p, ctas, s) : launch_sparse<128, true, 1>(p, ctas, s))
               : (wide ? launch_sparse<128, false, 2>(p, ctas, s) : launch_sparse<128, false, 1>(p, ctas, s));
  return fp8 ? (wide ? launch_sparse<64, true, 2>(p, ctas, s) : launch_sparse<64, true, 1>(p, ctas, s))
             : (wide ? launch_sparse<64, false, 2>(p, ctas, s) : launch_sparse<64, false, 1>(p, ctas, s));
}
