// cells.cuh — 16-key cells of a paged pool and one warp's heads against them, for
// the kernels that stream keys (pa_sparse_forward, pa_attention_mass).
//
// A cell is 16 consecutive keys of one (block, kv head). One TMA copy brings it
// as 16 rows of 128 bytes (two such halves for bf16 at D = 128) with the 128-byte
// swizzle: 16-byte piece c of row r lies at piece c ^ (r & 7). (E4M3 at D = 64:
// plain rows of 64 bytes.)
//
// The products are m16n8k16 MMAs with the 16 keys as rows and 8 query heads as
// columns: S^T = K Q^T, O^T += V^T P^T. Which head dims a lane takes is free as
// long as both operands of a product agree, and is chosen so that every 16-byte
// load of a quarter-warp falls on distinct banks:
//  - K: lane (grp, tig) reads pieces 2 tig and 2 tig + 1 of rows grp and grp + 8.
//    The quarter's two rows, an even and an odd one, swizzle these pieces to the
//    even and the odd ones. In rows as they lie in the pool (256 bytes apart)
//    both rows fall on the same banks.
//  - V: lane (grp, tig) reads piece grp of rows 2 tig, 2 tig + 1 and those + 8, so
//    that it holds, after O^T, dims 8 grp .. + 7 of each half (bf16), or all 16 of
//    piece grp (E4M3).
// E4M3 codes widen exactly to f16; a query row is multiplied by the power of two
// that puts its largest magnitude into [2^14, 2^15), undone in the score's factor.
#pragma once

#include "decode_rows.cuh"

namespace pa {
namespace {

template <int D, bool FP8>
struct Cells {
  static constexpr int kElt = FP8 ? 1 : 2;
  static constexpr int kHalves = D * kElt > 128 ? 2 : 1;
  static constexpr int kSpan = D * kElt / kHalves;  // bytes of a row of a half: 128 (64)
  static constexpr bool kSw = kSpan == 128;
  static constexpr int kHalfBytes = kChunk * kSpan;
  static constexpr int kBytes = kHalves * kHalfBytes;  // of one cell's keys
  static constexpr int KS = D / 16;                    // k-steps of S
  static constexpr int MT = D / 16;                    // m-tiles of O^T
  static constexpr int kWords = D / 16;                // 16-bit pairs of V that a lane reads of a row

  // First of the eight dims that lane tig takes for k-steps 2 q and 2 q + 1.
  static __device__ __forceinline__ int dim8(int q, int tig) {
    return FP8 ? D / 4 * tig + 8 * q : 64 * (q >> 1) + 16 * tig + 8 * (q & 1);
  }
  static __device__ __forceinline__ int piece(int row, int c) { return (kSw ? c ^ (row & 7) : c) << 4; }

  // Those dims of key `row` as 16-bit pairs.
  static __device__ __forceinline__ void key_words(const uint8_t* cell, int row, int q, int tig,
                                                   uint32_t (&w)[4]) {
    if constexpr (FP8) {
      const int byte = dim8(q, tig);
      const uint2 x = *reinterpret_cast<const uint2*>(cell + row * kSpan + piece(row, byte >> 4) +
                                                      (byte & 15));
      MmaRows<D, FP8>::widen8(x.x, x.y, w);
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(cell + (q >> 1) * kHalfBytes + row * kSpan +
                                                      piece(row, 2 * tig + (q & 1)));
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
  }
  // Lane grp's dims of value `row`; pair w is dims value_dim(w, grp), + 1.
  static __device__ __forceinline__ void value_words(const uint8_t* cell, int row, int grp,
                                                     uint32_t (&w)[kWords]) {
    if constexpr (FP8 && D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(cell + row * kSpan + piece(row, grp));
      MmaRows<D, FP8>::widen8(x.x, x.y, &w[0]);
      MmaRows<D, FP8>::widen8(x.z, x.w, &w[4]);
    } else if constexpr (FP8) {
      const uint2 x = *reinterpret_cast<const uint2*>(cell + row * kSpan + 8 * grp);
      MmaRows<D, FP8>::widen8(x.x, x.y, &w[0]);
    } else {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint4 x =
            *reinterpret_cast<const uint4*>(cell + h * kHalfBytes + row * kSpan + piece(row, grp));
        w[4 * h] = x.x; w[4 * h + 1] = x.y; w[4 * h + 2] = x.z; w[4 * h + 3] = x.w;
      }
    }
  }
  static __device__ __forceinline__ int value_dim(int w, int grp) {
    return FP8 ? D / 8 * grp + 2 * w : 64 * (w >> 2) + 8 * grp + 2 * (w & 3);
  }

  // One cell (keys row .. row + 15 of block id's lines) into shared memory.
  static __device__ __forceinline__ void load(void* dst, const CUtensorMap* map, int line, int id,
                                              uint64_t* bar) {
    tc::tma_load_4d(dst, map, 0, line, 0, id, bar);
  }
};

// The map of a pool half as [block][half][kv head * B + offset][dims of a half],
// one box a cell.
template <int D, bool FP8>
bool cell_map(CUtensorMap* m, const void* half, int num_blocks, int lines) {
  using C = Cells<D, FP8>;
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  constexpr cuuint64_t row = (cuuint64_t)D * C::kElt;
  cuuint64_t dims[4] = {C::kSpan / C::kElt, (cuuint64_t)lines, C::kHalves, (cuuint64_t)num_blocks};
  cuuint64_t strides[3] = {row, C::kSpan, row * (cuuint64_t)lines};
  cuuint32_t box[4] = {C::kSpan / C::kElt, kChunk, C::kHalves, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return encode(m, FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(half), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                C::kSw ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q^T fragments of up to 8 NH rows (row(c): the query of column c, or nullptr: zeros).
template <int D, bool FP8, int NH>
struct QueryCols {
  using C = Cells<D, FP8>;
  uint32_t qb[NH][C::KS][2];
  float sc[NH][2];  // score factors of columns 8 h + 2 tig, + 1

  template <class F>
  __device__ __forceinline__ void load(F row, float q_scale, int grp, int tig) {
    const unsigned full = 0xffffffffu;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const __nv_bfloat16* src = row(8 * h + grp);
      uint4 raw[D / 32];
      float amax = 0.f;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        raw[q] = src ? *reinterpret_cast<const uint4*>(src + C::dim8(q, tig)) : make_uint4(0u, 0u, 0u, 0u);
        if (FP8) {
          float f[8];
          bf16x8_to_f32(raw[q], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
        }
      }
      float up = 1.f, s = q_scale;
      if (FP8) {
        amax = fmaxf(amax, __shfl_xor_sync(full, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(full, amax, 2));
        int e2 = 0;
        if (amax > 0.f)
          e2 = min(100, max(-120, 14 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127)));
        up = __uint_as_float((uint32_t)(e2 + 127) << 23);
        s *= __uint_as_float((uint32_t)(127 - e2) << 23);
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const uint32_t w[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x = w[i];
          if (FP8) {
            const __half2 y = __floats2half2_rn(bf16_lo(x) * up, bf16_hi(x) * up);
            x = *reinterpret_cast<const uint32_t*>(&y);
          }
          qb[h][2 * q + (i >> 1)][i & 1] = x;
        }
      }
      const int lane = threadIdx.x & 31;
      sc[h][0] = __shfl_sync(full, s, (2 * (lane & 3)) * 4);
      sc[h][1] = __shfl_sync(full, s, (2 * (lane & 3) + 1) * 4);
    }
  }

  // Raw products of a cell's keys: s[h] = (key grp, column 2 tig), (grp, 2 tig + 1),
  // (grp + 8, 2 tig), (grp + 8, 2 tig + 1).
  __device__ __forceinline__ void scores(const uint8_t* keys, float (&s)[NH][4], int grp,
                                         int tig) const {
    float acc[NH][2][4];  // two chains of MMAs
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) acc[h][c][0] = acc[h][c][1] = acc[h][c][2] = acc[h][c][3] = 0.f;
#pragma unroll
    for (int q = 0; q < C::KS / 2; ++q) {
      uint32_t w0[4], w1[4];
      C::key_words(keys, grp, q, tig, w0);
      C::key_words(keys, grp + 8, q, tig, w1);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        MmaRows<D, FP8>::mma(acc[h][q & 1], w0[0], w1[0], w0[1], w1[1], qb[h][2 * q][0],
                             qb[h][2 * q][1]);
        MmaRows<D, FP8>::mma(acc[h][q & 1], w0[2], w1[2], w0[3], w1[3], qb[h][2 * q + 1][0],
                             qb[h][2 * q + 1][1]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[h][i] = acc[h][0][i] + acc[h][1][i];
  }
};

}  // namespace
}  // namespace pa
