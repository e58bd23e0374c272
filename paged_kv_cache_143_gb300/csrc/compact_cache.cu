// compact_cache.cu — pa_compact_cache: the cells that a request keeps move, in
// order, to the first cells of its (new) block table, with their mass.
//
// Copy work: two bytes moved for each byte kept. kept is ascending, so cell i
// comes from a place kept[i] >= i, and in the same blocks it may be written once
// the cells kept[0 .. i] have been read: one CTA goes through a request's cells
// in order, a tile at a time, and reads tile x + 1 into registers before it
// writes tile x. The CTAs divide what does not depend on each other: requests,
// K and V, kv heads and, where those are few, the 16-byte pieces of a row.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kDeep = 4;  // 16-byte pieces of a thread in flight

struct CompactParams {
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int32_t* src;   // [R][max_blocks]
  const int32_t* dst;   // [R][dst_blocks]
  const int32_t* kept;  // [R][k]
  const int32_t* kept_lens;
  const float* mass_in;
  float* mass_out;
  int64_t mass_stride;
  const int32_t* idx;
  int max_reqs, max_blocks, dst_blocks, R, k, Hkv, B, num_blocks, row_bytes, split;
  unsigned* err;
};

// The pool row of cell `n` of a request for a kv head, or -1 (flagged).
__device__ __forceinline__ int64_t pool_row(const CompactParams& p, const int32_t* table,
                                            int blocks, int n, int kvh) {
  const int b = n / p.B;
  if (n < 0 || b >= blocks) {
    raise_error(p.err, kErrBounds);
    return -1;
  }
  const int id = __ldg(table + b);
  if (id < 0 || id >= p.num_blocks) {
    raise_error(p.err, kErrBounds);
    return -1;
  }
  return ((int64_t)id * p.Hkv + kvh) * p.B + (n - b * p.B);
}

__global__ void __launch_bounds__(kThreads) compact_kernel(CompactParams p) {
  const int r = blockIdx.y;
  const int n = p.kept_lens[r];
  if (n < 0 || n > p.k) {
    if (threadIdx.x == 0) raise_error(p.err, kErrBounds);
    return;
  }
  const int32_t* kept = p.kept + (int64_t)r * p.k;
  const int lanes = p.Hkv * 2 * p.split;
  if ((int)blockIdx.x == lanes) {  // the request's mass
    if (!p.mass_in) return;
    const int at = p.idx ? p.idx[r] : r;
    if (at < 0 || at >= p.max_reqs || n > p.mass_stride) {
      if (threadIdx.x == 0) raise_error(p.err, kErrBounds);
      return;
    }
    const float* in = p.mass_in + (int64_t)at * p.mass_stride;
    float* out = p.mass_out + (int64_t)at * p.mass_stride;
    for (int base = 0; base < n; base += kThreads * kDeep) {
      float v[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int i = base + u * kThreads + (int)threadIdx.x;
        if (i < n) {
          const int from = kept[i];
          if (from < 0 || from >= p.mass_stride)
            raise_error(p.err, kErrBounds);
          else
            v[u] = in[from];
        }
      }
      __syncthreads();  // read by all before any is overwritten
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int i = base + u * kThreads + (int)threadIdx.x;
        if (i < n && kept[i] >= 0 && kept[i] < p.mass_stride) out[i] = v[u];
      }
    }
    return;
  }
  const int part = blockIdx.x % p.split;
  const int kvh = (int)blockIdx.x / p.split % p.Hkv;
  uint8_t* pool = (int)blockIdx.x / p.split / p.Hkv ? p.v_pool : p.k_pool;
  const int32_t* src = p.src + (int64_t)r * p.max_blocks;
  const int32_t* dst = p.dst + (int64_t)r * p.dst_blocks;
  const int pieces = p.row_bytes / 16 / p.split;      // of this CTA, a row
  const int step = kThreads / pieces;                 // rows that the CTA moves at once
  const int row = (int)threadIdx.x / pieces;
  const int64_t byte = ((int)threadIdx.x % pieces + part * pieces) * 16;
  uint4 v[2][kDeep];
  int64_t to[2][kDeep];
  auto read = [&](int base, uint4 (&x)[kDeep], int64_t (&w)[kDeep]) {
    int64_t from[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = base + u * step + row;
      from[u] = w[u] = -1;
      if (i < n) {
        from[u] = pool_row(p, src, p.max_blocks, __ldg(kept + i), kvh);
        w[u] = pool_row(p, dst, p.dst_blocks, i, kvh);
        if (from[u] < 0 || from[u] == w[u]) w[u] = -1;  // nothing to do
      }
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (w[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(pool + from[u] * p.row_bytes + byte);
  };
  auto write = [&](const uint4 (&x)[kDeep], const int64_t (&w)[kDeep]) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (w[u] >= 0) *reinterpret_cast<uint4*>(pool + w[u] * p.row_bytes + byte) = x[u];
  };
  const int tile = step * kDeep;
  read(0, v[0], to[0]);
  for (int base = 0; base < n; base += 2 * tile) {
    read(base + tile, v[1], to[1]);
    __syncthreads();  // what tile `base` overwrites has been read
    write(v[0], to[0]);
    read(base + 2 * tile, v[0], to[0]);
    __syncthreads();
    write(v[1], to[1]);
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_compact_cache(const pa_kv_pool* pool, const int32_t* src_tables,
                                      int32_t max_blocks, const int32_t* dst_tables,
                                      int32_t dst_blocks, const int32_t* kept, int32_t k,
                                      const int32_t* kept_lens, int32_t num_reqs,
                                      const float* mass_in, float* mass_out, int64_t mass_stride,
                                      int32_t max_reqs, const int32_t* idx_mapping,
                                      pa_stream_t stream) {
  using namespace pa;
  pa_status st = check_pool(pool);
  if (st != PA_OK) return st;
  if (max_blocks < 0 || dst_blocks < 0 || k < 0 || num_reqs < 0 || (mass_in == nullptr) != (mass_out == nullptr) ||
      (mass_in && (mass_stride < 0 || max_reqs < 0)))
    return PA_ERR_INVALID;
  if (num_reqs == 0 || k == 0) return PA_OK;
  if (!src_tables || !dst_tables || !kept || !kept_lens ||
      (reinterpret_cast<uintptr_t>(mass_in) & 3u) || (reinterpret_cast<uintptr_t>(mass_out) & 3u))
    return PA_ERR_INVALID;
  if (num_reqs > 65535) return PA_ERR_UNSUPPORTED;
  CompactParams p{};
  p.k_pool = static_cast<uint8_t*>(pool->k_pool);
  p.v_pool = static_cast<uint8_t*>(pool->v_pool);
  p.src = src_tables;
  p.dst = dst_tables;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.mass_in = mass_in;
  p.mass_out = mass_out;
  p.mass_stride = mass_stride;
  p.idx = idx_mapping;
  p.max_reqs = max_reqs;
  p.max_blocks = max_blocks;
  p.dst_blocks = dst_blocks;
  p.R = num_reqs;
  p.k = k;
  p.Hkv = pool->num_kv_heads;
  p.B = pool->block_size;
  p.num_blocks = pool->num_blocks;
  p.row_bytes = pool->head_dim * (pool->dtype == PA_KV_BF16 ? 2 : 1);
  p.err = error_word();
  if (!p.err) return PA_ERR_CUDA;
  // rows in 32-byte pieces (a sector) at the least, while two CTAs do not fill each SM
  p.split = 1;
  while ((int64_t)num_reqs * p.Hkv * 2 * p.split < 2 * num_sms() && p.row_bytes / p.split > 32)
    p.split *= 2;
  const dim3 grid((unsigned)(p.Hkv * 2 * p.split + 1), (unsigned)num_reqs);
  compact_kernel<<<grid, kThreads, 0, as_stream(stream)>>>(p);
  return launch_status();
}
