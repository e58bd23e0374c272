// compact_cache.cu — pa_compact_cache: the cells that a request keeps move, in
// order, to the first cells of its (new) block table, with their mass.
//
// Copy work: two bytes moved for each byte kept. kept is ascending, so cell i
// comes from a place kept[i] >= i, and in the same blocks it may be written once
// the cells kept[0 .. i] have been read: one CTA goes through a request's cells
// in order, a tile at a time, and reads tile x + 1 into registers before it
// writes tile x. The CTAs divide what does not depend on each other: requests,
// K and V, kv heads and, where those leave SMs idle, the 16-byte pieces of a row
// (a row's 64 to 256 bytes are what a gather brings at once: halves of them, read by
// two CTAs at different times, take 57 us where whole rows take 50). Where 1024 cells
// come from and go to is worked out once for all threads of a row and kept in shared
// memory, the next 1024 cells' while these are moved. 16 requests cut to 4096 tokens of
// 8 kv heads, E4M3: 50 us for 269 MB moved, 5.4 TB/s (0.80 of the copy rate); what is
// left is the gather's latency, 16 loads of 16 bytes in flight a thread.
#include "batch_rows.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kDeep = 8;     // 16-byte pieces of a thread in flight, twice
constexpr int kBatch = 1024;  // cells whose places are known at once
constexpr uint32_t kNone = 0xffffffffu;

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
  // Places of a batch's cells: pool rows of the kv head (below 2^32: the pool fits the GPU)
  // from which and to which they move, kNone where there is nothing to do.
  __shared__ uint32_t from[2][kBatch], to[2][kBatch];
  constexpr int kMine = kBatch / kThreads;  // cells whose places a thread works out
  int place[kMine], id[2][kMine];
  auto fetch_kept = [&](int base) {
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int i = base + u * kThreads + (int)threadIdx.x;
      place[u] = i < n ? __ldg(kept + i) : 0;
    }
  };
  auto fetch_ids = [&](int base) {
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int i = base + u * kThreads + (int)threadIdx.x;
      const int a = place[u] / p.B, b = i / p.B;
      id[0][u] = i < n && place[u] >= 0 && a < p.max_blocks ? __ldg(src + a) : -1;
      id[1][u] = i < n && b < p.dst_blocks ? __ldg(dst + b) : -1;
    }
  };
  auto settle = [&](int base, int turn) {
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int at = u * kThreads + (int)threadIdx.x, i = base + at;
      uint32_t a = kNone, b = kNone;
      if (id[0][u] >= 0 && id[0][u] < p.num_blocks && id[1][u] >= 0 && id[1][u] < p.num_blocks) {
        a = (uint32_t)(((int64_t)id[0][u] * p.Hkv + kvh) * p.B + place[u] % p.B);
        b = (uint32_t)(((int64_t)id[1][u] * p.Hkv + kvh) * p.B + i % p.B);
        if (a == b) a = b = kNone;  // it stays where it is
      } else if (i < n) {
        raise_error(p.err, kErrBounds);
      }
      from[turn][at] = a;
      to[turn][at] = b;
    }
  };
  fetch_kept(0);
  fetch_ids(0);
  settle(0, 0);
  __syncthreads();
  uint4 v[2][kDeep];
  const int tile = step * kDeep;  // divides kBatch: both are powers of two
  auto read = [&](int base, uint4 (&x)[kDeep]) {
    if (base >= n) return;
    const uint32_t* f = from[(base / kBatch) & 1] + base % kBatch;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t a = f[u * step + row];
      if (a != kNone) x[u] = *reinterpret_cast<const uint4*>(pool + (int64_t)a * p.row_bytes + byte);
    }
  };
  auto write = [&](int base, const uint4 (&x)[kDeep]) {
    if (base >= n) return;
    const uint32_t* t = to[(base / kBatch) & 1] + base % kBatch;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t b = t[u * step + row];
      if (b != kNone) *reinterpret_cast<uint4*>(pool + (int64_t)b * p.row_bytes + byte) = x[u];
    }
  };
  read(0, v[0]);
  fetch_kept(kBatch);
  // One tile a turn: the next one is read, then, when all threads have read theirs, this
  // one written. In the first turn of a batch the next batch's places are worked out, in
  // the halves of `from` and `to` that the batch before used, which is all written: after
  // this turn's barrier, or where a batch has no third turn before they are read, ahead of it.
  const bool early = 2 * tile >= kBatch;
  auto turn = [&](int base, uint4 (&mine)[kDeep], uint4 (&other)[kDeep]) {
    const bool opens = base % kBatch == 0;
    if (opens) {
      fetch_ids(base + kBatch);
      if (early) {
        __syncthreads();
        settle(base + kBatch, (base / kBatch + 1) & 1);
        __syncthreads();
      }
    }
    read(base + tile, other);
    __syncthreads();
    write(base, mine);
    if (opens) {
      if (!early) settle(base + kBatch, (base / kBatch + 1) & 1);
      fetch_kept(base + 2 * kBatch);
    }
  };
  for (int base = 0; base < n; base += 2 * tile) {
    turn(base, v[0], v[1]);
    if (base + tile < n) turn(base + tile, v[1], v[0]);
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
  if (num_reqs > 65535 || k > kMostTokens ||
      (int64_t)pool->num_blocks * pool->num_kv_heads * pool->block_size >= 0xffffffffll)
    return PA_ERR_UNSUPPORTED;
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
  // rows in 32-byte pieces (a sector) at the least, while SMs are idle
  p.split = 1;
  while ((int64_t)num_reqs * p.Hkv * 2 * p.split < num_sms() && p.row_bytes / p.split > 32) p.split *= 2;
  const dim3 grid((unsigned)(p.Hkv * 2 * p.split + 1), (unsigned)num_reqs);
  compact_kernel<<<grid, kThreads, 0, as_stream(stream)>>>(p);
  return launch_status();
}
