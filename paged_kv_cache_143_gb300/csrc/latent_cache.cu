// latent_cache.cu — the latent cache: pa_write_latent (rotary turn of the key's
// rotary part, quantisation, scatter by slot), pa_read_latent (gather through
// the block table, widened to bf16) and pa_copy_latent_blocks (copy-on-write).
//
// [vLLM-wiki "블록 테이블"]: token t goes to slot s = block * B + offset. A cell
// holds one latent row c [L] (keys and values of every head are products of
// it) and one rotary row k_r [64] shared by the heads.
//
// E4M3 cells keep c as codes and one fp32 scale per token:
//   scale = 2^e, e the smallest integer with max |c| <= 448 * 2^e (finite
//   elements; e >= -60; 1 for a row of zeros), code = e4m3(c / scale).
// E4M3 is a floating format, so a scale between two powers of two would gain
// no relative precision, only part of a bit at the subnormal end; with a power
// of two the division and code * scale in bf16 are both exact, so a cell is
// rounded once in its life, when it is written. The scale is per token and not
// per pool because rows differ in size and the pool's maximum is unknown while
// it fills. The rotary part stays bf16: its rounding moves scores directly.
//
// All three are HBM scatter / gather work. One warp owns one row, every lane
// moves 16-byte vectors of it, and the row maximum is one warp reduction, so a
// row is read once and written once. Measured: 256 bf16 rows of 512 written in 2.9 us
// (a launch); 8192 E4M3 rows written and read back in 9.1 us; 106 000 E4M3 rows read
// in 33.2 us, 5750 GB/s, four rows of a warp in flight.
#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "rope_angle.cuh"

namespace {

using pa::kErrBounds;

constexpr int kRope = 64;    // rotary dims of a cell: one pair per lane
constexpr int kWarps = 8;    // rows in flight per CTA
constexpr int kMinScaleExp = -60;

// Two fp32 values to E4M3 (nearest even, saturating); NaN is the canonical 0x7F.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  const __nv_fp8x2_storage_t c =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  uint32_t lo = c & 0xFF, hi = c >> 8;
  if (a != a) lo = 0x7F;
  if (b != b) hi = 0x7F;
  return lo | (hi << 8);
}

struct WriteParams {
  uint8_t* latent;         // [slots][L] bf16 or codes
  __nv_bfloat16* rope;     // [slots][64]
  float* scales;           // [slots] (E4M3)
  const __nv_bfloat16* c;  // [T] rows of L, token stride c_ts
  const __nv_bfloat16* kr; // [T] rows of 64, token stride kr_ts
  int64_t c_ts, kr_ts;
  const int64_t* slots;
  const int32_t* positions;  // NULL: the rotary part is stored as it comes
  const float* inv_freq;
  int32_t T, interleaved;
  int64_t num_slots;
  float factor;
  unsigned* err;
};

// One warp per token; lane l holds vectors l, l + 32, .. of the row (L / 256
// vectors of 8 dims) and rotary pair l.
template <int L, bool F8>
__global__ void __launch_bounds__(32 * kWarps) write_latent_kernel(const WriteParams p) {
  constexpr int kV = L / 256;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int64_t s = __ldg(p.slots + t);
  // the row is fetched beside its slot, not after it
  uint4 v[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
    v[i] = *reinterpret_cast<const uint4*>(p.c + t * p.c_ts + (i * 32 + lane) * 8);
  const __nv_bfloat16* kr = p.kr + t * p.kr_ts;
  const int d0 = p.interleaved ? 2 * lane : lane, d1 = p.interleaved ? d0 + 1 : lane + 32;
  __nv_bfloat16 r0 = kr[d0], r1 = kr[d1];
  if (s < 0) return;  // padding
  if (s >= p.num_slots) {
    if (lane == 0) pa::raise_error(p.err, kErrBounds);
    return;
  }
  if (p.positions) {
    float c, sn, x = __bfloat162float(r0), y = __bfloat162float(r1);
    pa::rope_cos_sin(__ldg(p.positions + t), __ldg(p.inv_freq + lane), p.factor, c, sn);
    pa::rope_turn(x, y, c, sn);
    r0 = __float2bfloat16_rn(x);
    r1 = __float2bfloat16_rn(y);
  }
  p.rope[s * kRope + d0] = r0;
  p.rope[s * kRope + d1] = r1;
  if constexpr (!F8) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      *reinterpret_cast<uint4*>(p.latent + (s * L + (i * 32 + lane) * 8) * 2) = v[i];
  } else {
    float f[kV][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      pa::bf16x8_to_f32(v[i], f[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(f[i][e]);
        if (a <= 3.4e38f) amax = fmaxf(amax, a);  // finite (every finite bf16 is below)
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // amax = m * 2^k with m in [1, 2) and 448 = 1.75 * 2^8: e = k - 8, one more
    // if m > 1.75 (subnormal amax falls under the floor of e)
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = amax > 0.f ? max(e, kMinScaleExp) : 0;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // e <= 120
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      uint2 w;
      w.x = to_e4m3x2(f[i][0] * inv, f[i][1] * inv) | to_e4m3x2(f[i][2] * inv, f[i][3] * inv) << 16;
      w.y = to_e4m3x2(f[i][4] * inv, f[i][5] * inv) | to_e4m3x2(f[i][6] * inv, f[i][7] * inv) << 16;
      *reinterpret_cast<uint2*>(p.latent + s * L + (i * 32 + lane) * 8) = w;
    }
    if (lane == 0) p.scales[s] = __uint_as_float((uint32_t)(127 + e) << 23);
  }
}

struct ReadParams {
  const uint8_t* latent;
  const __nv_bfloat16* rope;
  const float* scales;
  const int32_t* tables;  // [R][max_blocks]
  const int32_t* start;   // [R+1] output row of request r's first token
  const int32_t* first;   // [R] position of that token (NULL: 0)
  __nv_bfloat16* c;
  __nv_bfloat16* kr;
  int64_t c_ts, kr_ts;
  int32_t max_blocks, R, N, num_blocks, B;
  unsigned* err;
};

constexpr int kReadRows = 4;  // rows of one warp, all in flight together

// Lanes 0 .. kReadRows - 1 look their rows' slots up side by side (binary
// search of the request, then the block table), then the warp moves the rows.
template <int L, bool F8>
__global__ void __launch_bounds__(32 * kWarps) read_latent_kernel(const ReadParams p) {
  constexpr int kV = L / 256;
  const int lane = threadIdx.x & 31;
  const int64_t row0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kReadRows;
  int64_t slot = -1;
  if (lane < kReadRows && row0 + lane < p.N) {
    const int32_t i = (int32_t)(row0 + lane);
    int lo = 0, hi = p.R;  // the last r in [0, R] with start[r] <= i (start[0] = 0)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.start + mid) <= i) lo = mid; else hi = mid - 1;
    }
    if (lo < p.R) {  // rows at or past start[R] belong to nobody and stay as they are
      const int64_t pos = (int64_t)i - __ldg(p.start + lo) + (p.first ? __ldg(p.first + lo) : 0);
      bool ok = pos >= 0 && pos < (int64_t)p.max_blocks * p.B;
      if (ok) {
        const int32_t blk = __ldg(p.tables + (int64_t)lo * p.max_blocks + pos / p.B);
        ok = blk >= 0 && blk < p.num_blocks;
        if (ok) slot = (int64_t)blk * p.B + pos % p.B;
      }
      if (!ok) pa::raise_error(p.err, kErrBounds);
    }
  }
  if (row0 == 0 && lane == 0 && (__ldg(p.start) != 0 || __ldg(p.start + p.R) > p.N))
    pa::raise_error(p.err, kErrBounds);  // more rows than the outputs hold
  int64_t s[kReadRows];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) s[k] = __shfl_sync(0xffffffffu, slot, k);
  uint4 wide[kReadRows][F8 ? 1 : kV];
  uint2 codes[kReadRows][F8 ? kV : 1];
  uint32_t rot[kReadRows];
  float scale[kReadRows];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    if (s[k] < 0) continue;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (F8)
        codes[k][i] = __ldcs(reinterpret_cast<const uint2*>(p.latent + s[k] * L) + i * 32 + lane);
      else
        wide[k][i] =
            __ldcs(reinterpret_cast<const uint4*>(p.latent + s[k] * L * 2) + i * 32 + lane);
    }
    rot[k] = __ldcs(reinterpret_cast<const uint32_t*>(p.rope + s[k] * kRope) + lane);
    if constexpr (F8) scale[k] = __ldg(p.scales + s[k]);
  }
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    if (s[k] < 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.c + (row0 + k) * p.c_ts);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (F8) {
        float f[8];
        pa::e4m3x8_to_f32(codes[k][i], f);
        uint4 v;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j] * scale[k], f[2 * j + 1] * scale[k]);
          w[j] = *reinterpret_cast<uint32_t*>(&h);
        }
        dst[i * 32 + lane] = v;
      } else {
        dst[i * 32 + lane] = wide[k][i];
      }
    }
    reinterpret_cast<uint32_t*>(p.kr + (row0 + k) * p.kr_ts)[lane] = rot[k];
  }
}

// One CTA per pair: latents, rotary parts and scales of block src[i] to dst[i].
__global__ void __launch_bounds__(256) copy_latent_kernel(uint8_t* latent, uint8_t* rope,
                                                          float* scales, const int32_t* src,
                                                          const int32_t* dst, int32_t num_blocks,
                                                          int64_t latent_bytes, int32_t B,
                                                          unsigned* err) {
  const int32_t s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
    if (threadIdx.x == 0) pa::raise_error(err, kErrBounds);
    return;
  }
  auto copy = [&](uint8_t* pool, int64_t bytes) {
    const uint4* from = reinterpret_cast<const uint4*>(pool + s * bytes);
    uint4* to = reinterpret_cast<uint4*>(pool + d * bytes);
    for (int64_t j = threadIdx.x; j < bytes / 16; j += blockDim.x) to[j] = from[j];
  };
  copy(latent, latent_bytes);
  copy(rope, (int64_t)B * kRope * 2);
  if (scales && (int)threadIdx.x < B)
    scales[(int64_t)d * B + threadIdx.x] = scales[(int64_t)s * B + threadIdx.x];
}

bool row_stride_ok(int64_t stride, int width) { return stride >= width && stride % 8 == 0; }

}  // namespace

namespace pa {

pa_status check_latent_pool(const pa_latent_pool* pool) {
  if (!pool || !pool->latent || !pool->rope) return PA_ERR_INVALID;
  if (!aligned16(pool->latent) || !aligned16(pool->rope)) return PA_ERR_INVALID;
  if (pool->num_blocks < 0) return PA_ERR_INVALID;
  if (pool->latent_dim != 256 && pool->latent_dim != 512) return PA_ERR_UNSUPPORTED;
  if (pool->rope_dim != kRope) return PA_ERR_UNSUPPORTED;
  if (pool->block_size != 16 && pool->block_size != 32 && pool->block_size != 64)
    return PA_ERR_UNSUPPORTED;
  if (pool->dtype != PA_KV_BF16 && pool->dtype != PA_KV_FP8_E4M3) return PA_ERR_UNSUPPORTED;
  if (pool->dtype == PA_KV_FP8_E4M3 && (!pool->scales || !aligned16(pool->scales)))
    return PA_ERR_INVALID;
  // a row of the pool is addressed by a 32-bit tensor-map coordinate
  if ((int64_t)pool->num_blocks * pool->block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace pa

extern "C" pa_status pa_write_latent(const pa_latent_pool* pool, const void* latent,
                                     int64_t latent_stride, const void* k_rope,
                                     int64_t rope_stride, const int32_t* positions,
                                     const float* inv_freq, int32_t layout, float factor,
                                     const int64_t* slot_mapping, int32_t T,
                                     pa_stream_t stream) {
  pa_status st = pa::check_latent_pool(pool);
  if (st != PA_OK) return st;
  if (T < 0) return PA_ERR_INVALID;
  if (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED) return PA_ERR_INVALID;
  if ((positions == nullptr) != (inv_freq == nullptr)) return PA_ERR_INVALID;
  if (positions && (!(factor > 0.f) || factor > 3.0e38f)) return PA_ERR_INVALID;
  if (T == 0) return PA_OK;
  if (!latent || !k_rope || !slot_mapping || !pa::aligned16(latent) ||
      (reinterpret_cast<uintptr_t>(k_rope) & 1u) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
    return PA_ERR_INVALID;
  if (latent_stride < 0 || latent_stride % 8 != 0 || rope_stride < 0) return PA_ERR_INVALID;
  WriteParams p{};
  p.latent = static_cast<uint8_t*>(pool->latent);
  p.rope = static_cast<__nv_bfloat16*>(pool->rope);
  p.scales = pool->scales;
  p.c = static_cast<const __nv_bfloat16*>(latent);
  p.kr = static_cast<const __nv_bfloat16*>(k_rope);
  p.c_ts = latent_stride;
  p.kr_ts = rope_stride;
  p.slots = slot_mapping;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.T = T;
  p.interleaved = layout == PA_ROPE_INTERLEAVED;
  p.num_slots = (int64_t)pool->num_blocks * pool->block_size;
  p.factor = factor;
  p.err = pa::error_word();
  if (!p.err) return PA_ERR_CUDA;
  const unsigned grid = (unsigned)(((int64_t)T + kWarps - 1) / kWarps);
  cudaStream_t s = pa::as_stream(stream);
  const bool f8 = pool->dtype == PA_KV_FP8_E4M3;
  if (pool->latent_dim == 512) {
    if (f8) write_latent_kernel<512, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else write_latent_kernel<512, false><<<grid, 32 * kWarps, 0, s>>>(p);
  } else {
    if (f8) write_latent_kernel<256, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else write_latent_kernel<256, false><<<grid, 32 * kWarps, 0, s>>>(p);
  }
  return pa::launch_status();
}

extern "C" pa_status pa_read_latent(const pa_latent_pool* pool, const int32_t* block_tables,
                                    int32_t max_blocks, const int32_t* kv_start_loc,
                                    const int32_t* first, int32_t num_reqs, int32_t num_tokens,
                                    void* latent_out, int64_t latent_stride, void* rope_out,
                                    int64_t rope_stride, pa_stream_t stream) {
  pa_status st = pa::check_latent_pool(pool);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (num_reqs == 0 || !block_tables || !kv_start_loc || !latent_out || !rope_out ||
      !pa::aligned16(latent_out) || (reinterpret_cast<uintptr_t>(rope_out) & 3u))
    return PA_ERR_INVALID;
  if (!row_stride_ok(latent_stride, pool->latent_dim) || rope_stride < kRope ||
      rope_stride % 2 != 0)
    return PA_ERR_INVALID;
  ReadParams p{};
  p.latent = static_cast<const uint8_t*>(pool->latent);
  p.rope = static_cast<const __nv_bfloat16*>(pool->rope);
  p.scales = pool->scales;
  p.tables = block_tables;
  p.start = kv_start_loc;
  p.first = first;
  p.c = static_cast<__nv_bfloat16*>(latent_out);
  p.kr = static_cast<__nv_bfloat16*>(rope_out);
  p.c_ts = latent_stride;
  p.kr_ts = rope_stride;
  p.max_blocks = max_blocks;
  p.R = num_reqs;
  p.N = num_tokens;
  p.num_blocks = pool->num_blocks;
  p.B = pool->block_size;
  p.err = pa::error_word();
  if (!p.err) return PA_ERR_CUDA;
  const unsigned grid =
      (unsigned)(((int64_t)num_tokens + kWarps * kReadRows - 1) / (kWarps * kReadRows));
  cudaStream_t s = pa::as_stream(stream);
  const bool f8 = pool->dtype == PA_KV_FP8_E4M3;
  if (pool->latent_dim == 512) {
    if (f8) read_latent_kernel<512, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else read_latent_kernel<512, false><<<grid, 32 * kWarps, 0, s>>>(p);
  } else {
    if (f8) read_latent_kernel<256, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else read_latent_kernel<256, false><<<grid, 32 * kWarps, 0, s>>>(p);
  }
  return pa::launch_status();
}

extern "C" pa_status pa_copy_latent_blocks(const pa_latent_pool* pool, const int32_t* src,
                                           const int32_t* dst, int32_t n, pa_stream_t stream) {
  pa_status st = pa::check_latent_pool(pool);
  if (st != PA_OK) return st;
  if (n < 0) return PA_ERR_INVALID;
  if (n == 0) return PA_OK;
  if (!src || !dst) return PA_ERR_INVALID;
  unsigned* err = pa::error_word();
  if (!err) return PA_ERR_CUDA;
  const bool f8 = pool->dtype == PA_KV_FP8_E4M3;
  const int64_t latent_bytes = (int64_t)pool->block_size * pool->latent_dim * (f8 ? 1 : 2);
  copy_latent_kernel<<<(unsigned)n, 256, 0, pa::as_stream(stream)>>>(
      static_cast<uint8_t*>(pool->latent), static_cast<uint8_t*>(pool->rope),
      f8 ? pool->scales : nullptr, src, dst, pool->num_blocks, latent_bytes, pool->block_size, err);
  return pa::launch_status();
}
