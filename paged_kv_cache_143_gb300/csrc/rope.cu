// rope.cu — pa_rope: rotary positions applied to the leading part of each head.
//
// Pair i of a head at position p is turned by the angle p * inv_freq[i]:
//   (x, y) -> factor * (x cos - y sin, y cos + x sin),
// the pair being dims (2i, 2i + 1) or (i, i + rot / 2). The work is one read
// and one write of every element (HBM-bound when large, launch latency when
// small); the angles depend on (token, pair) only, so a CTA computes its
// tokens' cosines and sines once into shared memory, while its vectors of x are
// already on their way (four units of 16 or 32 bytes a thread), and every head
// reuses them. fp32 arithmetic, one rounding to bf16. Measured: 8192 tokens x 32
// heads x 128 dims (64 turned, half layout) in 24.9 us, 5390 GB/s (bound by HBM and by
// instructions about alike); x 128 heads x 64 dims, interleaved, 52 us, 5130 GB/s (three
// units in flight and five CTAs an SM: 23.1 and 58); 256 x 64 x 64 in 3.6 us, a launch.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "rope_angle.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;        // units of a thread that are loaded before the angles
constexpr int kUnits = kAhead * kThreads;  // units a CTA aims at
constexpr int kMaxPairs = 128;   // rot_dim <= 256
constexpr int kMaxTokens = 64;   // tokens of one CTA
constexpr int kMaxAngles = 1024; // (token, pair) angles of one CTA
constexpr int kMaxDim = 32768;   // of a head, for the exact reciprocals
constexpr int64_t kMaxStride = (int64_t)1 << 38;  // elements: more than any memory holds
constexpr int kMaxHeadGroups = 65535;             // CTAs along the heads

struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const int32_t* positions;
  const float* inv_freq;
  int64_t x_ts, x_hs, o_ts, o_hs;  // token and head strides, elements
  int32_t T, H, pairs, interleaved;
  int32_t rot_units, pass_units;   // units per head that are turned, and copied
  int32_t tokens, heads;           // of one CTA
  uint32_t by_rot, by_pass, by_heads;  // reciprocals of rot_units, pass_units and H
  float factor;
};

// i / d by d's reciprocal 2^32 / d + 1 (0 for d = 1), exact while i * d < 2^32.
uint32_t reciprocal(int32_t d) { return d <= 1 ? 0u : (uint32_t)((1ull << 32) / d + 1); }
__device__ __forceinline__ int divide(int i, uint32_t by) {
  return by == 0u ? i : (int)__umulhi((uint32_t)i, by);
}

// A unit of the vector form: 8 dims (4 pairs) of the interleaved layout; 8 + 8
// dims (8 pairs) of the half layout; 8 dims passed through.
struct VecUnit {
  uint4 a, b;
  __device__ __forceinline__ static int64_t dim(const RopeParams& p, int u) {
    if (u < p.rot_units || p.interleaved) return u * 8;
    return 2 * p.pairs + (u - p.rot_units) * 8;
  }
  __device__ __forceinline__ void load(const RopeParams& p, const __nv_bfloat16* x, int u) {
    const __nv_bfloat16* src = x + dim(p, u);
    a = *reinterpret_cast<const uint4*>(src);
    if (!p.interleaved && u < p.rot_units) b = *reinterpret_cast<const uint4*>(src + p.pairs);
  }
  __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return v;
  }
  __device__ __forceinline__ void store(const RopeParams& p, __nv_bfloat16* out, int u,
                                        const float2* cs) const {
    __nv_bfloat16* dst = out + dim(p, u);
    if (u >= p.rot_units) {
      *reinterpret_cast<uint4*>(dst) = a;
      return;
    }
    float f[8];
    pa::bf16x8_to_f32(a, f);
    if (p.interleaved) {
      const float4* cs2 = reinterpret_cast<const float4*>(cs + u * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 t = cs2[i];
        pa::rope_turn(f[4 * i], f[4 * i + 1], t.x, t.y);
        pa::rope_turn(f[4 * i + 2], f[4 * i + 3], t.z, t.w);
      }
      *reinterpret_cast<uint4*>(dst) = pack(f);
    } else {
      float g[8];
      pa::bf16x8_to_f32(b, g);
      const float4* cs2 = reinterpret_cast<const float4*>(cs + u * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = cs2[i];
        pa::rope_turn(f[2 * i], g[2 * i], t.x, t.y);
        pa::rope_turn(f[2 * i + 1], g[2 * i + 1], t.z, t.w);
      }
      *reinterpret_cast<uint4*>(dst) = pack(f);
      *reinterpret_cast<uint4*>(dst + p.pairs) = pack(g);
    }
  }
};

// A unit of the scalar form (odd sizes, strides or addresses): one pair, or
// one dim passed through.
struct ScalarUnit {
  __nv_bfloat16 a, b;
  __device__ __forceinline__ void load(const RopeParams& p, const __nv_bfloat16* x, int u) {
    if (u >= p.pairs) {
      a = x[p.pairs + u];
    } else {
      a = x[p.interleaved ? 2 * u : u];
      b = x[p.interleaved ? 2 * u + 1 : u + p.pairs];
    }
  }
  __device__ __forceinline__ void store(const RopeParams& p, __nv_bfloat16* out, int u,
                                        const float2* cs) const {
    if (u >= p.pairs) {
      out[p.pairs + u] = a;
      return;
    }
    float f = __bfloat162float(a), g = __bfloat162float(b);
    pa::rope_turn(f, g, cs[u].x, cs[u].y);
    out[p.interleaved ? 2 * u : u] = __float2bfloat16_rn(f);
    out[p.interleaved ? 2 * u + 1 : u + p.pairs] = __float2bfloat16_rn(g);
  }
};

// grid (token groups, head groups). A CTA's turned units come first, then its
// copied ones, so that a warp does one of the two (mixed, a warp went through both:
// 160 instructions for 16 bytes a lane). In place (out == x) is safe: a unit's dims
// are read and written by one thread, and its loads come first.
template <typename Unit>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeParams p) {
  __shared__ alignas(16) float2 cs[kMaxAngles];
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
  const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
  const int turned = nt * nh * p.rot_units, n = turned + nt * nh * p.pass_units;
  struct Place {
    int tok, head, unit;
  };
  auto place = [&](int i) {
    const bool rot = i < turned;
    const int j = rot ? i : i - turned;
    const int at = divide(j, rot ? p.by_rot : p.by_pass);  // token by token, head by head
    const int unit = j - at * (rot ? p.rot_units : p.pass_units) + (rot ? 0 : p.rot_units);
    const int tok = p.tokens == 1 ? 0 : divide(at, p.by_heads);  // (then nh = H)
    return Place{tok, at - tok * nh, unit};
  };
  const __nv_bfloat16* x = p.x + t0 * p.x_ts + h0 * p.x_hs;
  __nv_bfloat16* out = p.out + t0 * p.o_ts + h0 * p.o_hs;
  Unit ahead[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < n) {
      const Place at = place(i);
      ahead[k].load(p, x + at.tok * p.x_ts + at.head * p.x_hs, at.unit);
    }
  }
  for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
    const int tok = i / p.pairs;
    float c, s;
    pa::rope_cos_sin(__ldg(p.positions + t0 + tok), __ldg(p.inv_freq + i - tok * p.pairs),
                     p.factor, c, s);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < n) {
      const Place at = place(i);  // (found again: registers are in-flight bytes)
      ahead[k].store(p, out + at.tok * p.o_ts + at.head * p.o_hs, at.unit, cs + at.tok * p.pairs);
    }
  }
  for (int i = threadIdx.x + kAhead * kThreads; i < n; i += kThreads) {
    const Place at = place(i);
    Unit v;
    v.load(p, x + at.tok * p.x_ts + at.head * p.x_hs, at.unit);
    v.store(p, out + at.tok * p.o_ts + at.head * p.o_hs, at.unit, cs + at.tok * p.pairs);
  }
}

}  // namespace

extern "C" pa_status pa_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                             void* out, int64_t out_token_stride, int64_t out_head_stride,
                             const int32_t* positions, int32_t T, int32_t num_heads,
                             int32_t head_dim, const float* inv_freq, int32_t rot_dim,
                             int32_t layout, float factor, pa_stream_t stream) {
  if (T < 0 || num_heads <= 0 || head_dim <= 0 || rot_dim < 0 || rot_dim > head_dim)
    return PA_ERR_INVALID;
  if (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED) return PA_ERR_INVALID;
  if (!(factor > 0.f) || factor > 3.0e38f) return PA_ERR_INVALID;
  if (rot_dim % 2 != 0 || rot_dim > 2 * kMaxPairs || head_dim > kMaxDim)
    return PA_ERR_UNSUPPORTED;
  if (T == 0) return PA_OK;
  if (!x || !out || !positions || (rot_dim > 0 && !inv_freq)) return PA_ERR_INVALID;
  // rows [token][head] of out must not share elements: heads inside tokens, or
  // tokens inside heads
  // (the stride of a dimension of one entry is never used)
  const int64_t D = head_dim, xt = T > 1 ? x_token_stride : 0, ot = T > 1 ? out_token_stride : 0;
  const int64_t xh = num_heads > 1 ? x_head_stride : 0, oh = num_heads > 1 ? out_head_stride : 0;
  for (int64_t stride : {xt, xh, ot, oh})
    if (stride < 0 || stride >= kMaxStride) return PA_ERR_INVALID;
  // whether `outer` reaches past n rows of D that lie `inner` apart, by division
  auto past = [&](int64_t outer, int64_t n, int64_t inner) {
    return outer >= D && (n == 1 || inner <= (outer - D) / (n - 1));
  };
  const bool heads_inside = (num_heads == 1 || oh >= D) && (T == 1 || past(ot, num_heads, oh));
  const bool tokens_inside = (T == 1 || ot >= D) && (num_heads == 1 || past(oh, T, ot));
  if (!heads_inside && !tokens_inside) return PA_ERR_INVALID;
  if (x == out && ((T > 1 && xt != ot) || (num_heads > 1 && xh != oh))) return PA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(x) & 1u) || (reinterpret_cast<uintptr_t>(out) & 1u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 3u))
    return PA_ERR_INVALID;

  RopeParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.x_ts = xt; p.x_hs = xh; p.o_ts = ot; p.o_hs = oh;
  p.T = T;
  p.H = num_heads;
  p.pairs = rot_dim / 2;
  p.interleaved = layout == PA_ROPE_INTERLEAVED;
  p.factor = factor;
  // 16-byte vectors where every row and every half starts on 16 bytes
  const bool vec = pa::aligned16(x) && pa::aligned16(out) && (xt | xh | ot | oh | D) % 8 == 0 &&
                   (p.interleaved ? rot_dim : p.pairs) % 8 == 0;
  const int pass = x == out ? 0 : head_dim - rot_dim;  // dims copied
  p.rot_units = vec ? (p.interleaved ? rot_dim / 8 : p.pairs / 8) : p.pairs;
  p.pass_units = vec ? pass / 8 : pass;
  const int units = p.rot_units + p.pass_units;
  if (units == 0) return PA_OK;  // in place, nothing turned
  // CTAs of about kUnits units: several tokens of few heads, or some heads of one token
  const int64_t per_token = (int64_t)num_heads * units;
  p.tokens = 1;
  p.heads = num_heads;
  if (per_token > kUnits) {
    const int64_t groups = std::min<int64_t>((per_token + kUnits - 1) / kUnits, kMaxHeadGroups);
    p.heads = (int)((num_heads + groups - 1) / groups);
    // (then a token has 2^31 elements and more)
    if ((int64_t)p.heads * units * units >= (int64_t)1 << 32 && p.heads > 1)
      return PA_ERR_UNSUPPORTED;
  } else {
    p.tokens = (int)(kUnits / per_token);
    if (p.tokens > kMaxTokens) p.tokens = kMaxTokens;
    if (p.pairs > 0 && p.tokens > kMaxAngles / p.pairs) p.tokens = kMaxAngles / p.pairs;
    // no fewer than two CTAs an SM while there are tokens to spread
    const int spread = T / (2 * pa::num_sms());
    if (p.tokens > spread) p.tokens = spread > 0 ? spread : 1;
  }
  p.by_rot = reciprocal(p.rot_units);
  p.by_pass = reciprocal(p.pass_units);
  p.by_heads = reciprocal(num_heads);
  const dim3 grid((unsigned)(((int64_t)T + p.tokens - 1) / p.tokens),
                  (unsigned)(((int64_t)num_heads + p.heads - 1) / p.heads));
  if (vec)
    rope_kernel<VecUnit><<<grid, kThreads, 0, pa::as_stream(stream)>>>(p);
  else
    rope_kernel<ScalarUnit><<<grid, kThreads, 0, pa::as_stream(stream)>>>(p);
  return pa::launch_status();
}
