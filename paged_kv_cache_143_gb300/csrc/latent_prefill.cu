// latent_prefill.cu — pa_latent_prefill: attention in the expanded form, ragged
// query chunks against the expanded keys and values of their contexts.
//
// Head h of query i scores key n by q_n . k_nope[n][h] + q_r . k_r[n], the
// rotary key k_r shared by the heads, and averages v[n][h]: 192 dims in,
// 128 out. 2 (192 + 128) operations per visible (query, key, head) against 640
// bytes per (key, head) read once per 256 queries: bound by the tensor cores
// from a few hundred queries on.
//
// One CTA = two consecutive tiles (A, B) of 128 queries of one head; both share
// every key tile of 128. All products are full 128 x 128 tcgen05 instructions:
//   warpgroup 0  warp 0, one thread: TMA, the Q tiles once (6 chunks), then 5
//                chunks of 16 KB per key tile (k_nope 2, k_r 1, v 2) into one
//                ring of 8 slots in the order of use. Q takes 96 KB, so two whole
//                stages of K and V (160 KB) would not fit; a ring of chunks lets
//                V(j) arrive as soon as S(j - 1) has read its keys;
//                warp 1, one thread: MMAs in the order PV_A(j-1), S_A(j),
//                PV_B(j-1), S_B(j), one tile's products under the other's
//                softmax. S_t (128 fp32 columns) is overwritten by P_t (bf16), the
//                A operand of O_t += P_t V_j
//   warpgroups 1, 2  softmax of tiles A and B, one query row per thread; O_t is
//                rescaled only when the row's maximum grows by more than 2^8.
// CTAs go out longest first from a host-planned list of (request, tile pair). Where
// those are few, the keys of each are shared out over a cluster of CTAs, which join
// their O, maxima and sums through each other's shared memory: no workspace, and
// every output row still written once. 24 heads, 5 queries on 16000 keys: 258 -> 73 us.
// Long chunks (4 of 1900 to 4096 queries behind up to 16000 keys, 24 heads) take 815 to
// 850 us at 2.07 GHz (1375 to 1318 TFLOP/s) and 866 to 875 for seconds on end, under the
// power cap: a pair of tiles takes 3500 cycles, the softmax chain
// of one 3300 (S and P share TMEM columns), the products of both 2700.
// Every wait is bounded; a timeout sets the error word and the CTA unwinds.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kM = 128, kN = 128;      // queries and keys of a tile
constexpr int kNope = 128, kRope = 64, kV = 128;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;
// Registers: launched with 168 per thread; warpgroup 0 keeps 64, the softmax
// warpgroups raise to 216 (128 * 64 + 256 * 216 <= 384 * 168).
constexpr uint32_t kLaunchRegs = 168, kRegsProducer = 64, kRegsSoftmax = 216;
static_assert(128 * kRegsProducer + 256 * kRegsSoftmax <= kThreads * kLaunchRegs,
              "register split exceeds the registers the block is launched with");

constexpr int kSlot = kN * 128;                        // 128 rows x 64 bf16
constexpr int kQChunks = (kNope + kRope) / 64;         // 3
constexpr int kKChunks = kQChunks, kVChunks = kV / 64; // 3 and 2
constexpr int kTileChunks = kKChunks + kVChunks;
constexpr int kSlots = 8;
constexpr int kOffRing = 2 * kQChunks * kSlot;
constexpr int kOffBars = kOffRing + kSlots * kSlot;
constexpr int kSmem = kOffBars + 1024 + 1024;          // the base is rounded up to 1024 B
static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB per-block limit");

struct Bars {
  uint64_t q_full;
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t final_mma;
  uint32_t tmem;
  int abort;
  int any_cleared;               // some value element was: rows past cleared[dim] get a NaN
  int32_t cleared[kV];           // first key of the request whose element was, by dim
};
static_assert(sizeof(Bars) <= 1024, "the mbarriers overrun their slot");

constexpr int kMaxUnits = 1024;

struct ExpandedParams {
  __nv_bfloat16* out;    // [T][H][128]
  const int32_t* qsl;    // [R+1]
  const int32_t* ksl;    // [R+1]
  int32_t T, Tk, R, H, causal;
  float scale_log2;
  unsigned* err;
  int32_t split;         // CTAs of a unit
  // (request << 16 | last << 15 | tile pair), the most key tiles first; last
  // marks the request's highest pair: grid (H * split, units). n_units == 0: grid
  // (pairs, H, R), split 1.
  int32_t n_units;
  int32_t units[kMaxUnits];
};

// What the CTAs of a cluster leave in shared memory for each other: O of both tiles
// [row][128] in fp32, its 16-byte pieces permuted within a row, then (m, l) of the rows.
constexpr int kOffSums = 2 * kM * kV * 4;
static_assert(kOffSums + 2 * kM * 8 <= kOffBars, "partials overrun the tiles' shared memory");
constexpr int kMaxSplit = 8;           // CTAs of a cluster, the portable limit

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster: what they wrote before it is seen behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of this CTA's shared memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ bool aborted(Bars* b) {
  return *reinterpret_cast<volatile int*>(&b->abort) != 0;
}

__device__ __forceinline__ bool non_finite_pair(uint32_t x) {  // either bf16
  return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
}

// Zeros in the place of the infinities and NaN of one value row, by a warp; `key` is
// its position in the request. Rows that see the key have the NaN put back when they
// are written (0 or NaN times the element is that).
__device__ __forceinline__ void clear_value(uint8_t* const (&chunk)[kVChunks], int row, int32_t key,
                                         Bars* bars) {
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < kVChunks; ++c) {
    uint32_t* w = reinterpret_cast<uint32_t*>(chunk[c] + row * 128) + lane;
    uint32_t x = *w;
    if (!non_finite_pair(x)) continue;
    const int dim = c * 64 + (((lane >> 2) ^ (row & 7)) << 3) + (lane & 3) * 2;
    for (int half = 0; half < 2; ++half) {
      if ((x >> 16 * half & 0x7F80u) != 0x7F80u) continue;
      x &= half ? 0xFFFFu : 0xFFFF0000u;
      atomicMin(&bars->cleared[dim + half], key);
    }
    *w = x;
    *reinterpret_cast<volatile int*>(&bars->any_cleared) = 1;
  }
}

// For a tile in which rows hide keys and score some of them with no number (limit >= 0:
// this thread's row does; it sees the keys below limit): a later key may not be
// finite, and 0 times its value then a NaN. The keys at fault are those that rows with a
// finite query hide and score so; their values, and no others, are cleared. All lanes of
// a warp, before S is overwritten; v is the ring position of the tile's first value chunk.
__device__ __noinline__ bool clear_hidden(uint8_t* smem, Bars* bars, uint32_t tmem_s,
                                          int query, int v, int key0, int limit, int n_kv,
                                          unsigned* err) {
  bool here = mbar_wait(&bars->q_full, 0, err);
  uint8_t* chunk[kVChunks];
#pragma unroll
  for (int c = 0; c < kVChunks; ++c) {
    here = here && mbar_wait(&bars->full[(v + c) % kSlots], ((v + c) / kSlots) & 1, err);
    chunk[c] = smem + kOffRing + ((v + c) % kSlots) * kSlot;
  }
  if (!__all_sync(0xffffffffu, here)) return false;
  bool finite = limit >= 0;
#pragma unroll 1
  for (int i = 0; i < kQChunks * 8; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(smem + query + (i >> 3) * kSlot + (i & 7) * 16);
    if (non_finite_pair(x.x) || non_finite_pair(x.y) || non_finite_pair(x.z) ||
        non_finite_pair(x.w))
      finite = false;
  }
#pragma unroll 1
  for (int c = 0; c < kN / 32; ++c) {
    uint32_t x[32];
    tc::tmem_ld32(tmem_s + c * 32, x);
    tc::tmem_wait_ld();
    uint32_t bad = 0u;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int key = key0 + c * 32 + k;
      if (key >= limit && key < n_kv && !(fabsf(__uint_as_float(x[k])) < INFINITY)) bad |= 1u << k;
    }
    bad = __reduce_or_sync(0xffffffffu, finite ? bad : 0u);
    for (; bad != 0u; bad &= bad - 1) {
      const int n = c * 32 + __ffs(bad) - 1;
      clear_value(chunk, n, key0 + n, bars);
    }
  }
  tc::fence_proxy_async_smem();
  return true;
}

// NaN in the place of the elements of this thread's row (written by it before) that a
// cleared value of a key it sees, one below limit, belongs to: in out, or in the shared
// memory that the CTAs of a cluster join from.
__device__ __noinline__ void put_back(__nv_bfloat16* out, float* piece, int row, int limit,
                                      const Bars* bars) {
#pragma unroll 1
  for (int d = 0; d < kV; ++d) {
    if (limit <= bars->cleared[d]) continue;
    if (out)
      reinterpret_cast<uint16_t*>(out)[d] = 0x7FFFu;
    else
      piece[((d >> 2) ^ (row & 31)) * 4 + (d & 3)] = __uint_as_float(0x7FFFFFFFu);
  }
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_r,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ ExpandedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);

  const bool listed = p.n_units > 0;
  const int unit = listed ? p.units[blockIdx.y] : 0;
  const int r = listed ? unit >> 16 : (int)blockIdx.z;
  const int split = kSplit ? p.split : 1, rank = kSplit ? (int)cluster_rank() : 0;
  const int h = !listed ? blockIdx.y : kSplit ? blockIdx.x / split : blockIdx.x;
  const int q_begin = p.qsl[r], q_len = p.qsl[r + 1] - q_begin;
  const int k_begin = p.ksl[r], k_len = p.ksl[r + 1] - k_begin;
  const bool reporter = threadIdx.x == 0 && h == 0 && rank == 0 && (listed || blockIdx.x == 0);
  if (q_len < 0 || k_len < 0 || q_begin < 0 || k_begin < 0 || q_begin > p.T - q_len ||
      k_begin > p.Tk - k_len) {
    if (reporter) raise_error(p.err, kErrBounds);
    return;
  }
  const int npairs = (q_len + 2 * kM - 1) / (2 * kM);
  int pair;
  if (listed) {
    // the device lengths may disagree with the mirrors that the list came from: rows
    // past the request's last listed pair are an error, a pair past its rows (a padded
    // batch) is nothing to do
    pair = unit & 0x7FFF;
    if ((unit & 0x8000) != 0 && pair < npairs - 1 && reporter) raise_error(p.err, kErrBounds);
    if (pair >= npairs) return;
  } else {
    if (npairs > (int)gridDim.x && reporter) raise_error(p.err, kErrBounds);
    if ((int)blockIdx.x >= npairs) return;
    pair = npairs - 1 - blockIdx.x;  // the longest (latest) pairs start first
  }
  const int P = k_len - q_len;  // key position of query 0 (negative: no key for the first queries)
  int n_kv[2], ntk[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int q0 = (2 * pair + t) * kM;
    const int last = min(q_len, q0 + kM);
    n_kv[t] = q0 >= q_len ? 0 : p.causal ? max(0, min(k_len, P + last)) : k_len;
    ntk[t] = (n_kv[t] + kN - 1) / kN;
  }
  const int n_kv_all = max(n_kv[0], n_kv[1]);
  int j0 = 0;  // this CTA's key tiles: j0 ..; the counts below are its own
  if constexpr (kSplit) {
    const int share = (max(ntk[0], ntk[1]) + split - 1) / split;
    j0 = rank * share;
#pragma unroll
    for (int t = 0; t < 2; ++t) ntk[t] = max(0, min(ntk[t] - j0, share));
  }
  const int ntk_all = max(ntk[0], ntk[1]);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->pv_done[t], 1);
    }
    mbar_init(&bars->final_mma, 1);
    bars->abort = 0;
    bars->any_cleared = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < kV) bars->cleared[threadIdx.x] = INT32_MAX;
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem;  // S_t / P_t at column 128 t, O_t at 256 + 128 t

  // The role branches never merge before the block-wide barrier that each ends with.
  if (warp < 4) {
    tc::regs_dec<kRegsProducer>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------- TMA producer
      tc::prefetch_tensormap(&tmap_q);
      tc::prefetch_tensormap(&tmap_k);
      tc::prefetch_tensormap(&tmap_r);
      tc::prefetch_tensormap(&tmap_v);
      int issued = 0;
      bool ok = true;
      if (ntk_all > 0) {
        const int nq = ntk[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(nq * kQChunks * kSlot));
        for (int t = 0; t < nq; ++t)
          for (int c = 0; c < kQChunks; ++c)
            tc::tma_load_3d(smem + (t * kQChunks + c) * kSlot, &tmap_q, c * 64, h,
                            q_begin + (2 * pair + t) * kM, &bars->q_full);
      }
      for (int j = 0; ok && j < ntk_all; ++j) {
        const int row = k_begin + (j0 + j) * kN;
        for (int c = 0; c < kTileChunks; ++c, ++issued) {
          const int s = issued % kSlots;
          if (issued >= kSlots &&
              (!mbar_wait(&bars->empty[s], (issued / kSlots - 1) & 1, p.err) || aborted(bars))) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + kOffRing + s * kSlot;
          mbar_arrive_expect_tx(&bars->full[s], kSlot);
          if (c < kNope / 64)
            tc::tma_load_3d(dst, &tmap_k, c * 64, h, row, &bars->full[s]);
          else if (c < kKChunks)
            tc::tma_load_2d(dst, &tmap_r, 0, row, &bars->full[s]);
          else
            tc::tma_load_3d(dst, &tmap_v, (c - kKChunks) * 64, h, row, &bars->full[s]);
        }
      }
      if (!ok) bars->abort = 1;
      // every issued copy lands before the CTA may leave
      if (ntk_all > 0) mbar_wait(&bars->q_full, 0, p.err);
      for (int i = max(0, issued - kSlots); i < issued; ++i)
        mbar_wait(&bars->full[i % kSlots], (i / kSlots) & 1, p.err);
    } else if (warp == 1 && tc::elect_one()) {
      // --------------------------------------------------------- MMA issuer
      // Descriptors are bases plus constants: computed anew for every product in
      // a lane of its own they took 100 cycles a product, more than the product.
      constexpr uint32_t idesc_s = tc::idesc_16bit_f32(kM, kN, false, false, false);
      constexpr uint32_t idesc_o = tc::idesc_16bit_f32(kM, kV, false, true, false);
      constexpr uint32_t idesc_h = tc::idesc_16bit_f32(kM, 64, false, true, false);
      const uint64_t q_desc = tc::smem_desc_sw128(smem, 16, 1024);
      const uint64_t k_desc = tc::smem_desc_sw128(smem + kOffRing, 16, 1024);
      const uint64_t v_desc = tc::smem_desc_sw128(smem + kOffRing, kSlot, 1024);
      bool ok = ntk_all == 0 || mbar_wait(&bars->q_full, 0, p.err);
      auto landed = [&](int i) {
        return mbar_wait(&bars->full[i % kSlots], (i / kSlots) & 1, p.err);
      };
      auto issue_s = [&](int t, int j) -> bool {
        const uint64_t qt = tc::desc_at(q_desc, t * kQChunks * kSlot);
        const uint32_t d = tmem + t * kN;
#pragma unroll
        for (int c = 0; c < kKChunks; ++c) {
          const int i = j * kTileChunks + c;
          if (!landed(i)) return false;
          tc::fence_after_sync();
          const uint64_t ks = tc::desc_at(k_desc, (i % kSlots) * kSlot);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_bf16_ss(d, tc::desc_at(qt, c * kSlot + k * 32), tc::desc_at(ks, k * 32),
                            idesc_s, c > 0 || k > 0);
        }
        tc::mma_commit(&bars->s_full[t]);
        return true;
      };
      auto issue_pv = [&](int t, int j) -> bool {
        const int v = j * kTileChunks + kKChunks;
        if (!mbar_wait(&bars->p_full[t], j & 1, p.err) || !landed(v) || !landed(v + 1) ||
            aborted(bars))
          return false;
        tc::fence_after_sync();
        const uint32_t d = tmem + 2 * kN + t * kV, pt = tmem + t * kN;
        const uint64_t v0 = tc::desc_at(v_desc, (v % kSlots) * kSlot);
        // the two 64-column chunks of V may wrap around the ring: then each is a
        // product of its own (64 columns of O)
        if (v % kSlots != kSlots - 1) {
#pragma unroll
          for (int k = 0; k < kN / 16; ++k)
            tc::mma_bf16_ts(d, pt + k * 8, tc::desc_at(v0, k * 16 * 128), idesc_o, j > 0 || k > 0);
        } else {
#pragma unroll
          for (int c = 0; c < kVChunks; ++c)
#pragma unroll
            for (int k = 0; k < kN / 16; ++k)
              tc::mma_bf16_ts(d + c * 64, pt + k * 8,
                              tc::desc_at(c ? v_desc : v0, k * 16 * 128), idesc_h,
                              j > 0 || k > 0);
        }
        tc::mma_commit(&bars->pv_done[t]);
        return true;
      };
      auto release = [&](int j, int c0, int c1) {
        for (int c = c0; c < c1; ++c) tc::mma_commit(&bars->empty[(j * kTileChunks + c) % kSlots]);
      };
      for (int j = 0; ok && j < ntk_all; ++j) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // PV_t(j-1) reads P_t out of the S_t columns before S_t(j) overwrites them
          if (ok && j >= 1 && j - 1 < ntk[t] && !issue_pv(t, j - 1)) ok = false;
          if (t == 1 && ok && j >= 1) release(j - 1, kKChunks, kTileChunks);
          if (ok && j < ntk[t] && !issue_s(t, j)) ok = false;
        }
        if (ok) release(j, 0, kKChunks);
      }
      for (int t = 0; t < 2 && ok && ntk_all > 0; ++t)
        if (ntk_all - 1 < ntk[t] && !issue_pv(t, ntk_all - 1)) ok = false;
      if (!ok) bars->abort = 1;
      tc::mma_commit(&bars->final_mma);
      mbar_wait(&bars->final_mma, 0, p.err);
    }
    __syncwarp();
    tc::fence_before_sync();
    named_bar_sync(0, kThreads);
    if constexpr (kSplit) cluster_sync();
    if (warp == 1) {
      tc::fence_after_sync();
      tc::tmem_dealloc(tmem, kTmemCols);
    }
    if constexpr (kSplit) cluster_sync();
  } else {
    tc::regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------- softmax
    const int t = warp >= 8 ? 1 : 0;
    const int my_ntk = t ? ntk[1] : ntk[0];
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tmem_s = tmem + t * kN + lanes, tmem_o = tmem + 2 * kN + t * kV + lanes;
    const int tok = (2 * pair + t) * kM + row;
    const bool valid = tok < q_len;
    const int limit = !valid ? 0 : p.causal ? max(0, min(P + tok + 1, k_len)) : k_len;
    // keys that every row of the warp sees (rows past the chunk are never looked at)
    const int least = __reduce_min_sync(0xffffffffu, valid ? limit : INT32_MAX);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; ok && j < my_ntk; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[t], j & 1, p.err))) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      uint32_t sr[kN];
#pragma unroll
      for (int c = 0; c < kN / 32; ++c)
        tc::tmem_ld32(tmem_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + c * 32));
      tc::tmem_wait_ld();
      float* s = reinterpret_cast<float*>(sr);
      const int key0 = (j0 + j) * kN;
      if (key0 + kN > least) {
        // Scores that are no numbers in a tile where this row hides keys of its request
        // (32 at a time up to the last such key; past it lies anything)
        uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int k = 0; k < kN; k += 32)
          if (key0 + k < n_kv_all) {
#pragma unroll
            for (int u = 0; u < 16; ++u)
              sum2[u & 3] = f2_add(sum2[u & 3], f2_pack(s[k + 2 * u], s[k + 2 * u + 1]));
          }
        float lo, hi;
        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), lo, hi);
        const bool odd = limit > 0 && limit < min(key0 + kN, n_kv_all) &&
                         !(fabsf(lo + hi) < INFINITY);
        if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {  // rare
          if (!__all_sync(0xffffffffu, clear_hidden(smem, bars, tmem_s,
                                                    t * kQChunks * kSlot + row * 128,
                                                    j * kTileChunks + kKChunks, key0,
                                                    odd ? limit : -1, n_kv_all, p.err))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < kN / 32; ++c)
            tc::tmem_ld32(tmem_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + c * 32));
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < kN; ++k)
          if (key0 + k >= limit) s[k] = -INFINITY;
      }
      // eight partial maxima keep the reduction off one dependency chain
      float mx[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        mx[u] = fmaxf(s[u], s[u + 8]);
#pragma unroll
        for (int i = 2; i < kN / 8; i += 2) mx[u] = fmax3(mx[u], s[u + 8 * i], s[u + 8 * i + 8]);
      }
      const float mt = p.scale_log2 * fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                            fmaxf(mx[6], mx[7]));
      float alpha = 1.f;
      bool rescale = false;
      if (m_run == -INFINITY) {
        m_run = mt;
      } else if (mt > m_run + kRescaleLog2) {
        alpha = ex2_ftz(m_run - mt);
        m_run = mt;
        rescale = true;
      }
      const float neg = m_run == -INFINITY ? 0.f : -m_run;
      const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(neg, neg);
      uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int k = 0; k < kN; k += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float a, b;
          f2_unpack(f2_fma(f2_pack(s[k + 2 * u], s[k + 2 * u + 1]), sc2, nm2), a, b);
          s[k + 2 * u] = ex2_ftz(a);
          s[k + 2 * u + 1] = ex2_ftz(b);
          sum2[u] = f2_add(sum2[u], f2_pack(s[k + 2 * u], s[k + 2 * u + 1]));
        }
      float lo, hi;
      f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), lo, hi);
      l_run = l_run * alpha + (lo + hi);

      if (__any_sync(0xffffffffu, rescale)) {
        // (PV_t(j-1) precedes S_t(j) in the MMA stream: this wait only orders
        // the TMEM accesses)
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[t], (j - 1) & 1, p.err))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < kV / 32; ++c) {
          uint32_t o[32];
          tc::tmem_ld32(tmem_o + c * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tc::tmem_st32(tmem_o + c * 32, o);
        }
      }
#pragma unroll
      for (int c = 0; c < kN / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          __nv_bfloat162 x = __floats2bfloat162_rn(s[c * 64 + 2 * k], s[c * 64 + 2 * k + 1]);
          w[k] = *reinterpret_cast<uint32_t*>(&x);
        }
        tc::tmem_st32(tmem_s + c * 32, w);
      }
      tc::tmem_wait_st();
      if (j == ntk_all - 1 && key0 + kN > n_kv_all) {
        // value rows past the last visible key (another request's, or past
        // the array) are zeroed, so that P = 0 never meets a NaN
        const int v = j * kTileChunks + kKChunks;
        bool here = true;
#pragma unroll
        for (int c = 0; c < kVChunks; ++c)
          here = here && mbar_wait(&bars->full[(v + c) % kSlots], ((v + c) / kSlots) & 1, p.err);
        if (!__all_sync(0xffffffffu, here)) {
          ok = false;
          break;
        }
        if (key0 + row >= n_kv_all) {
#pragma unroll
          for (int c = 0; c < kVChunks; ++c)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(smem + kOffRing + ((v + c) % kSlots) * kSlot + row * 128 +
                                        q * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full[t]);
    }
    if (ok && my_ntk > 0 &&
        !__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[t], (my_ntk - 1) & 1, p.err)))
      ok = false;
    if (!ok) bars->abort = 1;
    // (all clears are done by now: those that matter to a tile precede its last product)
    auto any_cleared = [&] {
      return __builtin_expect(*reinterpret_cast<volatile int*>(&bars->any_cleared), 0) != 0;
    };
    if constexpr (kSplit) {
      // both tiles' products are done and every copy has landed: Q and the ring
      // make room for the partials
      tc::fence_before_sync();
      named_bar_sync(0, kThreads);
      tc::fence_after_sync();
      float2* sums = reinterpret_cast<float2*>(smem + kOffSums);
      // (a sum of -1: the row sees no key of this CTA's)
      sums[t * kM + row] = make_float2(m_run, my_ntk > 0 && limit > j0 * kN ? l_run : -1.f);
#pragma unroll 1
      for (int c = 0; c < kV / 32; ++c) {
        uint32_t o[32];
        if (my_ntk > 0) {
          tc::tmem_ld32(tmem_o + c * 32, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (my_ntk > 0)
            *reinterpret_cast<uint4*>(smem + (t * kM + row) * kV * 4 +
                                      (((c * 8 + q) ^ (row & 31)) << 4)) =
                make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      }
      if (any_cleared() && my_ntk > 0)
        put_back(nullptr, reinterpret_cast<float*>(smem) + (t * kM + row) * kV, row, limit, bars);
      tc::fence_before_sync();
      cluster_sync();
      // a warp joins a row: o = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k
      const int rows = 2 * kM / split;
#pragma unroll 1
      for (int i = warp - 4; i < rows; i += 8) {
        const int at = rank * rows + i, tok_i = 2 * pair * kM + at;
        if (tok_i >= q_len) break;
        const uint8_t* piece = smem + at * kV * 4 + ((lane ^ (at & 31)) << 4);
        float2 ml[kMaxSplit];
        float4 x[kMaxSplit];
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
          ml[k] = make_float2(-INFINITY, -1.f);
          if (k < split) {
            ml[k] = ld_cluster2(in_cta(sums + at, k));
            x[k] = ld_cluster4(in_cta(piece, k));  // (not used where the sum is -1)
          }
        }
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (!(ml[k].y < 0.f)) top = fmaxf(top, ml[k].x);  // (a NaN sum counts)
        bool some = false;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
          if (ml[k].y < 0.f) continue;
          some = true;
          // (scores of -inf alone weigh 0, which O may make a NaN)
          const float w = ml[k].x == -INFINITY ? 0.f : ex2_ftz(ml[k].x - top);
          sum = fmaf(w, ml[k].y, sum);
          o.x = fmaf(w, x[k].x, o.x);
          o.y = fmaf(w, x[k].y, o.y);
          o.z = fmaf(w, x[k].z, o.z);
          o.w = fmaf(w, x[k].w, o.w);
        }
        // zero without a visible key; NaN where every score is -inf
        const float inv = some ? 1.f / sum : 0.f;
        __nv_bfloat162 lo2 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(p.out + ((int64_t)(q_begin + tok_i) * p.H + h) * kV + lane * 4) =
            make_uint2(*reinterpret_cast<uint32_t*>(&lo2), *reinterpret_cast<uint32_t*>(&hi2));
      }
      cluster_sync();  // no CTA leaves while another reads it
      return;
    }
    if (ok && !aborted(bars)) {
      tc::fence_after_sync();
      // a row without a visible key is zero; one whose scores are all -inf is NaN (its
      // sum is 0)
      const bool some = limit > 0;
      const float inv = some ? 1.f / l_run : 0.f;
      __nv_bfloat16* orow = p.out + ((int64_t)(q_begin + tok) * p.H + h) * kV;
#pragma unroll 1
      for (int c = 0; c < kV / 32; ++c) {
        uint32_t o[32];
        if (my_ntk > 0) {
          tc::tmem_ld32(tmem_o + c * 32, o);
          tc::tmem_wait_ld();
        }
        if (valid) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[q * 8 + 2 * e]) * inv,
                                                       __uint_as_float(o[q * 8 + 2 * e + 1]) * inv);
              w[e] = some ? *reinterpret_cast<uint32_t*>(&x) : 0u;
            }
            *reinterpret_cast<uint4*>(orow + c * 32 + q * 8) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (any_cleared() && valid) put_back(orow, nullptr, row, limit, bars);
    }
    tc::fence_before_sync();
    named_bar_sync(0, kThreads);
  }
}

// ----------------------------------------------------------------- host side

// Rows [tokens][heads][cols] with strides in elements: box = 64 columns of one
// head of 128 tokens, 128-byte swizzled.
bool encode_heads(CUtensorMap* m, const void* base, int cols, int heads, int64_t tokens,
                  int64_t token_stride, int64_t head_stride) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, 1, kN};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* m, const void* base, int64_t tokens, int64_t token_stride) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {kRope, (cuuint64_t)tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)token_stride * 2};
  const cuuint32_t box[2] = {64, kN};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Writes the (request, tile pair) units, the most key tiles first, and returns
// their number; -1 if there are more than the list holds. most: key tiles of the first.
int plan_units(const int32_t* qsl, const int32_t* ksl, int R, bool causal, int32_t* units,
               int* most) {
  struct Unit {
    int32_t steps, id;
  };
  Unit list[kMaxUnits];
  int n = 0;
  for (int r = 0; r < R; ++r) {
    const int q_len = qsl[r + 1] - qsl[r], k_len = ksl[r + 1] - ksl[r];
    const int npairs = (int)(((int64_t)q_len + 2 * kM - 1) / (2 * kM));
    if (npairs > kMaxUnits - n) return -1;
    for (int i = npairs - 1; i >= 0; --i) {
      const int64_t last = std::min<int64_t>(q_len, (int64_t)(i + 1) * 2 * kM);
      const int64_t n_kv = causal ? std::max<int64_t>(0, k_len - q_len + last) : k_len;
      list[n++] = Unit{(int32_t)((n_kv + kN - 1) / kN),
                       r << 16 | (i == npairs - 1 ? 0x8000 : 0) | i};
    }
  }
  std::stable_sort(list, list + n, [](const Unit& a, const Unit& b) { return a.steps > b.steps; });
  for (int i = 0; i < n; ++i) units[i] = list[i].id;
  *most = n > 0 ? list[0].steps : 0;
  return n;
}

// Once per device. The register split assumes that the block is launched with
// kLaunchRegs per thread: a build that allocated fewer is refused.
template <bool kSplit>
bool prepare_kernel() {
  cudaFuncAttributes fa;
  return cudaFuncSetAttribute(latent_prefill_kernel<kSplit>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmem) == cudaSuccess &&
         cudaFuncGetAttributes(&fa, latent_prefill_kernel<kSplit>) == cudaSuccess &&
         fa.numRegs >= (int)kLaunchRegs;
}

cudaLaunchConfig_t cluster_config(int split, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = split;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of `split` (2, 4, 8) CTAs that the current device runs at once (76, 36 and
// 15 of the 152 SMs' 225 KB each: a cluster lies within a GPC); 0 if that is unknown.
int resident_clusters(int split) {
  static std::atomic<int> known[64][kMaxSplit + 1];  // plus one; 0: not asked yet
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][split].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = cluster_config(split, attr);
    if (!prepare_kernel<true>() ||
        cudaOccupancyMaxActiveClusters(&n, latent_prefill_kernel<true>, &cfg) != cudaSuccess ||
        n < 0)
      n = 0;
    known[dev][split].store(++n, std::memory_order_relaxed);
  }
  return n - 1;
}

bool stride_ok(int64_t s, int64_t least) {
  return s >= least && s % 8 == 0 && s < ((int64_t)1 << 38);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_latent_prefill(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_nope,
    int64_t k_token_stride, int64_t k_head_stride, const void* k_rope, int64_t rope_token_stride,
    const void* v, int64_t v_token_stride, int64_t v_head_stride, void* out,
    const int32_t* query_start_loc, const int32_t* kv_start_loc, const int32_t* qsl_host,
    const int32_t* ksl_host, int32_t num_reqs, int32_t num_tokens, int32_t num_kv_tokens,
    int32_t num_heads, int32_t nope_dim, int32_t rope_dim, int32_t v_dim, float scale,
    int32_t causal, pa_stream_t stream) {
  using namespace pa;
  const int R = num_reqs, T = num_tokens, Tk = num_kv_tokens, H = num_heads;
  if (R < 0 || T < 0 || Tk < 0 || H <= 0) return PA_ERR_INVALID;
  if (nope_dim != kNope || rope_dim != kRope || v_dim != kV) return PA_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  if (causal != 0 && causal != 1) return PA_ERR_INVALID;
  if (R == 0) return T == 0 && Tk == 0 ? PA_OK : PA_ERR_INVALID;
  if (!qsl_host || !ksl_host || !query_start_loc || !kv_start_loc) return PA_ERR_INVALID;
  if (qsl_host[0] != 0 || qsl_host[R] != T || ksl_host[0] != 0 || ksl_host[R] != Tk)
    return PA_ERR_INVALID;
  int max_pairs = 0;
  for (int r = 0; r < R; ++r) {
    const int ql = qsl_host[r + 1] - qsl_host[r];
    if (ql < 0 || ksl_host[r + 1] - ksl_host[r] < 0) return PA_ERR_INVALID;
    max_pairs = std::max(max_pairs, (int)(((int64_t)ql + 2 * kM - 1) / (2 * kM)));
  }
  if (T == 0) return PA_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return PA_ERR_INVALID;
  const int64_t qt = T > 1 ? q_token_stride : kNope + kRope;
  const int64_t qh = H > 1 ? q_head_stride : kNope + kRope;
  if (!stride_ok(qt, 1) || !stride_ok(qh, 1)) return PA_ERR_INVALID;
  // (the stride of a dimension of one entry is never used)
  const int64_t kt = Tk > 1 ? k_token_stride : kNope, kh = H > 1 ? k_head_stride : kNope;
  const int64_t vt = Tk > 1 ? v_token_stride : kV, vh = H > 1 ? v_head_stride : kV;
  const int64_t rt = Tk > 1 ? rope_token_stride : kRope;
  if (Tk > 0) {
    if (!k_nope || !k_rope || !v || !aligned16(k_nope) || !aligned16(k_rope) || !aligned16(v))
      return PA_ERR_INVALID;
    if (!stride_ok(kt, 1) || !stride_ok(kh, 1) || !stride_ok(vt, 1) || !stride_ok(vh, 1) ||
        !stride_ok(rt, 1))
      return PA_ERR_INVALID;
  }
  if (R > 32767) return PA_ERR_UNSUPPORTED;
  unsigned* err = error_word();
  if (!err) return PA_ERR_CUDA;
  ExpandedParams p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.qsl = query_start_loc;
  p.ksl = kv_start_loc;
  p.T = T;
  p.Tk = Tk;
  p.R = R;
  p.H = H;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = err;
  int most = 0;
  p.n_units = std::max(0, plan_units(qsl_host, ksl_host, R, causal != 0, p.units, &most));
  // Few units: each is split along its keys over a cluster of 2, 4 or 8 CTAs, as far
  // as the GPU holds all clusters at once. The join costs about 3 key tiles, so the
  // longest unit has to become 4 shorter, and 2 by every doubling (8 heads: 1000
  // queries on 1000 keys 33 us whole, 25 in four; 300 on 400, 23 whole, 28 in two).
  p.split = 1;
  auto tiles = [&](int split) { return (most + split - 1) / split; };
  while (p.n_units > 0 && p.split < kMaxSplit && tiles(p.split) - tiles(2 * p.split) >= 2 &&
         (int64_t)H * p.n_units <= resident_clusters(2 * p.split))
    p.split *= 2;
  if (tiles(1) - tiles(p.split) < 4) p.split = 1;
  const dim3 grid = p.n_units > 0 ? dim3(H * p.split, p.n_units, 1) : dim3(max_pairs, H, R);
  if (grid.y > 65535u || grid.z > 65535u) return PA_ERR_UNSUPPORTED;
  // an empty key side has nothing to map: the queries' own map stands in (no
  // copy is issued from it)
  CUtensorMap tq, tk, tr, tv;
  if (!encode_heads(&tq, q, kNope + kRope, H, T, qt, qh)) return PA_ERR_CUDA;
  if (Tk == 0) {
    tk = tr = tv = tq;
  } else if (!encode_heads(&tk, k_nope, kNope, H, Tk, kt, kh) ||
             !encode_rows(&tr, k_rope, Tk, rt) ||
             !encode_heads(&tv, v, kV, H, Tk, vt, vh)) {
    return PA_ERR_CUDA;
  }
  const cudaStream_t s = as_stream(stream);
  if (p.split == 1) {
    static OncePerDevice attribute;
    if (!attribute.done(prepare_kernel<false>)) return PA_ERR_CUDA;
    latent_prefill_kernel<false><<<grid, kThreads, kSmem, s>>>(tq, tk, tr, tv, p);
    return launch_status();
  }
  static OncePerDevice attribute;
  if (!attribute.done(prepare_kernel<true>)) return PA_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = cluster_config(p.split, attr);
  cfg.gridDim = grid;
  cfg.stream = s;
  if (cudaLaunchKernelEx(&cfg, latent_prefill_kernel<true>, tq, tk, tr, tv, p) != cudaSuccess)
    return PA_ERR_CUDA;
  count_launches(1);
  return PA_OK;
}
