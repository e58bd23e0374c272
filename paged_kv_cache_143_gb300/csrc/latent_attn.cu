// latent_attn.cu — pa_latent_forward: attention in the absorbed form over the
// paged latent cache, decode tokens and chunks alike.
//
// Every query row (token, head) of a request scores the same keys [c ; k_r] and
// averages the same values c, so one pass over the request's cells serves all
// its rows: s = scale * (q_c . c + q_r . k_r), o = softmax(s) c, the softmax
// running over key tiles with a reference maximum and sum per row.
//
// What bounds it: a cell is (L + 64) * 2 bytes and each row spends 2 (2 L + 64)
// operations on it; up to about 128 rows per request that is less tensor time
// than the cell takes from HBM, so the design is laid out for streaming.
//
// One CTA per SM walks an equal share of all (row tile, 64-key tile) pairs
// (pa::LatentParams). Both products run on the 5th-generation tensor cores:
//   S [64 rows x 64 keys] = Q K^T     Q and the cells K-major in shared memory
//   O^T [L x NR]        += c^T P^T    the same cells read again, MN-major, as
//                                     the A operand; P from shared memory
// O is kept transposed (lane = latent dim, column = row) because a row of O is
// L fp32 values: NR x 512 of them as [dim][row] take 4 NR TMEM columns, and the
// products stay full 128-row instructions for few query rows, where rows
// down the lanes would leave most of the tensor core (and 16 of every 32 lanes)
// idle. NR is 16, 32 or 64.
//   warp 0      TMA producer: the Q tile, then per key tile one box per physical
//               block and 64-column chunk into a ring of stages
//   warp 1      TMEM, and one thread that issues the MMAs: S(j + 1) goes in
//               before PV(j), so the tensor core works while softmax(j) does
//   warps 4-7   softmax of 16 rows each (S read as 16 x 256-bit fragments: a row
//               in four lanes), P written by stmatrix; then the output
// Every wait is bounded; a timeout sets the error word and the CTA unwinds.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "latent_attn.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kRope = 64;
constexpr int KT = kLatentKeys;
constexpr int kChunk = KT * 128;   // one 64-column bf16 chunk of a key tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;   // S buffers at columns 256, 320
constexpr float kRescaleLog2 = 8.f;

template <int L, int NR>
struct Smem {
  static constexpr int kChunks = L / 64 + 1;          // the last one is the rotary part
  static constexpr int kQBytes = kChunks * NR * 128;
  static constexpr int kStage = kChunks * kChunk;
  static constexpr int kPBytes = NR * 128;
  static constexpr int kTail = 2048;                  // barriers and row statistics
  static constexpr int kStages = (232448 - 1024 - kTail - kQBytes - kPBytes) / kStage;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffP = kOffK + kStages * kStage;
  static constexpr int kOffTail = kOffP + kPBytes;
  static constexpr int kAlloc = kOffTail + kTail + 1024;  // the base is rounded up to 1024 B
  static_assert(kStages >= 2, "needs two key tiles in flight");
  static_assert(kAlloc <= 232448, "dynamic shared memory above the 227 KB per-block limit");
  static_assert(kOffK % 1024 == 0 && kOffP % 1024 == 0, "swizzled tiles start on 1024 bytes");
  // S always reads 64 rows of Q: the rows past NR are whatever follows in
  // shared memory (their scores are never looked at)
  static_assert(kQBytes + (64 - NR) * 128 <= kAlloc - 1024, "Q over-read leaves the allocation");
};

constexpr int kMaxStages = 5;
struct Tail {
  uint64_t q_full, q_empty;
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t s_full[2];
  uint64_t p_full, pv_done, o_empty, final_mma;
  float alpha[2][kLatentRows];
  float l[kLatentRows];
  int fail[3];         // a softmax warp gave up: tiles by parity, then outputs
  int64_t warp_sum[kThreads / 32];
  int64_t base;        // flat start of the request that holds the CTA's first tile
  int32_t req;         // that request
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail) <= 2048, "Tail overruns its slot");

__device__ __forceinline__ bool aborted(Tail* t) {
  return *reinterpret_cast<volatile int*>(&t->abort) != 0;
}

// The softmax warps meet at named barriers, so they must leave together: one
// that gave up (bad) says so before the barrier, and all read it after. The
// flag read behind one barrier is not written again before the next.
__device__ __forceinline__ bool agreed_to_stop(Tail* t, int which) {
  return *reinterpret_cast<volatile int*>(&t->fail[which]) != 0;
}

// 16 lanes x 64 columns as mma-style fragments: of each 8-column group i,
// r[4 i], r[4 i + 1] are columns 2 (lane % 4), + 1 of row lane / 4, and
// r[4 i + 2], r[4 i + 3] those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void stmatrix_x4(void* row, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   smem_u32(row)),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// ------------------------------------------------------------ the flat space

struct Request {
  int32_t q_begin, q_len, seq, tiles, keys;  // row tiles, key tiles
  int64_t weight;                            // tiles * keys; 0 for one without work
};

// Reads request r; one whose device entries do not fit the buffers has no
// work (and is reported once).
template <int NR>
__device__ __forceinline__ Request load_request(const LatentParams& p, int r, bool report) {
  Request q{};
  q.q_begin = __ldg(p.qsl + r);
  q.q_len = __ldg(p.qsl + r + 1) - q.q_begin;
  q.seq = __ldg(p.seq_lens + r);
  if (q.q_len == 0) return q;
  if (q.q_len < 0 || q.q_begin < 0 || q.q_begin > p.T - q.q_len || q.seq < q.q_len ||
      (int64_t)q.seq > (int64_t)p.max_blocks * p.B) {
    if (report) raise_error(p.err, kErrBounds);
    return q;
  }
  q.tiles = (int)(((int64_t)q.q_len * p.Hq + NR - 1) / NR);
  q.keys = (q.seq + KT - 1) / KT;
  q.weight = (int64_t)q.tiles * q.keys;
  return q;
}

// A CTA's part of one unit: key tiles [k0, k1) of row tile `tile` of request r.
struct Piece {
  int32_t r, tile, k0, k1;
  int32_t n_keys;      // keys any row of the tile sees (k1 is cut to it)
  int32_t rows;        // valid query rows of the tile
  int32_t slot;        // partial slot 0 / 1 of the CTA, or -1: the whole unit
};

template <int NR>
struct Walk {
  int64_t pos, end, base;
  int r;
  bool loaded;
  Request q;

  __device__ Walk(const Tail* t, int64_t begin, int64_t stop)
      : pos(begin), end(stop), base(t->base), r(t->req), loaded(false), q{} {}

  __device__ bool next(const LatentParams& p, Piece& out) {
    if (pos >= end) return false;
    if (!loaded) {
      q = load_request<NR>(p, r, false);
      loaded = true;
    }
    while (pos >= base + q.weight) {
      base += q.weight;
      if (++r >= p.R) return false;
      q = load_request<NR>(p, r, false);
    }
    const int64_t off = pos - base;
    out.r = r;
    out.tile = (int)(off / q.keys);
    out.k0 = (int)(off - (int64_t)out.tile * q.keys);
    const int64_t left = end - pos;
    const int k1 = left < q.keys - out.k0 ? out.k0 + (int)left : q.keys;
    pos += k1 - out.k0;
    out.slot = out.k0 > 0 ? 0 : k1 < q.keys ? 1 : -1;
    const int64_t row0 = (int64_t)out.tile * NR;
    const int64_t left_rows = (int64_t)q.q_len * p.Hq - row0;
    out.rows = left_rows < NR ? (int)left_rows : NR;
    const int last_tok = (int)((row0 + out.rows - 1) / p.Hq);
    out.n_keys = p.causal ? q.seq - q.q_len + last_tok + 1 : q.seq;
    out.k1 = min(k1, (out.n_keys + KT - 1) / KT);
    return true;
  }
};

template <int L, int NR>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_c,
                       const __grid_constant__ CUtensorMap tmap_r, const LatentParams p) {
  using S = Smem<L, NR>;
  constexpr int kStages = S::kStages;
  static_assert(kStages <= kMaxStages, "");
  constexpr int kBlocks = L / 128;  // 128-dim blocks of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + S::kOffTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  launch_dependents();  // the join that follows may be scheduled now

  // ---- this CTA's range: W, then the request that holds tile cta * Q
  if (warp == 1) {
    tc::tmem_alloc(&tail->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    mbar_init(&tail->q_full, 1);
    mbar_init(&tail->q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&tail->k_full[s], 1);
      mbar_init(&tail->k_empty[s], 1);
    }
    mbar_init(&tail->s_full[0], 1);
    mbar_init(&tail->s_full[1], 1);
    mbar_init(&tail->p_full, 4);   // one arrival per softmax warp
    mbar_init(&tail->pv_done, 1);
    mbar_init(&tail->o_empty, 4);
    mbar_init(&tail->final_mma, 1);
    tail->abort = 0;
    tail->fail[0] = tail->fail[1] = tail->fail[2] = 0;
    tail->req = p.R;
    tail->base = 0;
    fence_mbar_init();
  }
  // running sum over the requests, kThreads at a time (one step up to 256)
  auto scan = [&](int64_t w, int64_t& total) -> int64_t {  // exclusive sum of w
    int64_t x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tail->warp_sum[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      const int64_t s = tail->warp_sum[i];
      if (i < warp) before += s;
      total += s;
    }
    return before + x - w;
  };
  int64_t W = 0, kept_w = 0, kept_before = 0;
  for (int r0 = 0; r0 < p.R; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    kept_w = r < p.R ? load_request<NR>(p, r, cta == 0).weight : 0;
    int64_t total;
    kept_before = W + scan(kept_w, total);
    W += total;
  }
  const int64_t Q = (W + gridDim.x - 1) / gridDim.x;
  const int64_t begin = min(W, cta * Q), end = min(W, begin + Q);
  if (p.R > kThreads) {  // the sums of all but the last step are taken again
    int64_t sum = 0;
    for (int r0 = 0; r0 < p.R; r0 += kThreads) {
      const int r = r0 + threadIdx.x;
      const int64_t w = r < p.R ? load_request<NR>(p, r, false).weight : 0;
      int64_t total;
      const int64_t before = sum + scan(w, total);
      sum += total;
      if (begin >= before && begin < before + w) {
        tail->req = r;
        tail->base = before;
      }
    }
  } else if (begin >= kept_before && begin < kept_before + kept_w) {
    tail->req = threadIdx.x;
    tail->base = kept_before;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tail->tmem;
  if (threadIdx.x == 0) {
    // the unit cut at this CTA's start, for the join: handled at its first cut
    LatentJoin j{};
    if (begin < end) {
      const Request q = load_request<NR>(p, tail->req, false);
      const int64_t tile = (begin - tail->base) / q.keys;
      const int64_t a = tail->base + tile * q.keys;  // the unit's start
      if (begin > a && a / Q + 1 == cta) {
        const int64_t rows = (int64_t)q.q_len * p.Hq - tile * NR;
        j.rows = (int32_t)min(rows, (int64_t)NR);
        j.last = (int32_t)((a + q.keys - 1) / Q);
        j.out_row = (int64_t)q.q_begin * p.Hq + tile * NR;
      }
    }
    p.joins[cta] = j;
  }

  if (begin < end) {
    if (warp == 0) {
      // --------------------------------------------------------- TMA producer
      const unsigned full = 0xffffffffu;
      if (lane == 0) {
        tc::prefetch_tensormap(&tmap_q);
        tc::prefetch_tensormap(&tmap_c);
        tc::prefetch_tensormap(&tmap_r);
      }
      const int bpt = KT / p.B;  // blocks per key tile: 4, 2 or 1
      Walk<NR> walk(tail, begin, end);
      Piece pc;
      int g = 0, pieces = 0;     // key tiles and pieces so far
      bool ok = true;
      while (ok && walk.next(p, pc)) {
        if (pc.k0 >= pc.k1) continue;  // no row of the tile sees these keys
        if (pieces > 0) {
          if (lane == 0) ok = mbar_wait(&tail->q_empty, (pieces - 1) & 1, p.err);
          ok = __shfl_sync(full, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&tail->q_full, S::kQBytes);
        __syncwarp();
        const int row = walk.q.q_begin * p.Hq + pc.tile * NR;
        if (lane < S::kChunks)
          tc::tma_load_2d(smem + lane * NR * 128, &tmap_q, lane * 64, row, &tail->q_full);
        ++pieces;
        const int32_t* table = p.block_tables + (int64_t)pc.r * p.max_blocks;
        auto fetch = [&](int j) -> int {  // block `lane` of key tile j
          const int lb = j * bpt + lane;
          return (j < pc.k1 && lane < bpt && (int64_t)lb * p.B < pc.n_keys) ? __ldg(table + lb) : 0;
        };
        int ids = fetch(pc.k0);
        for (int j = pc.k0; j < pc.k1; ++j, ++g) {
          const int next = fetch(j + 1);
          const int st = g % kStages;
          int nload = 0;
          while (nload < bpt && (j * bpt + nload) * p.B < pc.n_keys) ++nload;
          const bool bad = lane < nload && (ids < 0 || ids >= p.num_blocks);
          if (__any_sync(full, bad) && lane == 0) raise_error(p.err, kErrBounds);
          const int blk_lane = bad ? 0 : ids;  // a valid block; the output is then unspecified
          if (lane == 0 && g >= kStages)
            ok = mbar_wait(&tail->k_empty[st], (g / kStages - 1) & 1, p.err);
          if (!__shfl_sync(full, ok ? 1 : 0, 0) || aborted(tail)) {
            ok = false;
            break;
          }
          uint8_t* stage = smem + S::kOffK + st * S::kStage;
          if (lane == 0)
            mbar_arrive_expect_tx(&tail->k_full[st], (uint32_t)(nload * p.B * 128 * S::kChunks));
          __syncwarp();
          for (int i0 = 0; i0 < nload * S::kChunks; i0 += 32) {
            const int i = i0 + lane;
            const int b = i / S::kChunks, c = i - b * S::kChunks;
            const int y = __shfl_sync(full, blk_lane, b & 3) * p.B;
            if (b < nload) {
              uint8_t* dst = stage + c * kChunk + b * p.B * 128;
              if (c < L / 64)
                tc::tma_load_2d(dst, &tmap_c, c * 64, y, &tail->k_full[st]);
              else
                tc::tma_load_2d(dst, &tmap_r, 0, y, &tail->k_full[st]);
            }
          }
          ids = next;
        }
      }
      // every issued copy lands before the CTA may leave
      if (lane == 0) {
        if (!ok) tail->abort = 1;
        if (pieces > 0) mbar_wait(&tail->q_full, (pieces - 1) & 1, p.err);
        for (int i = max(0, g - kStages); i < g; ++i)
          mbar_wait(&tail->k_full[i % kStages], (i / kStages) & 1, p.err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc_s = tc::idesc_16bit_f32(64, KT, false, false, false);
        constexpr uint32_t idesc_o = tc::idesc_16bit_f32(128, NR, true, false, false);
        const uint8_t* ps = smem + S::kOffP;
        Walk<NR> walk(tail, begin, end);
        Piece pc;
        int g = 0, pieces = 0;
        bool ok = true;
        auto issue_s = [&](int i, bool last) -> bool {  // S of the CTA's key tile i
          const int st = i % kStages;
          if (!mbar_wait(&tail->k_full[st], (i / kStages) & 1, p.err) || aborted(tail))
            return false;
          tc::fence_after_sync();
          const uint8_t* ks = smem + S::kOffK + st * S::kStage;
#pragma unroll
          for (int k = 0; k < S::kChunks * 4; ++k) {
            const uint64_t a =
                tc::smem_desc_sw128(smem + (k >> 2) * NR * 128 + (k & 3) * 32, 16, 1024);
            const uint64_t b = tc::smem_desc_sw128(ks + (k >> 2) * kChunk + (k & 3) * 32, 16, 1024);
            tc::mma_bf16_ss(tmem + kTmemS + (i & 1) * KT, a, b, idesc_s, k > 0);
          }
          tc::mma_commit(&tail->s_full[i & 1]);
          if (last) tc::mma_commit(&tail->q_empty);
          return true;
        };
        while (ok && walk.next(p, pc)) {
          if (pc.k0 >= pc.k1) continue;
          const int n = pc.k1 - pc.k0;
          ok = mbar_wait(&tail->q_full, pieces & 1, p.err);
          ok = ok && issue_s(g, n == 1);
          for (int j = 0; ok && j < n; ++j, ++g) {
            if (j + 1 < n && !issue_s(g + 1, j + 2 == n)) ok = false;
            if (!ok || !mbar_wait(&tail->p_full, g & 1, p.err) || aborted(tail)) {
              ok = false;
              break;
            }
            // the first product of a piece overwrites O: the last piece is out
            if (j == 0 && pieces > 0 && !mbar_wait(&tail->o_empty, (pieces - 1) & 1, p.err)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const int st = g % kStages;
            const uint8_t* ks = smem + S::kOffK + st * S::kStage;
#pragma unroll
            for (int m = 0; m < kBlocks; ++m)
#pragma unroll
              for (int k = 0; k < KT / 16; ++k) {
                const uint64_t a =
                    tc::smem_desc_sw128(ks + 2 * m * kChunk + k * 16 * 128, kChunk, 1024);
                const uint64_t b = tc::smem_desc_sw128(ps + k * 32, 16, 1024);
                tc::mma_bf16_ss(tmem + m * NR, a, b, idesc_o, j > 0 || k > 0);
              }
            tc::mma_commit(&tail->k_empty[st]);
            tc::mma_commit(&tail->pv_done);
          }
          ++pieces;
        }
        if (!ok) tail->abort = 1;
        tc::mma_commit(&tail->final_mma);
        mbar_wait(&tail->final_mma, 0, p.err);
      }
      __syncwarp();
    } else if (warp >= 4) {
      // ---------------------------------------------------- softmax and output
      const int w4 = warp - 4;
      const bool scores = w4 * 16 < NR;          // this warp's rows w4 * 16 .. + 15
      const int ra = w4 * 16 + (lane >> 2), rb = ra + 8;  // the thread's two rows
      const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
      uint8_t* ps = smem + S::kOffP;
      const int tid = threadIdx.x - 128;
      Walk<NR> walk(tail, begin, end);
      Piece pc;
      int g = 0;
      bool bad = false, stop = false;
      while (!stop && walk.next(p, pc)) {
        const bool none = pc.k0 >= pc.k1;
        const int row0 = pc.tile * NR;
        int lim_a = 0, lim_b = 0;  // keys the rows see
        if (scores) {
          const int vis = walk.q.seq - walk.q.q_len + 1;
          if (ra < pc.rows) lim_a = p.causal ? vis + (row0 + ra) / p.Hq : walk.q.seq;
          if (rb < pc.rows) lim_b = p.causal ? vis + (row0 + rb) / p.Hq : walk.q.seq;
        }
        float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
        for (int j = pc.k0; j < pc.k1; ++j, ++g) {
          bad = bad ||
                !__all_sync(0xffffffffu, mbar_wait(&tail->s_full[g & 1], (g >> 1) & 1, p.err)) ||
                aborted(tail);
          if (bad && lane == 0) tail->fail[g & 1] = 1;
          tc::fence_after_sync();
          uint32_t sr[32];
          float* s = reinterpret_cast<float*>(sr);
          float aa = 1.f, ab = 1.f;
          bool rescale = false;
          const int key0 = j * KT;
          if (scores && !bad) {
            tmem_ld_16x64(tmem + kTmemS + (g & 1) * KT + lanes, sr);
            tc::tmem_wait_ld();
            if (key0 + KT > min(lim_a, lim_b)) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int key = key0 + (i >> 2) * 8 + 2 * (lane & 3) + (i & 1);
                if (key >= ((i & 2) ? lim_b : lim_a)) s[i] = -INFINITY;
              }
            }
            float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              ta = fmax3(ta, s[i], s[i + 1]);
              tb = fmax3(tb, s[i + 2], s[i + 3]);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, o));
              tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, o));
            }
            ta *= p.scale_log2;
            tb *= p.scale_log2;
            // the reference maximum moves only when it grows by more than 2^8
            // (any reference gives the same softmax; P stays below 2^8)
            if (ma == -INFINITY) {
              ma = ta;
            } else if (ta > ma + kRescaleLog2) {
              aa = ex2_ftz(ma - ta);
              ma = ta;
              rescale = true;
            }
            if (mb == -INFINITY) {
              mb = tb;
            } else if (tb > mb + kRescaleLog2) {
              ab = ex2_ftz(mb - tb);
              mb = tb;
              rescale = true;
            }
            const float na = ma == -INFINITY ? 0.f : -ma, nb = mb == -INFINITY ? 0.f : -mb;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              s[i] = ex2_ftz(fmaf(s[i], p.scale_log2, na));
              s[i + 1] = ex2_ftz(fmaf(s[i + 1], p.scale_log2, na));
              s[i + 2] = ex2_ftz(fmaf(s[i + 2], p.scale_log2, nb));
              s[i + 3] = ex2_ftz(fmaf(s[i + 3], p.scale_log2, nb));
              sa += s[i] + s[i + 1];
              sb += s[i + 2] + s[i + 3];
            }
            la = la * aa + sa;
            lb = lb * ab + sb;
            if ((lane & 3) == 0) {
              tail->alpha[g & 1][ra] = aa;
              tail->alpha[g & 1][rb] = ab;
            }
          }
          // O is rescaled by all four warps (a warp holds 32 latent dims of
          // every row) when any row asks for it
          const bool any = named_bar_or(1, 128, rescale);
          if (agreed_to_stop(tail, g & 1)) {
            stop = true;
            break;
          }
          if (g > 0 && (any || scores)) {
            // P is free, and O complete, once PV(g - 1) is done
            if (!__all_sync(0xffffffffu, mbar_wait(&tail->pv_done, (g - 1) & 1, p.err))) {
              bad = true;
              continue;
            }
          }
          if (any) {
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < kBlocks * NR; c += 16) {
              uint32_t o[16];
              tmem_ld16(tmem + lanes + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * tail->alpha[g & 1][c % NR + i]);
              tmem_st16(tmem + lanes + c, o);
            }
            tc::tmem_wait_st();
          }
          if (scores) {
            const int mi = lane >> 3;  // the 8x8 matrix whose row this lane addresses
            const int row = w4 * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int gran = 2 * i + (mi >> 1);
              stmatrix_x4(ps + row * 128 + ((gran ^ (row & 7)) << 4),
                          pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                          pack_bf16(s[8 * i + 4], s[8 * i + 5]),
                          pack_bf16(s[8 * i + 6], s[8 * i + 7]));
            }
          }
          if (key0 + KT > pc.n_keys) {
            // the tile holds keys past the last visible one (unloaded blocks,
            // unwritten cells): zero them, so that P = 0 never meets a NaN
            uint8_t* ks = smem + S::kOffK + (g % kStages) * S::kStage;
            for (int i = tid; i < (L / 64) * KT * 8; i += 128) {
              const int c = i / (KT * 8), n = (i / 8) % KT;
              if (key0 + n >= pc.n_keys)
                *reinterpret_cast<uint4*>(ks + c * kChunk + n * 128 + (i & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
          }
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->p_full);
        }
        if (stop) break;

        // ---- the piece's rows: normalised to out, or a partial
        if (scores) {
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            la += __shfl_xor_sync(0xffffffffu, la, o);
            lb += __shfl_xor_sync(0xffffffffu, lb, o);
          }
          if ((lane & 3) == 0) {
            if (pc.slot < 0) {
              tail->l[ra] = la > 0.f ? 1.f / la : 0.f;
              tail->l[rb] = lb > 0.f ? 1.f / lb : 0.f;
            } else {
              float2* ml = p.part_ml + (int64_t)(2 * cta + pc.slot) * NR;
              ml[ra] = make_float2(ma, la);
              ml[rb] = make_float2(mb, lb);
            }
          }
        }
        if (none) continue;  // sums of zero: the join skips it
        bad = bad ||
              !__all_sync(0xffffffffu, mbar_wait(&tail->pv_done, (g - 1) & 1, p.err)) ||
              aborted(tail);
        if (bad && lane == 0) tail->fail[2] = 1;
        named_bar_sync(1, 128);
        if (agreed_to_stop(tail, 2)) {
          stop = true;
          break;
        }
        tc::fence_after_sync();
        const int64_t out_row = (int64_t)walk.q.q_begin * p.Hq + row0;
        __nv_bfloat16* orow = p.out + out_row * L + w4 * 32 + lane;
        float* prow = p.part_o + (int64_t)(2 * cta + max(pc.slot, 0)) * NR * L + w4 * 32 + lane;
#pragma unroll 1
        for (int m = 0; m < kBlocks; ++m)
#pragma unroll 1
          for (int c = 0; c < NR; c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem + lanes + m * NR + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c + i >= pc.rows) break;
              const float v = __uint_as_float(o[i]);
              if (pc.slot < 0)
                orow[(int64_t)(c + i) * L + m * 128] = __float2bfloat16_rn(v * tail->l[c + i]);
              else
                prow[(c + i) * L + m * 128] = v;
            }
          }
        tc::fence_before_sync();
        named_bar_sync(1, 128);  // tail->l is free again
        if (lane == 0) mbar_arrive(&tail->o_empty);
      }
      if (stop) tail->abort = 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partials of the units cut at CTA boundaries: grid (attention CTAs,
// row groups), one warp per row. o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
constexpr int kJoinWarps = 8;

template <int L, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const LatentParams p) {
  grid_dependency_wait();  // the partials are complete and visible
  const int b = blockIdx.x;
  const LatentJoin j = p.joins[b];
  const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= j.rows) return;
  // piece i: slot 2 b - 1 for i = 0, then slots 2 (b + i - 1)
  const int n = j.last - b + 2;
  auto slot = [&](int i) -> int64_t { return i == 0 ? 2 * b - 1 : 2 * (b + i - 1); };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float2 ml = p.part_ml[slot(i) * NR + row];
    if (ml.y > 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  constexpr int kV = L / 128;
  float4 acc[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < n) {
      const float2 ml = p.part_ml[slot(i0 + lane) * NR + row];
      if (ml.y > 0.f) {  // a piece without a visible key has no partial
        w = ex2_ftz(ml.x - m);
        l += w * ml.y;
      }
    }
    const int cnt = min(32, n - i0);
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (wi == 0.f) continue;
      const float4* src =
          reinterpret_cast<const float4*>(p.part_o + (slot(i0 + i) * NR + row) * L) + lane;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const float4 x = __ldcg(src + v * 32);
        acc[v].x = fmaf(wi, x.x, acc[v].x);
        acc[v].y = fmaf(wi, x.y, acc[v].y);
        acc[v].z = fmaf(wi, x.z, acc[v].z);
        acc[v].w = fmaf(wi, x.w, acc[v].w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(p.out + (j.out_row + row) * L) + lane;
#pragma unroll
  for (int v = 0; v < kV; ++v)
    dst[v * 32] = make_uint2(pack_bf16(acc[v].x * inv, acc[v].y * inv),
                             pack_bf16(acc[v].z * inv, acc[v].w * inv));
}

// ----------------------------------------------------------------- host side

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// joins, statistics and partials of a grid of n CTAs with NR-row tiles
size_t scratch_bytes(int n, int NR, int L) {
  return align256((size_t)n * sizeof(LatentJoin)) + align256((size_t)2 * n * NR * sizeof(float2)) +
         (size_t)2 * n * NR * L * sizeof(float);
}

bool encode_2d(CUtensorMap* m, CUtensorMapDataType type, int elt, const void* base, int64_t cols,
               int64_t rows, int box_cols, int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * elt};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, type, 2, const_cast<void*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int L, int NR>
pa_status launch(const LatentParams& p, const void* q, const pa_latent_pool* pool, int grid,
                 cudaStream_t s) {
  using S = Smem<L, NR>;
  CUtensorMap tq, tc, tr;
  const int64_t cells = (int64_t)pool->num_blocks * pool->block_size;
  if (!encode_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q, L + kRope, (int64_t)p.T * p.Hq, 64,
                 NR) ||
      !encode_2d(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool->latent, L, cells, 64, p.B) ||
      !encode_2d(&tr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool->rope, kRope, cells, 64, p.B))
    return PA_ERR_CUDA;
  if (cudaFuncSetAttribute(latent_attn_kernel<L, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           S::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  latent_attn_kernel<L, NR><<<grid, kThreads, S::kAlloc, s>>>(tq, tc, tr, p);
  pa_status st = launch_status();
  if (st != PA_OK || grid == 1) return st;  // one CTA cuts nothing
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, NR / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, latent_join_kernel<L, NR>, p) != cudaSuccess) return PA_ERR_CUDA;
  count_launches(1);
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_latent_workspace_size(int32_t num_q_heads, int32_t latent_dim) {
  if (num_q_heads <= 0 || (latent_dim != 256 && latent_dim != 512)) return 0;
  return pa::scratch_bytes(std::min(pa::num_sms(), pa::kLatentMaxCtas), pa::kLatentRows, latent_dim);
}

extern "C" pa_status pa_latent_forward(const void* q, void* out, const int32_t* query_start_loc,
                                       const int32_t* seq_lens, const int32_t* qsl_host,
                                       const int32_t* seq_lens_host, const int32_t* block_tables,
                                       int32_t max_blocks, int32_t num_reqs, int32_t num_tokens,
                                       int32_t num_q_heads, const pa_latent_pool* pool,
                                       float scale, int32_t causal, void* workspace,
                                       size_t workspace_bytes, pa_stream_t stream) {
  pa_status st = pa::check_latent_pool(pool);
  if (st != PA_OK) return st;
  const int R = num_reqs, T = num_tokens, Hq = num_q_heads, L = pool->latent_dim;
  if (R < 0 || T < 0 || Hq <= 0 || max_blocks < 0) return PA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  if (causal != 0 && causal != 1) return PA_ERR_INVALID;
  if (R == 0) return T == 0 ? PA_OK : PA_ERR_INVALID;
  if (T > 0 && pool->num_blocks == 0) return PA_ERR_INVALID;  // no block a table could name
  if (!qsl_host || !seq_lens_host || !query_start_loc || !seq_lens || !block_tables)
    return PA_ERR_INVALID;
  if (T > 0 && (!q || !out || !pa::aligned16(q) || !pa::aligned16(out))) return PA_ERR_INVALID;
  if (workspace_bytes > 0 && (!workspace || !pa::aligned16(workspace))) return PA_ERR_INVALID;
  if (qsl_host[0] != 0 || qsl_host[R] != T) return PA_ERR_INVALID;
  for (int r = 0; r < R; ++r) {
    const int ql = qsl_host[r + 1] - qsl_host[r];
    if (ql < 0) return PA_ERR_INVALID;
    if (ql == 0) continue;
    const int seq = seq_lens_host[r];
    if (seq < ql || (int64_t)seq > (int64_t)max_blocks * pool->block_size) return PA_ERR_INVALID;
  }
  if (T == 0) return PA_OK;
  if (pool->dtype != PA_KV_BF16) return PA_ERR_UNSUPPORTED;
  // rows are addressed by 32-bit tensor-map coordinates
  if ((int64_t)T * Hq > INT32_MAX - pa::kLatentRows) return PA_ERR_UNSUPPORTED;

  // Row tiles: the smallest of 16, 32 and 64 rows that covers the widest
  // request in one pass over its cells; 64 past that.
  int64_t widest = 0, W = 0;
  for (int r = 0; r < R; ++r)
    widest = std::max<int64_t>(widest, (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq);
  const int NR = widest <= 16 ? 16 : widest <= 32 ? 32 : 64;
  for (int r = 0; r < R; ++r) {
    const int64_t rows = (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq;
    if (rows > 0)
      W += (rows + NR - 1) / NR * ((seq_lens_host[r] + pa::kLatentKeys - 1) / pa::kLatentKeys);
  }
  const int grid = (int)std::min<int64_t>(W, std::min(pa::num_sms(), pa::kLatentMaxCtas));
  if (workspace_bytes < pa::scratch_bytes(grid, NR, L)) return PA_ERR_INVALID;

  pa::LatentParams p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.block_tables = block_tables;
  p.scales = pool->scales;
  p.T = T;
  p.R = R;
  p.Hq = Hq;
  p.max_blocks = max_blocks;
  p.num_blocks = pool->num_blocks;
  p.B = pool->block_size;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.joins = reinterpret_cast<pa::LatentJoin*>(ws);
  ws += pa::align256((size_t)grid * sizeof(pa::LatentJoin));
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += pa::align256((size_t)2 * grid * NR * sizeof(float2));
  p.part_o = reinterpret_cast<float*>(ws);
  p.err = pa::error_word();
  if (!p.err) return PA_ERR_CUDA;
  cudaStream_t s = pa::as_stream(stream);
  auto go = [&](auto l) {
    constexpr int kL = decltype(l)::value;
    return NR == 16   ? pa::launch<kL, 16>(p, q, pool, grid, s)
           : NR == 32 ? pa::launch<kL, 32>(p, q, pool, grid, s)
                      : pa::launch<kL, 64>(p, q, pool, grid, s);
  };
  return L == 512 ? go(std::integral_constant<int, 512>{}) : go(std::integral_constant<int, 256>{});
}
