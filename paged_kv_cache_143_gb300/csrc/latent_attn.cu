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
// One CTA per SM walks an equal share of all (row tile, 32-key tile) pairs
// (pa::LatentParams). Both products run on the 5th-generation tensor cores:
//   S [64 rows x 32 keys] = Q K^T     Q and the cells K-major in shared memory
//   O^T [L x NR]        += c^T P^T    the same cells read again, MN-major, as
//                                     the A operand; P from shared memory
// O is kept transposed (lane = latent dim, column = row) because a row of O is
// L fp32 values: NR x 512 of them as [dim][row] take 4 NR TMEM columns, and the
// products stay full 128-row instructions for few query rows, where rows
// down the lanes would leave most of the tensor core idle. NR is 16, 32 or 64.
// Tiles are 32 keys (36 KB at L 512) so that four of them fit beside 64 rows of
// Q: a stage is loading for about 2000 cycles and in use (S, softmax, PV and
// their hand-overs) for 2700, and what HBM delivers a tile in is 1570.
//   warp 0      TMA producer: the Q tile, then the key tiles into a ring of stages
//   warp 1      TMEM and, one elected lane, S, up to four tiles ahead
//   warp 2      one elected lane, PV. (One lane for both spent a third of a tile's
//               time between the two batches of products.)
//   warps 4-7   softmax of 16 rows each (S read as 16 x 256-bit fragments: a row
//               in four lanes), P written by stmatrix; then the output
// The softmax warps share nothing tile by tile. A warp that moves a row's
// reference maximum says so beside P; warp 2 then asks all four to rescale
// their dims of O before it issues that PV (rare: growth by more than 2^8).
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
constexpr int kChunk = KT * 128;   // 64 bf16 columns of a key tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;   // S buffers at columns 256, 288, 320, 352
constexpr int kSBufs = 4, kMaxStages = 10;
constexpr float kRescaleLog2 = 8.f;

template <int L, int NR>
struct Smem {
  static constexpr int kChunks = L / 64 + 1;          // the last one is the rotary part
  static constexpr int kQBytes = kChunks * NR * 128;
  static constexpr int kStage = kChunks * kChunk;
  static constexpr int kPBytes = NR * 128;            // two tiles of P side by side
  static constexpr int kTail = 2048;                  // barriers and row statistics
  static constexpr int kFit = (232448 - 1024 - kTail - kQBytes - kPBytes) / kStage;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffP = kOffK + kStages * kStage;
  static constexpr int kOffTail = kOffP + kPBytes;
  static constexpr int kAlloc = kOffTail + kTail + 1024;  // the base is rounded up to 1024 B
  static_assert(kStages >= 4, "needs four key tiles in flight");
  static_assert(kAlloc <= 232448, "dynamic shared memory above the 227 KB per-block limit");
  static_assert(kOffK % 1024 == 0 && kOffP % 1024 == 0, "swizzled tiles start on 1024 bytes");
  // S always reads 64 rows of Q: the rows past NR are whatever follows in
  // shared memory (their scores are never looked at)
  static_assert(kQBytes + (64 - NR) * 128 <= kAlloc - 1024, "Q over-read leaves the allocation");
};

struct Tail {
  uint64_t q_full, q_empty;
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t s_full[kSBufs], s_empty[kSBufs];
  uint64_t p_full[2], pv_done[2];
  uint64_t fix, fixed;           // O is to be rescaled for tile fix_tile; it has been
  uint64_t o_empty, final_mma;
  float alpha[2][kLatentRows];   // by tile: factors of the rows of a warp that asks
  float l[2][kLatentRows];       // by piece: 1 / sum
  uint8_t ask[2][4];             // by tile: softmax warps that ask for a rescale
  int32_t fix_tile;
  int64_t warp_sum[kThreads / 32];
  int32_t base;        // flat start of the request that holds the CTA's first tile
  int32_t req;         // that request
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail) <= 2048, "Tail overruns its slot");

__device__ __forceinline__ bool aborted(Tail* t) {
  return *reinterpret_cast<volatile int*>(&t->abort) != 0;
}

// 16 lanes x 32 columns as mma-style fragments: of each 8-column group i,
// r[4 i], r[4 i + 1] are columns 2 (lane % 4), + 1 of row lane / 4, and
// r[4 i + 2], r[4 i + 3] those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
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
  int32_t q_begin, q_len, seq, rows, keys;  // query rows, key tiles
  int64_t weight;                           // passes * keys; 0 for one without work
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
  q.rows = q.q_len * p.Hq;  // (T * Hq fits 32 bits)
  q.keys = (q.seq + KT - 1) / KT;
  const int tiles = (q.rows + NR - 1) / NR;
  q.weight = (int64_t)((tiles + p.lanes - 1) / p.lanes) * q.keys;
  return q;
}

// A CTA's part of one pass: key tiles [k0, k1) for row tile `tile` of request r.
struct Piece {
  int32_t r, tile, k0, k1;
  int32_t n_keys;      // keys any row of the tile sees (k1 is cut to it)
  int32_t rows;        // valid query rows of the tile (none: the pass has fewer tiles)
  int32_t slot;        // partial slot 0 / 1 of the CTA, or -1: the whole pass
};

// (The whole flat space fits 31 bits, so do all positions.)
template <int NR>
struct Walk {
  int32_t pos, end, base, r, lane;
  bool loaded;
  Request q;

  __device__ Walk(const Tail* t, int32_t begin, int32_t stop, int32_t in_group)
      : pos(begin), end(stop), base(t->base), r(t->req), lane(in_group), loaded(false), q{} {}

  __device__ bool next(const LatentParams& p, Piece& out) {
    if (pos >= end) return false;
    if (!loaded) {
      q = load_request<NR>(p, r, false);
      loaded = true;
    }
    while (pos - base >= (int32_t)q.weight) {
      base += (int32_t)q.weight;
      if (++r >= p.R) return false;
      q = load_request<NR>(p, r, false);
    }
    const unsigned off = pos - base;
    out.r = r;
    const int pass = (int)(off / (unsigned)q.keys);
    out.tile = pass * p.lanes + lane;
    out.k0 = (int)off - pass * q.keys;
    const int k1 = min(q.keys, out.k0 + (end - pos));
    pos += k1 - out.k0;
    out.slot = out.k0 > 0 ? 0 : k1 < q.keys ? 1 : -1;
    out.rows = min(NR, q.rows - out.tile * NR);
    if (out.rows <= 0) {
      out.rows = 0;
      out.k1 = out.k0;
      return true;
    }
    out.n_keys = q.seq;
    if (p.causal && q.q_len > 1) {  // up to the last row's token
      const unsigned last_row = out.tile * NR + out.rows - 1;
      out.n_keys = q.seq - q.q_len + (int)(last_row / (unsigned)p.Hq) + 1;
    }
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
  constexpr int kBlocks = L / 128;  // 128-dim blocks of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + S::kOffTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, group = cta / p.lanes, in_group = cta - group * p.lanes;
  const int groups = gridDim.x / p.lanes;
  launch_dependents();  // the join that follows may be scheduled now

  // ---- this group's range: W, then the request that holds tile group * Q
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
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&tail->s_full[s], 1);
      mbar_init(&tail->s_empty[s], NR / 16);  // the warps that read S
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail->p_full[s], 4);   // one arrival per softmax warp
      mbar_init(&tail->pv_done[s], 1);
    }
    mbar_init(&tail->fix, 1);
    mbar_init(&tail->fixed, 4);
    mbar_init(&tail->o_empty, 4);
    mbar_init(&tail->final_mma, 2);
    tail->abort = 0;
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
  if (W > INT32_MAX) {  // (the host has checked its mirrors)
    if (cta == 0 && threadIdx.x == 0) raise_error(p.err, kErrBounds);
    W = 0;
  }
  const unsigned Q = ((unsigned)W + groups - 1) / groups;
  const int begin = (int)min(W, (int64_t)group * Q), end = (int)min(W, (int64_t)begin + Q);
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
        tail->base = (int)before;
      }
    }
  } else if (begin >= kept_before && begin < kept_before + kept_w) {
    tail->req = threadIdx.x;
    tail->base = (int)kept_before;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tail->tmem;
  if (threadIdx.x == 96) {
    // the pass cut at this group's start, for the join: handled at its first cut
    LatentJoin j{};
    if (begin < end) {
      const Request q = load_request<NR>(p, tail->req, false);
      const int pass = (begin - tail->base) / q.keys;
      const unsigned a = tail->base + pass * q.keys;  // the pass's start
      const int row0 = (pass * p.lanes + in_group) * NR;
      if ((unsigned)begin > a && a / Q + 1 == (unsigned)group && row0 < q.rows) {
        j.rows = min(q.rows - row0, NR);
        j.pieces = (int32_t)((a + q.keys - 1) / Q - a / Q) + 1;
        j.out_row = (int64_t)q.q_begin * p.Hq + row0;
      }
    }
    p.joins[cta] = j;
  }

  if (begin < end) {
    if (warp == 0) {
      // --------------------------------------------------------- TMA producer
      // (one lane: a copy instruction with several lanes active costs about
      // 120 cycles a lane, and the ring then waits for its producer)
      if (tc::elect_one()) {
        tc::prefetch_tensormap(&tmap_q);
        tc::prefetch_tensormap(&tmap_c);
        tc::prefetch_tensormap(&tmap_r);
        Walk<NR> walk(tail, begin, end, in_group);
        Piece pc;
        int g = 0, pieces = 0;     // key tiles and pieces so far
        int st = 0, phase = 1;     // stage, and the parity its emptying waits for
        bool ok = true;
        while (ok && walk.next(p, pc)) {
          if (pc.k0 >= pc.k1) continue;  // no row of the tile sees these keys
          if (pieces > 0 && !mbar_wait(&tail->q_empty, (pieces - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&tail->q_full, S::kQBytes);
          tc::tma_load_3d(smem, &tmap_q, 0, walk.q.q_begin * p.Hq + pc.tile * NR, 0, &tail->q_full);
          ++pieces;
          const int32_t* table = p.block_tables + (int64_t)pc.r * p.max_blocks;
          // physical row of the first key of half i of tile j (16-token blocks
          // fill a tile in two halves)
          auto fetch = [&](int j, int i) -> int {
            const int key = j * KT + i * 16;
            return j < pc.k1 && key < pc.n_keys ? __ldg(table + (key >> p.b_shift)) : 0;
          };
          const bool halves = p.b_shift == 4;
          int id0 = fetch(pc.k0, 0), id1 = halves ? fetch(pc.k0, 1) : 0;
          for (int j = pc.k0; j < pc.k1; ++j, ++g) {
            const int next0 = fetch(j + 1, 0), next1 = halves ? fetch(j + 1, 1) : 0;
            if (id0 < 0 || id0 >= p.num_blocks || id1 < 0 || id1 >= p.num_blocks) {
              raise_error(p.err, kErrBounds);  // a valid block; the output is then unspecified
              if (id0 < 0 || id0 >= p.num_blocks) id0 = 0;
              if (id1 < 0 || id1 >= p.num_blocks) id1 = 0;
            }
            if (g >= kStages && (!mbar_wait(&tail->k_empty[st], phase, p.err) || aborted(tail))) {
              ok = false;
              break;
            }
            uint8_t* dst = smem + S::kOffK + st * S::kStage;
            uint64_t* bar = &tail->k_full[st];
            if (!halves) {
              const int y = (id0 << p.b_shift) + ((j * KT) & ((1 << p.b_shift) - 1));
              mbar_arrive_expect_tx(bar, S::kStage);
              tc::tma_load_3d(dst, &tmap_c, 0, y, 0, bar);
              tc::tma_load_2d(dst + (L / 64) * kChunk, &tmap_r, 0, y, bar);
            } else {
              const bool both = j * KT + 16 < pc.n_keys;
              mbar_arrive_expect_tx(bar, both ? S::kStage : S::kStage / 2);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (i == 1 && !both) break;
                const int y = (i ? id1 : id0) << 4;
#pragma unroll
                for (int c = 0; c < L / 64; ++c)
                  tc::tma_load_3d(dst + c * kChunk + i * 2048, &tmap_c, 0, y, c, bar);
                tc::tma_load_2d(dst + (L / 64) * kChunk + i * 2048, &tmap_r, 0, y, bar);
              }
            }
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
            id0 = next0;
            id1 = next1;
          }
        }
        // every issued copy lands before the CTA may leave
        if (!ok) tail->abort = 1;
        if (pieces > 0) mbar_wait(&tail->q_full, (pieces - 1) & 1, p.err);
        for (int i = max(0, g - kStages); i < g; ++i)
          mbar_wait(&tail->k_full[i % kStages], (i / kStages) & 1, p.err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------------- S
      if (tc::elect_one()) {
        constexpr uint32_t idesc = tc::idesc_16bit_f32(64, KT, false, false, false);
        const uint64_t q_desc = tc::smem_desc_sw128(smem, 16, 1024);
        const uint64_t k_desc = tc::smem_desc_sw128(smem + S::kOffK, 16, 1024);
        Walk<NR> walk(tail, begin, end, in_group);
        Piece pc;
        int g = 0, st = 0, phase = 0, pieces = 0;
        bool ok = true;
        while (ok && walk.next(p, pc)) {
          if (pc.k0 >= pc.k1) continue;
          if (!(ok = mbar_wait(&tail->q_full, pieces & 1, p.err))) break;
          ++pieces;
          for (int j = pc.k0; j < pc.k1; ++j, ++g) {
            const int buf = g % kSBufs;
            ok = (g < kSBufs || mbar_wait(&tail->s_empty[buf], (g / kSBufs - 1) & 1, p.err)) &&
                 mbar_wait(&tail->k_full[st], phase, p.err);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t ks = tc::desc_at(k_desc, st * S::kStage);
            const uint32_t d = tmem + kTmemS + buf * KT;
#pragma unroll
            for (int k = 0; k < S::kChunks * 4; ++k)
              tc::mma_bf16_ss(d, tc::desc_at(q_desc, (k >> 2) * NR * 128 + (k & 3) * 32),
                              tc::desc_at(ks, (k >> 2) * kChunk + (k & 3) * 32), idesc, k > 0);
            tc::mma_commit(&tail->s_full[buf]);
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
          }
          tc::mma_commit(&tail->q_empty);
        }
        if (!ok) tail->abort = 1;
        tc::mma_commit(&tail->final_mma);
        mbar_wait(&tail->final_mma, 0, p.err);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------------ PV
      if (tc::elect_one()) {
        constexpr uint32_t idesc = tc::idesc_16bit_f32(128, NR, true, false, false);
        const uint64_t p_desc = tc::smem_desc_sw128(smem + S::kOffP, 16, 1024);
        const uint64_t v_desc = tc::smem_desc_sw128(smem + S::kOffK, kChunk, 1024);
        Walk<NR> walk(tail, begin, end, in_group);
        Piece pc;
        int g = 0, st = 0, pieces = 0, fixes = 0;
        bool ok = true;
        while (ok && walk.next(p, pc)) {
          if (pc.k0 >= pc.k1) continue;
          for (int j = pc.k0; j < pc.k1; ++j, ++g) {
            if (!(ok = mbar_wait(&tail->p_full[g & 1], (g >> 1) & 1, p.err))) break;
            if (j == pc.k0) {
              // the first product of a piece overwrites O: the last piece is out
              if (pieces > 0 && !(ok = mbar_wait(&tail->o_empty, (pieces - 1) & 1, p.err))) break;
            } else if (*reinterpret_cast<volatile uint32_t*>(&tail->ask[g & 1][0]) != 0) {
              // rows of this tile have a new reference: O, complete up to the
              // tile before, is rescaled first
              *reinterpret_cast<volatile int32_t*>(&tail->fix_tile) = g;
              ok = mbar_wait(&tail->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err);
              mbar_arrive(&tail->fix);
              ok = ok && mbar_wait(&tail->fixed, fixes & 1, p.err);
              if (!ok) break;
              ++fixes;
            }
            tc::fence_after_sync();
            const uint64_t vs = tc::desc_at(v_desc, st * S::kStage);
            const uint64_t ps = tc::desc_at(p_desc, (g & 1) * 64);
#pragma unroll
            for (int m = 0; m < kBlocks; ++m)
#pragma unroll
              for (int k = 0; k < KT / 16; ++k)
                tc::mma_bf16_ss(tmem + m * NR, tc::desc_at(vs, 2 * m * kChunk + k * 16 * 128),
                                tc::desc_at(ps, k * 32), idesc, j > pc.k0 || k > 0);
            tc::mma_commit(&tail->k_empty[st]);
            tc::mma_commit(&tail->pv_done[g & 1]);
            if (++st == kStages) st = 0;
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
      int fixes = 0;
      // this warp's dims of O times the new factors of the rows that ask
      auto rescale = [&]() {
        tc::fence_after_sync();
        const int slot = *reinterpret_cast<volatile int32_t*>(&tail->fix_tile) & 1;
        const uint32_t asked = *reinterpret_cast<volatile uint32_t*>(&tail->ask[slot][0]);
#pragma unroll 1
        for (int c = 0; c < kBlocks * NR; c += 16) {
          const int r = c % NR;  // the rows of softmax warp r / 16
          if (((asked >> (r / 2)) & 0xFF) == 0) continue;
          uint32_t o[16];
          tmem_ld16(tmem + lanes + c, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * tail->alpha[slot][r + i]);
          tmem_st16(tmem + lanes + c, o);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->fixed);
        ++fixes;
      };
      // Waits for a barrier, doing the rescales that are asked for meanwhile.
      auto wait = [&](uint64_t* bar, int parity) -> bool {
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity & 1))) return true;
        unsigned long long t0 = 0;
        for (int spin = 1;; ++spin) {
          if (__all_sync(0xffffffffu, mbar_test_wait(&tail->fix, fixes & 1))) rescale();
          if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity & 1))) return true;
          if ((spin & 1023) == 0) {
            const unsigned long long now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
              if (lane == 0) raise_error(p.err, kErrTimeout);
              return false;
            }
          }
        }
      };
      Walk<NR> walk(tail, begin, end, in_group);
      Piece pc;
      int g = 0, pieces = 0;
      bool ok = true;
      while (ok && walk.next(p, pc)) {
        const int row0 = pc.tile * NR;
        int lim_a = 0, lim_b = 0;  // keys the rows see
        if (scores) {
          const int vis = walk.q.seq - walk.q.q_len + 1;
          if (ra < pc.rows) lim_a = p.causal ? vis + (row0 + ra) / p.Hq : walk.q.seq;
          if (rb < pc.rows) lim_b = p.causal ? vis + (row0 + rb) / p.Hq : walk.q.seq;
        }
        float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
        for (int j = pc.k0; j < pc.k1; ++j, ++g) {
          uint32_t sr[16];
          float* s = reinterpret_cast<float*>(sr);
          float aa = 1.f, ab = 1.f;
          const int key0 = j * KT;
          if (scores) {
            if (!(ok = wait(&tail->s_full[g % kSBufs], g / kSBufs))) break;
            tc::fence_after_sync();
            tmem_ld_16x32(tmem + kTmemS + (g % kSBufs) * KT + lanes, sr);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            if (lane == 0) mbar_arrive(&tail->s_empty[g % kSBufs]);
            if (key0 + KT > min(lim_a, lim_b)) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int key = key0 + (i >> 2) * 8 + 2 * (lane & 3) + (i & 1);
                if (key >= ((i & 2) ? lim_b : lim_a)) s[i] = -INFINITY;
              }
            }
            float ta = fmax3(fmaxf(s[0], s[1]), s[4], s[5]);
            float tb = fmax3(fmaxf(s[2], s[3]), s[6], s[7]);
            ta = fmax3(ta, fmaxf(s[8], s[9]), fmaxf(s[12], s[13]));
            tb = fmax3(tb, fmaxf(s[10], s[11]), fmaxf(s[14], s[15]));
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
            }
            if (mb == -INFINITY) {
              mb = tb;
            } else if (tb > mb + kRescaleLog2) {
              ab = ex2_ftz(mb - tb);
              mb = tb;
            }
            const float na = ma == -INFINITY ? 0.f : -ma, nb = mb == -INFINITY ? 0.f : -mb;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              s[i] = ex2_ftz(fmaf(s[i], p.scale_log2, na));
              s[i + 1] = ex2_ftz(fmaf(s[i + 1], p.scale_log2, na));
              s[i + 2] = ex2_ftz(fmaf(s[i + 2], p.scale_log2, nb));
              s[i + 3] = ex2_ftz(fmaf(s[i + 3], p.scale_log2, nb));
              sa += s[i] + s[i + 1];
              sb += s[i + 2] + s[i + 3];
            }
            la = la * aa + sa;
            lb = lb * ab + sb;
          }
          // PV(g - 2) has read this half of P, and what was published with it
          if (g >= 2 && !(ok = wait(&tail->pv_done[g & 1], (g >> 1) - 1))) break;
          if (scores) {
            const int mi = lane >> 3;  // the 8x8 matrix whose row this lane addresses
            const int row = w4 * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int gran = (g & 1) * 4 + 2 * i + (mi >> 1);
              stmatrix_x4(ps + row * 128 + ((gran ^ (row & 7)) << 4),
                          pack_bf16(s[8 * i], s[8 * i + 1]), pack_bf16(s[8 * i + 2], s[8 * i + 3]),
                          pack_bf16(s[8 * i + 4], s[8 * i + 5]),
                          pack_bf16(s[8 * i + 6], s[8 * i + 7]));
            }
          }
          const bool ask = __any_sync(0xffffffffu, aa < 1.f || ab < 1.f);
          if (ask && (lane & 3) == 0) {
            tail->alpha[g & 1][ra] = aa;
            tail->alpha[g & 1][rb] = ab;
          }
          if (lane == 0) tail->ask[g & 1][w4] = ask;
          if (key0 + KT > pc.n_keys) {
            // the tile holds keys past the last visible one (unloaded blocks,
            // unwritten cells): zero them, so that P = 0 never meets a NaN (S of
            // this tile has read them: every warp waits for it)
            if (!scores && !(ok = wait(&tail->s_full[g % kSBufs], g / kSBufs))) break;
            constexpr int kCols = L / 64;  // chunks: the thread's is (tid / 8) % kCols
            uint8_t* ks = smem + S::kOffK + (g % kStages) * S::kStage +
                          ((tid >> 3) & (kCols - 1)) * kChunk + (tid & 7) * 16;
            for (int n = pc.n_keys - key0 + tid / (8 * kCols); n < KT; n += 16 / kCols)
              *reinterpret_cast<uint4*>(ks + n * 128) = make_uint4(0, 0, 0, 0);
          }
          if (j == pc.k1 - 1 && scores) {
            // the piece's sums, before the arrival that its output waits behind
            float ua = la, ub = lb;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              ua += __shfl_xor_sync(0xffffffffu, ua, o);
              ub += __shfl_xor_sync(0xffffffffu, ub, o);
            }
            if ((lane & 3) == 0) {
              tail->l[pieces & 1][ra] = ua > 0.f ? 1.f / ua : 0.f;
              tail->l[pieces & 1][rb] = ub > 0.f ? 1.f / ub : 0.f;
              if (pc.slot >= 0) {
                float2* ml = p.part_ml + (int64_t)(2 * cta + pc.slot) * NR;
                ml[ra] = make_float2(ma, ua);
                ml[rb] = make_float2(mb, ub);
              }
            }
          }
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->p_full[g & 1]);
        }
        if (!ok) break;

        if (pc.k0 >= pc.k1) {  // no key for any row: sums of zero, which the join skips
          if (scores && pc.slot >= 0 && (lane & 3) == 0) {
            float2* ml = p.part_ml + (int64_t)(2 * cta + pc.slot) * NR;
            ml[ra] = ml[rb] = make_float2(-INFINITY, 0.f);
          }
          continue;
        }
        // ---- the piece's rows: normalised to out, or a partial
        if (!(ok = wait(&tail->pv_done[(g - 1) & 1], (g - 1) >> 1))) break;
        tc::fence_after_sync();
        const int64_t out_row = (int64_t)walk.q.q_begin * p.Hq + row0;
        if (pc.slot < 0) {
          // lane = dim, register = row: three exchanges between lanes whose
          // numbers differ in one bit leave 8 dims of two rows in each lane
          __nv_bfloat16* orow = p.out + out_row * L + w4 * 32 + (lane >> 3) * 8;
#pragma unroll 1
          for (int c = 0; c < NR; c += 16) {
            if (c >= pc.rows) break;
            float inv[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(inv + i) =
                  *reinterpret_cast<const float4*>(&tail->l[pieces & 1][c + i]);
            // row of the lane's first output: bit 0, 1, 2 of the lane pick bits
            // 3, 2, 1 of the row
            const int row = c + (lane & 1) * 8 + (lane & 2) * 2 + ((lane & 4) >> 1);
#pragma unroll 1
            for (int m = 0; m < kBlocks; ++m) {
              uint32_t o[16];
              tmem_ld16(tmem + lanes + m * NR + c, o);
              tc::tmem_wait_ld();
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // lane pairs: bf16 of two dims, 8 rows each
                const float x = __uint_as_float(o[i]) * inv[i];
                const float y = __uint_as_float(o[i + 8]) * inv[i + 8];
                const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
                w[i] = (lane & 1) ? pack_bf16(got, y) : pack_bf16(x, got);
              }
              uint32_t u[4][2];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // four dims, 4 rows each
                const uint32_t got = __shfl_xor_sync(0xffffffffu, (lane & 2) ? w[i] : w[i + 4], 2);
                u[i][0] = (lane & 2) ? got : w[i];
                u[i][1] = (lane & 2) ? w[i + 4] : got;
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // eight dims, 2 rows each
                const bool up = (lane & 4) != 0;
                const uint32_t g0 = __shfl_xor_sync(0xffffffffu, up ? u[i][0] : u[i + 2][0], 4);
                const uint32_t g1 = __shfl_xor_sync(0xffffffffu, up ? u[i][1] : u[i + 2][1], 4);
                if (row + i < pc.rows)
                  *reinterpret_cast<uint4*>(orow + (int64_t)(row + i) * L + m * 128) =
                      up ? make_uint4(g0, g1, u[i + 2][0], u[i + 2][1])
                         : make_uint4(u[i][0], u[i][1], g0, g1);
              }
            }
          }
        } else {
          float* prow = p.part_o + (int64_t)(2 * cta + pc.slot) * NR * L + w4 * 32 + lane;
#pragma unroll 1
          for (int c = 0; c < NR; c += 16) {
            if (c >= pc.rows) break;
#pragma unroll 1
            for (int m = 0; m < kBlocks; ++m) {
              uint32_t o[16];
              tmem_ld16(tmem + lanes + m * NR + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)  // (rows past the unit's are scratch)
                prow[(c + i) * L + m * 128] = __uint_as_float(o[i]);
            }
          }
        }
        ++pieces;
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->o_empty);
      }
      if (!ok) tail->abort = 1;
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
  // piece 0 is slot 1 of the CTA one group back, piece i slot 0 of the CTA
  // i - 1 groups on
  const int n = j.pieces;
  auto slot = [&](int i) -> int64_t { return 2 * (b + (i - 1) * p.lanes) + (i == 0 ? 1 : 0); };
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

// Rows of `chunks` times 64 bf16 columns, row_bytes apart, as [chunk][row][64]:
// one box is `box_rows` rows of `box_chunks` chunks, chunk after chunk in shared
// memory, each 128-byte swizzled.
bool encode_chunks(CUtensorMap* m, const void* base, int chunks, int64_t row_bytes, int64_t rows,
                   int box_rows, int box_chunks) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)chunks};
  const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rope(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {kRope, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {kRope * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int L, int NR>
pa_status launch(const LatentParams& p, const void* q, const pa_latent_pool* pool, int grid,
                 cudaStream_t s) {
  using S = Smem<L, NR>;
  CUtensorMap tq, tc, tr;
  const int64_t cells = (int64_t)pool->num_blocks * pool->block_size;
  const int box_rows = std::min(pool->block_size, KT);
  if (!encode_chunks(&tq, q, L / 64 + 1, (L + kRope) * 2, (int64_t)p.T * p.Hq, NR, L / 64 + 1) ||
      !encode_chunks(&tc, pool->latent, L / 64, L * 2, cells, box_rows,
                     box_rows == KT ? L / 64 : 1) ||
      !encode_rope(&tr, pool->rope, cells, box_rows))
    return PA_ERR_CUDA;
  if (cudaFuncSetAttribute(latent_attn_kernel<L, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           S::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  latent_attn_kernel<L, NR><<<grid, kThreads, S::kAlloc, s>>>(tq, tc, tr, p);
  pa_status st = launch_status();
  if (st != PA_OK || grid == p.lanes) return st;  // one group cuts nothing
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
  int64_t widest = 0;
  for (int r = 0; r < R; ++r)
    widest = std::max<int64_t>(widest, (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq);
  const int NR = widest <= 16 ? 16 : widest <= 32 ? 32 : 64;
  // CTAs side by side (LatentParams): a tile of keys costs a CTA about 1300
  // cycles of products and HBM 1570 cycles of an SM's share; two CTAs on the same
  // keys share the latter (more would gain nothing: the products then bound).
  const int sms = std::min(pa::num_sms(), pa::kLatentMaxCtas);
  int64_t W = 0, best = INT64_MAX;
  int G = 1;
  for (int lanes = 1; lanes <= 2; ++lanes) {
    int64_t w = 0;
    for (int r = 0; r < R; ++r) {
      const int64_t rows = (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq;
      if (rows > 0)
        w += ((rows + NR - 1) / NR + lanes - 1) / lanes *
             ((seq_lens_host[r] + pa::kLatentKeys - 1) / pa::kLatentKeys);
    }
    const int64_t cost = w * std::max(1570, 1300 * lanes);
    if (lanes <= sms && cost < best) {
      best = cost;
      W = w;
      G = lanes;
    }
    if (w > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (widest <= NR) break;  // one row tile each
  }
  const int grid = G * (int)std::min<int64_t>(W, sms / G);
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
  p.b_shift = p.B == 16 ? 4 : p.B == 32 ? 5 : 6;
  p.causal = causal;
  p.lanes = G;
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
