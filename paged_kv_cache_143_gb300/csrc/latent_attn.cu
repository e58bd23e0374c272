// latent_attn.cu — pa_latent_forward: attention in the absorbed form over the
// paged latent cache, decode tokens and chunks alike.
//
// Every query row (token, head) of a request scores the same keys [c ; k_r] and
// averages the same values c, so one pass over the request's cells serves all
// its rows: s = scale * (q_c . c + q_r . k_r), o = softmax(s) c, the softmax
// running over key tiles with a reference maximum and sum per row.
//
// What bounds it: a bf16 cell is (L + 64) * 2 bytes and each row spends
// 2 (2 L + 64) operations on it; up to about 64 rows per request that is less
// tensor time than the cell takes from HBM, so the design is laid out for streaming.
// Measured, 152 requests x 4096 keys, L 512, blocks of 64 (HBM's share of the time
// at 6783 GB/s 106 us; E4M3 59): 16 heads 118 us, 32 120, 64 128, 128 215 (there shared
// memory bounds: a 32-key tile takes 1450 cycles, 1250 of them the products' reads);
// E4M3 16 heads 83 us, 64 117 (2750 cycles a 64-key tile, 2400 of them reads).
// 160 decodes of 128 to 2048 keys x 32 heads: 57.0 us (35.3).
//
// One CTA per SM walks an equal share of all (row tile, key tile) pairs, a pass
// over a request counting as four tiles more than it has (pa::LatentParams). Both
// products run on the 5th-generation tensor cores:
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
//   warp 0      TMA producer (one lane): the key tiles into a ring of stages, and
//               the Q tile
//   warp 1      TMEM and, one lane, S, up to four tiles ahead (E4M3: two)
//   warp 2      one lane, PV. (One lane for both products spent a third of a
//               tile's time between the two batches of them.)
//   warp 3      the CTA's pieces, found once and handed to the others through a
//               ring of four; it also asks L2 for a coming piece's first cells
//   warps 4-7   softmax (S read as 16 x 256-bit fragments: a row in four lanes),
//               P to shared memory; then the output
//   warps 8-11  (E4M3) the query tile as E4M3 parts; at L 256 then the softmax of
//               the odd tiles, warps 4-7 that of the even ones
// The instruction cache is cold at launch and, once all SMs stream, a miss takes
// microseconds: S, PV and softmax run once on whatever memory holds while the
// first keys are on their way (S and O are overwritten by the first real products).
// The softmax warps of a group share nothing tile by tile (the two groups of E4M3
// pools hand the rows' references on). A warp that moves a row's
// reference maximum says so beside P; warp 2 then asks all four to rescale
// their dims of O before it issues that PV (rare: growth by more than 2^8).
// Every wait is bounded; a timeout sets the error word and the CTA unwinds.
//
// E4M3 pools: both products take the codes as they are stored (kind::f8f6f4),
// nothing is widened. The other operand is a sum of 8-bit numbers:
//   q 2^e = hi + lo in E4M3, 2^e bringing the row's largest magnitude to
//     [2^7, 2^8). A bf16 number has 8 significant bits and each part 4, so the sum
//     is exact down to half of E4M3's smallest step, 2^-17 of the row's maximum.
//   p s_n, the weight of key n of scale s_n, = three parts in E5M2 (3 bits each):
//     below 2^-9 of the weight off, or 2^-17 absolute. The reference maximum is
//     that of p s_n, placed at 2^7, so that is 2^-24 of the row's largest weight:
//     a long context's many small weights keep their share beside one large one.
//     (Two E4M3 parts would do for weights within 2^-8 of the largest, but lose
//     every weight below 2^-14 of it.)
// The parts of q are stacked in the rows of S (64, or 128 for 64 query rows),
// those of hi above those of lo, 8 or 16 a softmax warp: the keys are read once for
// both, and the thread that reads a row's hi scores reads its lo scores too. The
// rotary part of q and k stays bf16 and has S columns of its own (64 rows), since
// s_n does not apply to it.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include <cuda_fp8.h>

#include "latent_attn.h"
#include "mbar_poll.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "tc_ptx.cuh"

namespace pa {
namespace {

constexpr int kRope = 64;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;   // S buffers from column 256 on
constexpr uint32_t kTmemR = 384;   // E4M3: the rotary part of S from 384 on
constexpr int kMaxStages = 8, kPieces = 4;
constexpr float kNoKey = -1.f;     // as a partial's sum: the row sees none of its keys
// The reference maximum moves when it grows by more than 2^kRescaleLog2; weights
// of the maximum are placed at 2^kTargetLog2 (E5M2 weights must stay below 57344).
template <bool F8> constexpr float kRescaleLog2 = F8 ? 7.f : 8.f;
template <bool F8> constexpr float kTargetLog2 = F8 ? 7.f : 0.f;

template <int L, int NR, bool F8>
struct Smem {
  static constexpr int kThreads = F8 ? 384 : 256;
  static constexpr int KT = latent_tile_keys(L, F8);
  static constexpr int kChunk = KT * 128;             // 128 bytes of each row of a key tile
  static constexpr int kSBufs = F8 ? 2 : 4;           // S buffers of KT columns
  static constexpr int kM = F8 && NR > 32 ? 128 : 64; // rows of S: E4M3, hi and lo of q
  // E4M3: the warps that convert queries also take the softmax of odd tiles. With
  // weights in three parts it takes one group 2500 cycles a tile; at L 256 the
  // products take 1200 (152 x 4096 keys: 64 rows 103 us with one group, 84 with two,
  // 16 rows 79 and 66), at L 512 as long as the softmax (119 and 122)
  static constexpr bool kTwo = F8 && L == 256;
  static constexpr int kCols = F8 ? L / 128 : L / 64; // 128-byte chunks of a latent row
  // the latent chunks (E4M3: rows of hi and of lo), then the rotary part (64 rows
  // of S at most)
  static constexpr int kQChunk = (F8 ? 2 * NR : NR) * 128;
  static constexpr int kOffQR = kCols * kQChunk;
  static constexpr int kQBytes = kOffQR + (kM == 128 ? NR * 128 : kQChunk);
  static constexpr int kStage = (kCols + 1) * kChunk; // the last chunk is the rotary part
  // P of two tiles in 128-byte rows, a tile's part (bf16: all of it) in 64 bytes
  // of a row (bf16 with 64 keys: 128); part `i` of tile g starts at p_part
  static constexpr int kPartBytes = F8 ? KT : KT * 2;
  static constexpr int kPartsP = F8 ? 3 : 1;
  static constexpr int kPBytes = 2 * kPartsP * kPartBytes * NR;
  __host__ __device__ static constexpr int p_part(int g, int part) {
    const int u = (g & 1) * kPartsP + part;
    return kPartBytes == 128 ? u * NR * 128 : (u >> 1) * NR * 128 + (u & 1) * 64;
  }
  static constexpr int kTail = F8 ? 8192 : 2048;      // barriers, pieces, row statistics
  static constexpr int kFit = (232448 - 1024 - kTail - kQBytes - kPBytes) / kStage;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffP = kOffK + kStages * kStage;
  static constexpr int kOffTail = kOffP + kPBytes;
  static constexpr int kAlloc = kOffTail + kTail + 1024;  // the base is rounded up to 1024 B
  static_assert(kStages * KT >= 128 && kStages >= 3, "needs several key tiles in flight");
  static_assert(kAlloc <= 232448, "dynamic shared memory above the 227 KB per-block limit");
  static_assert(kOffK % 1024 == 0 && kOffP % 1024 == 0, "swizzled tiles start on 1024 bytes");
  // S reads at least 64 rows of Q: the rows past the tile's are whatever follows
  // in shared memory (their scores are never looked at)
  static_assert(kQBytes + 64 * 128 <= kAlloc - 1024, "Q over-read leaves the allocation");
};

// A CTA's part of one pass, as the roles need it.
struct Piece {
  int32_t r;           // request; -1: no more pieces
  int32_t k0, k1;      // key tiles [k0, k1)
  int32_t n_keys;      // keys any row of the tile sees (k1 is cut to it)
  int32_t rows;        // valid query rows of the tile
  int32_t slot;        // partial slot 0 / 1 of the CTA, or -1: the whole pass
  int32_t row;         // the tile's first row in q and out
  int32_t first;       // the same within the request; -1: every row sees n_keys
  int32_t sees;        // keys that the request's first token sees
};

template <bool F8>
struct Tail {
  uint64_t q_full, q_empty;
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t s_full[4], s_empty[4];
  uint64_t p_full[2], pv_done[2];
  uint64_t fix, fixed;           // O is to be rescaled for tile fix_tile; it has been
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t o_empty, final_mma;
  // two softmax groups, by warp: the reference after an even / odd tile is
  // there; the second group's sums of a piece are; and (all) 1 / sum is
  uint64_t m_full[4][2], sum_full[4][kPieces], l_full;
  Piece piece[kPieces];
  alignas(16) float alpha[2][kLatentRows];   // by tile: factors of the rows of a warp that asks
  alignas(16) float l[2][kLatentRows];       // by piece: 1 / sum
  alignas(16) float scale[F8 ? kMaxStages : 1][64];      // E4M3: of the stage's keys
  float q_scale[F8 ? kPieces : 1][F8 ? kLatentRows : 1]; // E4M3: 2^-e of the rows
  float m_ref[2][F8 ? kLatentRows : 1];                  // by tile: the rows' references
  float2 sums[F8 ? kPieces : 1][F8 ? kLatentRows : 1];            // (reference, sum) of a piece
  alignas(4) uint8_t ask[2][4];  // by tile: softmax warps that ask for a rescale
  int32_t fix_tile;
  int32_t cleared[2];            // by piece: the last one (+ 1) with a cell cleared
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Tail<true>) <= 8192 && sizeof(Tail<false>) <= 2048, "Tail overruns its slot");

template <bool F8>
__device__ __forceinline__ bool aborted(Tail<F8>* t) {
  return *reinterpret_cast<volatile int*>(&t->abort) != 0;
}

// 16 lanes x 32 columns as mma-style fragments: of each 8-column group i,
// r[4 i], r[4 i + 1] are columns 2 (lane % 4), + 1 of row lane / 4, and
// r[4 i + 2], r[4 i + 3] those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 16 lanes x 16 columns, and the same 32 columns on: thread t has the 16 of row
// t % 16 that start at column 32 (t / 16).
__device__ __forceinline__ void tmem_ld_16x2x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], 32;"
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

// Asks L2 for `bytes` contiguous bytes (address and size multiples of 16).
__device__ __forceinline__ void prefetch_l2(const void* gmem, unsigned bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(gmem), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Two fp32 to E4M3 (nearest even), x in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// Zeros in the place of infinities and NaN in the cells of a stage from row r0 on, by
// a warp.
template <bool F8, int KT, int kCols>
__device__ __noinline__ void clear_cells(uint8_t* stage, int r0) {
  constexpr uint32_t kField = F8 ? 0xFFu : 0xFFFFu, kOdd = F8 ? 0x7Fu : 0x7F80u;
#pragma unroll 1
  for (int i = r0 * kCols; i < KT * kCols; ++i) {
    uint32_t* at = reinterpret_cast<uint32_t*>(stage + (i % kCols) * KT * 128 + i / kCols * 128) +
                   (threadIdx.x & 31);
    const uint32_t w = *at;
    uint32_t keep = w;
#pragma unroll 1
    for (int b = 0; b < 32; b += F8 ? 8 : 16)
      if ((w >> b & kOdd) == kOdd) keep &= ~(kField << b);
    if (keep != w) *at = keep;
  }
}

// NaN in the place of O's elements of the rows that see a cell in [key0, key1) which
// is not finite in that dim (bf16 cells; all lanes of a warp, `dim` the lane's in the
// first block of 128). The cells are read again: this is rare.
template <int L, int NR>
__device__ __noinline__ void put_back(uint32_t tmem_o, const uint8_t* latent, const int32_t* table,
                                      int b_shift, int num_blocks, int dim, int key0, int key1,
                                      int first, int sees, int heads) {
  int32_t from[L / 128];  // the first such key, by block
#pragma unroll
  for (int b = 0; b < L / 128; ++b) from[b] = INT32_MAX;
#pragma unroll 1
  for (int key = key1 - 1; key >= key0; --key) {
    const int32_t listed = __ldg(table + (key >> b_shift));
    const int64_t id = listed < 0 || listed >= num_blocks ? 0 : listed;  // as the producer reads
    const int64_t cell = (id << b_shift) + (key & ((1 << b_shift) - 1));
    const uint16_t* c = reinterpret_cast<const uint16_t*>(latent) + cell * L + dim;
#pragma unroll
    for (int b = 0; b < L / 128; ++b)
      if ((c[b * 128] & 0x7F80u) == 0x7F80u) from[b] = key;
  }
#pragma unroll 1
  for (int i = 0; i < NR; i += 16) {
#pragma unroll
    for (int b = 0; b < L / 128; ++b) {
      uint32_t o[16];
      tmem_ld16(tmem_o + b * NR + i, o);
      tc::tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (sees + (int)((unsigned)(first + i + k) / (unsigned)heads) > from[b])
          o[k] = 0x7FC00000u;
      tmem_st16(tmem_o + b * NR + i, o);
    }
  }
  tc::tmem_wait_st();
}

// ------------------------------------------------------------ the flat space

// Sums of weights stop here. The host refuses batches that could come this far with
// a query_start_loc that only rises; one that goes back and forth on the device can,
// its requests overlapping, and is then taken for an empty batch.
constexpr int32_t kMaxWork = INT32_MAX;
__device__ __forceinline__ int32_t add_work(int32_t a, int32_t b) {
  return (int32_t)min((uint32_t)a + (uint32_t)b, (uint32_t)kMaxWork);
}

struct Request {
  int32_t q_begin, q_len, seq, rows, keys;  // query rows, key tiles
  int32_t weight;                           // passes * (skip + keys); 0 for one without work
};

// Reads request r; one whose device entries do not fit the buffers has no
// work (and is reported once).
template <int NR, int KT>
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
  // (within the host's bound on the sum, kMaxWork, for each request by itself)
  q.weight = (p.lanes == 1 ? tiles : (tiles + 1) / 2) * (p.skip + q.keys);
  return q;
}

template <int NR, int KT>
struct Walk {
  int32_t pos, end, base, r, lane;
  bool loaded;
  Request q;

  __device__ Walk(int32_t begin, int32_t stop, int32_t first_req, int32_t first_base,
                  int32_t in_group)
      : pos(begin), end(stop), base(first_base), r(first_req), lane(in_group), loaded(false), q{} {}

  __device__ bool next(const LatentParams& p, Piece& out) {
    if (pos >= end) return false;
    if (!loaded) {
      q = load_request<NR, KT>(p, r, false);
      loaded = true;
    }
    while (pos - base >= q.weight) {
      base += q.weight;
      if (++r >= p.R) return false;
      q = load_request<NR, KT>(p, r, false);
    }
    const unsigned off = pos - base, span = p.skip + q.keys;
    const int pass = (int)(off / span), tile = pass * p.lanes + lane;
    const int at = (int)(off - pass * span), stop = min((int)span, at + (end - pos));
    pos += stop - at;
    if (stop <= p.skip) return false;  // (the range ends before the pass's keys)
    out.r = r;
    out.k0 = max(0, at - p.skip);
    const int k1 = stop - p.skip;
    out.slot = out.k0 > 0 ? 0 : k1 < q.keys ? 1 : -1;
    out.row = q.q_begin * p.Hq + tile * NR;
    out.rows = max(0, min(NR, q.rows - tile * NR));  // 0: the pass has fewer tiles
    out.n_keys = q.seq;
    out.first = -1;
    out.sees = q.seq - q.q_len + 1;
    if (p.causal && q.q_len > 1 && out.rows > 0) {  // up to the last row's token
      out.first = tile * NR;
      out.n_keys = out.sees + (int)((unsigned)(out.first + out.rows - 1) / (unsigned)p.Hq);
    }
    out.k1 = out.rows > 0 ? min(k1, (out.n_keys + KT - 1) / KT) : out.k0;
    return true;
  }
};

template <int L, int NR, bool F8>
__global__ void __launch_bounds__(Smem<L, NR, F8>::kThreads, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_c,
                       const __grid_constant__ CUtensorMap tmap_r, const LatentParams p) {
  using S = Smem<L, NR, F8>;
  constexpr int kThreads = S::kThreads, kStages = S::kStages, kCols = S::kCols;
  constexpr int KT = S::KT, kChunk = S::kChunk, kSBufs = S::kSBufs;
  constexpr int kBlocks = L / 128;              // 128-dim blocks of O^T
  constexpr bool kWide = S::kM == 128;          // S: 16 rows of hi, their 16 of lo per warp
  constexpr int RT = F8 ? 1 : 2;                // query rows of a softmax thread
  constexpr int VT = kWide ? KT / 2 : KT / 4;   // and its scores of each
  constexpr int kWarpRows = F8 && !kWide ? 8 : 16;  // query rows of a softmax warp
  constexpr bool kTwo = S::kTwo;                // two softmax groups
  constexpr int kScoreWarps = NR / kWarpRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Tail<F8>* tail = reinterpret_cast<Tail<F8>*>(smem + S::kOffTail);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  // ---- the weights of the requests, summed by thread over consecutive ones (the
  // ring is still empty). What runs before the first copy is kept short: cold
  // instructions cost as much as cold data.
  int32_t* weights = reinterpret_cast<int32_t*>(smem + S::kOffK);
  const int per_thread = (p.R + kThreads - 1) / kThreads;
  {
    int32_t w = 0;
#pragma unroll 1
    for (int i = 0; i < per_thread; ++i) {
      const int r = threadIdx.x * per_thread + i;
      if (r < p.R) w = add_work(w, load_request<NR, KT>(p, r, cta == 0).weight);
    }
    weights[threadIdx.x] = w;
  }
  if (warp == 1) {
    tc::tmem_alloc(&tail->tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    mbar_init(&tail->q_full, F8 ? 4 : 1);  // E4M3: the warps that convert
    mbar_init(&tail->q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&tail->k_full[s], 1);
      mbar_init(&tail->k_empty[s], 1);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&tail->s_full[s], 1);
      mbar_init(&tail->s_empty[s], 4);  // the softmax warps
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tail->p_full[s], 4);   // one arrival per softmax warp
      mbar_init(&tail->pv_done[s], 1);
    }
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&tail->piece_full[s], 1);
      mbar_init(&tail->piece_empty[s], F8 ? 11 : 7);  // one arrival per reading warp
    }
    mbar_init(&tail->fix, 1);
    mbar_init(&tail->fixed, 4);
    mbar_init(&tail->o_empty, 4);
    mbar_init(&tail->final_mma, 2);
    if (kTwo) {
      for (int w = 0; w < 4; ++w) {
        for (int s = 0; s < 2; ++s) mbar_init(&tail->m_full[w][s], 1);
        for (int s = 0; s < kPieces; ++s) mbar_init(&tail->sum_full[w][s], 1);
      }
      mbar_init(&tail->l_full, 4);
    }
    tail->abort = 0;
    tail->cleared[0] = tail->cleared[1] = 0;
    fence_mbar_init();
  }
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tail->tmem;

  // waits end early where another role has given up (not those for what is in flight
  // when a role ends)
  auto wait_for = [&](uint64_t* bar, unsigned parity) {
    return mbar_wait_quiet(bar, parity, &tail->abort, p.err);
  };
  // the next piece (n-th of the CTA) for one thread; r < 0 at the end
  // (n = -1: a tile of nothing, for the instruction cache)
  auto piece = [&](int n, bool& ok) -> Piece {
    Piece pc{0, 0, 1, KT, 0, -1, 0, -1, 0};
    if (n < 0) return pc;
    ok = wait_for(&tail->piece_full[n % kPieces], (n / kPieces) & 1);
    if (ok)
      pc = tail->piece[n % kPieces];
    else
      pc.r = -1;
    return pc;
  };
  auto release = [&](int n) { mbar_arrive(&tail->piece_empty[n % kPieces]); };

  {
    if (warp == 0) {
      // --------------------------------------------------------- TMA producer
      // (one lane: a copy instruction with several lanes active costs about
      // 120 cycles a lane, and the ring then waits for its producer)
      if (tc::elect_one()) {
        tc::prefetch_tensormap(&tmap_c);
        tc::prefetch_tensormap(&tmap_r);
        if (!F8) tc::prefetch_tensormap(&tmap_q);
        int g = 0, queries = 0;    // key tiles so far; pieces whose Q is on its way
        int st = 0, phase = 1;     // stage, and the parity its emptying waits for
        bool ok = true;
        for (int n = 0;; ++n) {
          const Piece pc = piece(n, ok);
          if (pc.r < 0) break;
          const int32_t* table = p.block_tables + (int64_t)pc.r * p.max_blocks;
          // the Q tile as soon as the last piece's S are done; its keys need not
          // wait for that
          auto load_q = [&](bool may_wait) -> bool {
            if (F8 || queries > n) return true;
            if (n > 0) {
              uint64_t* bar = &tail->q_empty;
              if (may_wait) {
                if (!wait_for(bar, (n - 1) & 1)) return false;
              } else if (!mbar_test_wait(bar, (n - 1) & 1)) {
                return true;
              }
            }
            mbar_arrive_expect_tx(&tail->q_full, S::kQBytes);
            tc::tma_load_3d(smem, &tmap_q, 0, pc.row, 0, &tail->q_full);
            queries = n + 1;
            return true;
          };
          // physical block of part i of tile j (a tile is 1, 2 or 4 parts of
          // min(block, tile) keys, each in one block)
          const int part_shift = min(p.b_shift, KT == 64 ? 6 : 5), parts = KT >> part_shift;
          auto fetch = [&](int j, int (&id)[KT / 16]) {
#pragma unroll
            for (int i = 0; i < KT / 16; ++i) {
              const int key = j * KT + (i << part_shift);
              id[i] = i < parts && j < pc.k1 && key < pc.n_keys ? __ldg(table + (key >> p.b_shift))
                                                                 : 0;
            }
          };
          int ids[KT / 16], next[KT / 16];
          fetch(pc.k0, ids);
          load_q(false);
          for (int j = pc.k0; j < pc.k1; ++j, ++g) {
            fetch(j + 1, next);
#pragma unroll
            for (int i = 0; i < KT / 16; ++i)
              if (ids[i] < 0 || ids[i] >= p.num_blocks) {
                raise_error(p.err, kErrBounds);
                ids[i] = 0;  // a valid block; the output is then unspecified
              }
            if (g >= kStages && !mbar_test_wait(&tail->k_empty[st], phase)) {
              // the stage may be waiting for products that wait for this Q
              ok = load_q(true) && wait_for(&tail->k_empty[st], phase) && !aborted(tail);
              if (!ok) break;
            }
            load_q(false);
            uint8_t* dst = smem + S::kOffK + st * S::kStage;
            uint64_t* bar = &tail->k_full[st];
            constexpr int kRowBytes = (kCols + 1) * 128 + (F8 ? 4 : 0);
            if (parts == 1) {
              const int y = (ids[0] << p.b_shift) + ((j * KT) & ((1 << p.b_shift) - 1));
              mbar_arrive_expect_tx(bar, KT * kRowBytes);
              tc::tma_load_3d(dst, &tmap_c, 0, y, 0, bar);
              tc::tma_load_2d(dst + kCols * kChunk, &tmap_r, 0, y, bar);
              if (F8) bulk_g2s(tail->scale[st], p.scales + y, KT * 4, bar);
            } else {
              const int live =
                  min(parts, (pc.n_keys - j * KT + (1 << part_shift) - 1) >> part_shift);
              mbar_arrive_expect_tx(bar, (live << part_shift) * kRowBytes);
#pragma unroll
              for (int i = 0; i < KT / 16; ++i) {
                if (i >= live) break;
                const int y = ids[i] << p.b_shift, at = (i << part_shift) * 128;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                  tc::tma_load_3d(dst + c * kChunk + at, &tmap_c, 0, y, c, bar);
                tc::tma_load_2d(dst + kCols * kChunk + at, &tmap_r, 0, y, bar);
                if (F8)
                  bulk_g2s(tail->scale[st] + (i << part_shift), p.scales + y, 4 << part_shift, bar);
              }
            }
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
#pragma unroll
            for (int i = 0; i < KT / 16; ++i) ids[i] = next[i];
          }
          ok = ok && load_q(true);
          if (!ok) break;
          release(n);
        }
        // every issued copy lands before the CTA may leave
        if (!ok) tail->abort = 1;
        if (queries > 0) mbar_wait_quiet(&tail->q_full, (queries - 1) & 1, nullptr, p.err);
        for (int i = max(0, g - kStages); i < g; ++i)
          mbar_wait_quiet(&tail->k_full[i % kStages], (i / kStages) & 1, nullptr, p.err);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------------- S
      if (tc::elect_one()) {
        constexpr uint32_t idesc = tc::idesc_16bit_f32(64, KT, false, false, false);
        constexpr uint32_t idesc8 = tc::idesc_e4m3_f32(S::kM, KT);
        const uint64_t q_desc = tc::smem_desc_sw128(smem, 16, 1024);
        const uint64_t k_desc = tc::smem_desc_sw128(smem + S::kOffK, 16, 1024);
        int g = 0, st = 0, phase = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = -1;; ++n) {
          const bool live = n >= 0;
          const Piece pc = piece(n, ok);
          if (pc.r < 0) break;
          if (live && !(ok = wait_for(&tail->q_full, n & 1))) break;
#pragma unroll 1
          for (int j = pc.k0; j < pc.k1; ++j) {
            const int buf = g % kSBufs;
            ok = !live ||
                 ((g < kSBufs || wait_for(&tail->s_empty[buf], (g / kSBufs - 1) & 1)) &&
                  wait_for(&tail->k_full[st], phase));
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t ks = tc::desc_at(k_desc, st * S::kStage);
            const uint32_t d = tmem + kTmemS + buf * KT, dr = F8 ? tmem + kTmemR + buf * KT : d;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_bf16_ss(dr, tc::desc_at(q_desc, S::kOffQR + k * 32),
                              tc::desc_at(ks, kCols * kChunk + k * 32), idesc, k > 0);
#pragma unroll
            for (int k = 0; k < kCols * 4; ++k) {
              const uint64_t qa = tc::desc_at(q_desc, (k >> 2) * S::kQChunk + (k & 3) * 32);
              const uint64_t kb = tc::desc_at(ks, (k >> 2) * kChunk + (k & 3) * 32);
              if (F8)
                tc::mma_e4m3_ss(d, qa, kb, idesc8, k > 0);
              else
                tc::mma_bf16_ss(d, qa, kb, idesc, true);
            }
            if (!live) break;
            tc::mma_commit(&tail->s_full[buf]);
            ++g;
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          if (!live) continue;
          tc::mma_commit(&tail->q_empty);
          release(n);
        }
        if (!ok) tail->abort = 1;
        tc::mma_commit(&tail->final_mma);
        mbar_wait_quiet(&tail->final_mma, 0, nullptr, p.err);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------------ PV
      if (tc::elect_one()) {
        constexpr uint32_t idesc = tc::idesc_16bit_f32(128, NR, true, false, false);
        // A the codes, MN-major (bit 15); B E5M2 (type 1 in bits 10..)
        constexpr uint32_t idesc8 = tc::idesc_e4m3_f32(128, NR) | (1u << 15) | (1u << 10);
        const uint64_t p_desc = tc::smem_desc_sw128(smem + S::kOffP, 16, 1024);
        const uint64_t v_desc = tc::smem_desc_sw128(smem + S::kOffK, kChunk, 1024);
        int g = 0, st = 0, fixes = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = -1;; ++n) {
          const bool live = n >= 0;
          const Piece pc = piece(n, ok);
          if (pc.r < 0) break;
#pragma unroll 1
          for (int j = pc.k0; j < pc.k1; ++j) {
            if (live && !(ok = wait_for(&tail->p_full[g & 1], (g >> 1) & 1))) break;
            if (j == pc.k0) {
              // the first product of a piece overwrites O: the last piece is out
              if (n > 0 && !(ok = wait_for(&tail->o_empty, (n - 1) & 1))) break;
            } else if (*reinterpret_cast<volatile uint32_t*>(&tail->ask[g & 1][0]) != 0) {
              // rows of this tile have a new reference: O, complete up to the
              // tile before, is rescaled first
              *reinterpret_cast<volatile int32_t*>(&tail->fix_tile) = g;
              ok = wait_for(&tail->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
              mbar_arrive(&tail->fix);
              ok = ok && wait_for(&tail->fixed, fixes & 1);
              if (!ok) break;
              ++fixes;
            }
            tc::fence_after_sync();
            const uint64_t vs = tc::desc_at(v_desc, st * S::kStage);
            const bool add = j > pc.k0;
            // a part of the weights after the other (bf16: one), 32 bytes of keys at
            // a time: 16 bf16 or 32 codes
#pragma unroll
            for (int m = 0; m < kBlocks; ++m)
#pragma unroll
              for (int part = 0; part < S::kPartsP; ++part)
#pragma unroll
                for (int k = 0; k < S::kPartBytes / 32; ++k) {
                  const uint64_t pb = tc::desc_at(
                      p_desc, ((g & 1) ? S::p_part(1, part) : S::p_part(0, part)) + k * 32);
                  const bool acc = add || part > 0 || k > 0;
                  if (F8)
                    tc::mma_e4m3_ss(tmem + m * NR, tc::desc_at(vs, m * kChunk + k * 32 * 128), pb,
                                    idesc8, acc);
                  else
                    tc::mma_bf16_ss(tmem + m * NR,
                                    tc::desc_at(vs, 2 * m * kChunk + k * 16 * 128), pb, idesc, acc);
                }
            if (!live) break;
            tc::mma_commit(&tail->k_empty[st]);
            tc::mma_commit(&tail->pv_done[g & 1]);
            ++g;
            if (++st == kStages) st = 0;
          }
          if (!ok) break;
          if (live) release(n);
        }
        if (!ok) tail->abort = 1;
        tc::mma_commit(&tail->final_mma);
        mbar_wait_quiet(&tail->final_mma, 0, nullptr, p.err);
      }
      __syncwarp();
    } else if (warp == 3) {
      // -------------------------------------------------------------- pieces
      // This group's range [begin, end) of the flat space, from the running sum of
      // the weights, and the request that holds its first tile.
      const int group = cta / p.lanes, in_group = cta - group * p.lanes;
      const int groups = gridDim.x / p.lanes;
      constexpr int kEach = kThreads / 32;
      int32_t mine = 0;
#pragma unroll 1
      for (int i = 0; i < kEach; ++i) mine = add_work(mine, weights[lane * kEach + i]);
      int32_t upto = mine;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = add_work(upto, y);
      }
      int W = __shfl_sync(0xffffffffu, upto, 31);
      if (W == kMaxWork) {
        if (cta == 0 && lane == 0) raise_error(p.err, kErrBounds);
        W = 0;
      }
      const unsigned Q = max(1u, ((unsigned)W + groups - 1) / groups);
      const int begin = (int)min((unsigned)W, group * Q), end = (int)min((unsigned)W, begin + Q);
      // the lane, its thread's sum, then the request
      const int owner = __popc(__ballot_sync(0xffffffffu, upto <= begin)) & 31;
      int base = __shfl_sync(0xffffffffu, upto - mine, owner);
      int r = owner * kEach;
#pragma unroll 1
      while (r < owner * kEach + kEach - 1 && base + weights[r] <= begin) base += weights[r++];
      r *= per_thread;
      __syncwarp();
      Walk<NR, KT> walk(begin, end, r, base, in_group);
      Piece pc;
      Request q{};
      bool first = true;
      int n = 0;
      bool ok = true;
      for (bool more = true; ok && more;) {
        more = walk.next(p, pc);
        if (first) {  // the request that holds this group's first tile
          first = false;
          q = walk.q;
          base = walk.base;
        }
        if (!more) {
          pc.r = -1;
        } else if (pc.k0 >= pc.k1) {
          // no row of the tile sees these keys: the join skips them
          if (pc.slot >= 0) {
            float2* ml = p.part_ml + (int64_t)(2 * cta + pc.slot) * NR;
            for (int i = lane; i < NR; i += 32) ml[i] = make_float2(-INFINITY, kNoKey);
          }
          continue;
        }
        if (n >= kPieces)
          ok = __all_sync(0xffffffffu, wait_for(&tail->piece_empty[n % kPieces],
                                                 (n / kPieces - 1) & 1));
        if (!ok) break;
        // (the weights lie where the first copies will go)
        if (n == 0) tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tail->piece[n % kPieces] = pc;
          mbar_arrive(&tail->piece_full[n % kPieces]);
        }
        __syncwarp();
        if (n == 0) {
          // the pass cut at this group's start, for the join
          LatentJoin join{};
          if (begin < end) {
            const int at = begin - base, pass = at / (p.skip + q.keys);
            // the pass's first tile
            const unsigned a = begin - (at - pass * (p.skip + q.keys)) + p.skip;
            const int row0 = (pass * p.lanes + in_group) * NR;
            if ((unsigned)begin > a && row0 < q.rows) {
              join.rows = min(q.rows - row0, NR);
              join.cut = group - (int)(a / Q) - 1;
              join.pieces = (int32_t)((a + q.keys - 1) / Q - a / Q) + 1;
              join.out_row = (int64_t)q.q_begin * p.Hq + row0;
            }
          }
          if (lane == 0) p.joins[cta] = join;
        }
        // a later piece's first tiles and queries, towards L2 while the ones
        // before are worked on (16 keys a lane; E4M3: queries of the first one too,
        // which are read in two rounds)
        if (more && (n > 0 || F8)) {
          const int key = pc.k0 * KT + lane * 16;
          if (n > 0 && lane < 8 && key < pc.n_keys) {
            const int32_t id = __ldg(p.block_tables + (int64_t)pc.r * p.max_blocks +
                                     (key >> p.b_shift));
            if (id >= 0 && id < p.num_blocks) {
              const int64_t cell = ((int64_t)id << p.b_shift) + (key & ((1 << p.b_shift) - 1));
              prefetch_l2(p.latent + cell * L * (F8 ? 1 : 2), 16 * L * (F8 ? 1 : 2));
              prefetch_l2(p.rope + cell * kRope * 2, 16 * kRope * 2);
            }
          } else if (lane == 8) {
            prefetch_l2(reinterpret_cast<const uint8_t*>(p.q) + (int64_t)pc.row * (L + kRope) * 2,
                        pc.rows * (L + kRope) * 2);
          }
        }
        ++n;
      }
      if (!ok && lane == 0) tail->abort = 1;
      __syncwarp();
    } else {
      // ---------------------------------------------------- softmax and output
      const int w4 = warp & 3;
      const bool second = F8 && warp >= 8;       // the group of the odd tiles
      const bool scores = w4 < kScoreWarps;
      int row[RT];                               // the thread's rows of the tile
#pragma unroll
      for (int t = 0; t < RT; ++t)
        row[t] = w4 * kWarpRows + (kWide ? lane & 15 : t * 8 + (lane >> 2));
      // the key of the tile that score i of a thread belongs to; a row is in the
      // threads whose numbers differ in kRowLanes
      constexpr int kRowLanes = kWide ? 16 : 3;
      auto key_of = [&](int i) {
        return kWide ? (lane >> 4) * 32 + i : (i >> 1) * 8 + 2 * (lane & 3) + (i & 1);
      };
      const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
      uint8_t* ps = smem + S::kOffP;
      const int tid = threadIdx.x & 127;
      int fixes = 0;
      // this warp's dims of O times the new factors of the rows that ask
      auto rescale = [&]() {
        tc::fence_after_sync();
        const int slot = *reinterpret_cast<volatile int32_t*>(&tail->fix_tile) & 1;
        const uint32_t asked = *reinterpret_cast<volatile uint32_t*>(&tail->ask[slot][0]);
#pragma unroll 1
        for (int c = 0; c < kBlocks * NR; c += 16) {
          const int r = c % NR;  // the rows of softmax warp r / kWarpRows (and the next)
          if (((asked >> (r / kWarpRows * 8)) & (kWarpRows == 8 ? 0xFFFF : 0xFF)) == 0) continue;
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
      // Waits for a barrier, doing the rescales that are asked for meanwhile (warps
      // 4-7: they hold all lanes of O between them).
      auto wait = [&](uint64_t* bar, int parity) -> bool {
        WaitLimit limit;
#pragma unroll 1
        do {
#pragma unroll 1
          for (unsigned i = 0; i < kTries; ++i) {
            if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity & 1))) return true;
            if (!second && __all_sync(0xffffffffu, mbar_test_wait(&tail->fix, fixes & 1)))
              rescale();
          }
        } while (!__any_sync(0xffffffffu, limit.over(&tail->abort, p.err)));
        return false;
      };
      // E4M3: the rows of the piece's query tile as two parts (warps 8-11)
      auto convert = [&](const Piece& pc, int n) {
        constexpr int kPer = L / 32;             // dims of a lane: 16 or 8
        // Four rows of a warp on their way at a time: once the keys stream, a load takes
        // microseconds (12 long contexts x 64 heads: two rows at a time 118.5 us, four
        // 101.6; eight 103.2, for the code that is fetched cold)
        constexpr int kBatch = 4;
#pragma unroll 1
        for (int i0 = 0; i0 < NR / 4; i0 += kBatch) {
          uint4 v[kBatch][kPer / 8], rot[kBatch / 4];  // rot: 8 lanes a row
          const __nv_bfloat16* src = p.q + (int64_t)pc.row * (L + kRope);
          auto piece_of = [&](int row, int dim) {
            return __ldg(reinterpret_cast<const uint4*>(src + (int64_t)row * (L + kRope) + dim));
          };
          // (rows past the tile's are zeros)
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int row = (i0 + b) * 4 + w4;
#pragma unroll
            for (int k = 0; k < kPer / 8; ++k)
              v[b][k] = row < pc.rows ? piece_of(row, lane * kPer + k * 8)
                                      : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < kBatch / 4; ++u) {
            const int row = (i0 + u * 4 + (lane >> 3)) * 4 + w4;
            rot[u] = row < pc.rows ? piece_of(row, L + (lane & 7) * 8) : make_uint4(0, 0, 0, 0);
          }
          // a softmax warp's rows of hi, then of lo
          auto hi_row = [&](int row) { return row / kWarpRows * 2 * kWarpRows + row % kWarpRows; };
#pragma unroll
          for (int u = 0; u < kBatch / 4; ++u) {
            const int row = (i0 + u * 4 + (lane >> 3)) * 4 + w4, at = kWide ? row : hi_row(row);
            *reinterpret_cast<uint4*>(smem + S::kOffQR + at * 128 +
                                      (((lane & 7) ^ (at & 7)) << 4)) = rot[u];
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int row = (i0 + b) * 4 + w4;
            float f[kPer], amax = 0.f;
#pragma unroll
            for (int k = 0; k < kPer / 8; ++k) bf16x8_to_f32(v[b][k], f + 8 * k);
#pragma unroll
            for (int k = 0; k < kPer; ++k) amax = fmaxf(amax, fabsf(f[k]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // 2^e brings the largest magnitude to [2^7, 2^8), if it is 2^-119 at least
            // (2^-e is kept a normal number); exact
            const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            const int e = amax > 0.f ? min(126, 7 - ex) : 0;
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            uint32_t hi[kPer / 4], lo[kPer / 4];
#pragma unroll
            for (int k = 0; k < kPer / 4; ++k) {
              hi[k] = lo[k] = 0u;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = f[4 * k + 2 * h] * up, y = f[4 * k + 2 * h + 1] * up;
                const uint32_t code = e4m3_pair(x, y);
                float hx, hy;
                e4m3x2_to_f32((uint16_t)code, hx, hy);
                hi[k] |= code << (16 * h);
                lo[k] |= e4m3_pair(x - hx, y - hy) << (16 * h);
              }
            }
            const int qrow = hi_row(row), lrow = qrow + kWarpRows;
            const int block = lane * kPer / 128, byte = lane * kPer % 128;
            auto place = [&](int off, int at) {
              return smem + off + at * 128 + (((byte >> 4) ^ (at & 7)) << 4) + (byte & 15);
            };
            uint8_t* dh = place(block * S::kQChunk, qrow);
            uint8_t* dl = place(block * S::kQChunk, lrow);
            if constexpr (kPer == 16) {
              *reinterpret_cast<uint4*>(dh) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(dl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            } else {
              *reinterpret_cast<uint2*>(dh) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(dl) = make_uint2(lo[0], lo[1]);
            }
            if (lane == 0)
              // (an infinity saturates as a code: the row's scores are NaN by its scale)
              tail->q_scale[n % kPieces][row] =
                  __uint_as_float(ex == 128 ? 0x7FC00000u : (uint32_t)(127 - e) << 23);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->q_full);
      };
      int g = second ? 1 : 0;  // tiles so far (the tile of nothing: one of the group's)
      bool ok = true;
#pragma unroll 1
      for (int n = -1;; ++n) {
        const bool live = n >= 0;
        const Piece pc = piece(n, ok);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || pc.r < 0) break;
        if constexpr (F8) {
          if (second && live) {
            if (n > 0 && !(ok = wait(&tail->q_empty, n - 1))) break;
            convert(pc, n);
          }
          if (second && !kTwo) {
            if (live && lane == 0) release(n);
            continue;
          }
        }
        int lim[RT];                 // keys the rows see
        float m[RT], l[RT], qs[RT];  // reference (log2), sum; E4M3: 2^-e of the query
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          lim[t] = !scores || row[t] >= pc.rows ? 0
                   : pc.first < 0
                       ? pc.n_keys
                       : pc.sees + (int)((unsigned)(pc.first + row[t]) / (unsigned)p.Hq);
          m[t] = -INFINITY;
          l[t] = 0.f;
          qs[t] = 1.f;
        }
        const int lim_min = RT == 2 ? min(lim[0], lim[RT - 1]) : lim[0];
#pragma unroll 1
        for (int j = pc.k0; j < pc.k1; ++j) {
          if (kTwo && (g & 1) != (int)second) {  // the other group's tile
            ++g;
            continue;
          }
          float x[RT][VT];           // of keys key_of(0), ..
          float alpha[RT];
#pragma unroll
          for (int t = 0; t < RT; ++t) alpha[t] = 1.f;
          float sc[VT];              // E4M3: scales of those keys
          const int key0 = j * KT, buf = g % kSBufs;
          // (warps without rows wait too: all four release S, so that none can fall
          // two phases of s_full behind, where a parity says nothing)
          if (live && !(ok = wait(&tail->s_full[buf], g / kSBufs))) break;
          bool p_free = false;
          // rows of a chunk hide keys of this tile that others see; scores there that
          // are no numbers
          const bool hiding = pc.first >= 0 && key0 + KT > pc.sees;
          bool odd = false;
          if (scores) {
            // (a test of a barrier answers after about 200 cycles beside the products'
            // reads of shared memory: they are asked ahead of their use)
            bool keys_in = true;
            if constexpr (F8) keys_in = mbar_test_wait(&tail->k_full[g % kStages],
                                                       (g / kStages) & 1);
            tc::fence_after_sync();
            uint32_t sr[kWide ? KT : KT / 2];
            const float* s = reinterpret_cast<const float*>(sr);
            const uint32_t ts = tmem + kTmemS + buf * KT + lanes;
            const uint32_t tr = tmem + kTmemR + buf * KT + lanes;
#pragma unroll
            for (int c = 0; c < KT; c += 32) {
              if constexpr (kWide) {  // 16 columns of hi, of lo
                tmem_ld_16x2x16(ts + c / 2, sr + c);
                tmem_ld_16x2x16(ts + c / 2 + (16u << 16), sr + c + 16);
              } else {
                tmem_ld_16x32(ts + c, sr + c / 2);
              }
            }
            if constexpr (F8) {
              // (the stage's scales came with its keys)
              if (live && !__all_sync(0xffffffffu, keys_in) &&
                  !(ok = wait(&tail->k_full[g % kStages], g / kStages)))
                break;
              uint32_t rr[KT / 2];
              const float* rs = reinterpret_cast<const float*>(rr);
              if constexpr (kWide) {
                tmem_ld_16x2x16(tr, rr);
                tmem_ld_16x2x16(tr + 16, rr + 16);
              } else {
#pragma unroll
                for (int c = 0; c < KT; c += 32) tmem_ld_16x32(tr + c, rr + c / 2);
              }
              if (j < pc.k0 + (kTwo ? 2 : 1)) qs[0] = tail->q_scale[n & (kPieces - 1)][row[0]];
              const float* st = tail->scale[g % kStages];
              if constexpr (kWide) {
#pragma unroll
                for (int i = 0; i < VT; i += 4)
                  *reinterpret_cast<float4*>(sc + i) =
                      *reinterpret_cast<const float4*>(st + key_of(i));
              } else {
#pragma unroll
                for (int i = 0; i < VT; i += 2)
                  *reinterpret_cast<float2*>(sc + i) =
                      *reinterpret_cast<const float2*>(st + key_of(i));
              }
              if (key0 + KT > pc.n_keys) {  // unwritten cells' scales may be anything
#pragma unroll
                for (int i = 0; i < VT; ++i)
                  if (key0 + key_of(i) >= pc.n_keys) sc[i] = 0.f;
              }
              tc::tmem_wait_ld();
              if constexpr (kWide) {
#pragma unroll
                for (int i = 0; i < VT; ++i) {
                  const int a = (i & 16) * 2 + (i & 15);
                  x[0][i] = fmaf((s[a] + s[a + 16]) * qs[0], sc[i], rs[i]);
                }
              } else {
#pragma unroll
                for (int i = 0; i < VT; ++i) {
                  const int a = (i >> 1) * 4 + (i & 1);
                  x[0][i] = fmaf((s[a] + s[a + 2]) * qs[0], sc[i], rs[a]);
                }
              }
            } else {
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < VT; ++i) {
                x[0][i] = s[(i >> 1) * 4 + (i & 1)];
                x[RT - 1][i] = s[(i >> 1) * 4 + (i & 1) + 2];
              }
            }
            tc::fence_before_sync();
            if (lane == 0 && live) mbar_arrive(&tail->s_empty[buf]);
            // (not for 64 bf16 rows: there PV(g - 2) is rarely done by now; 1.3% slower)
            if ((F8 || NR <= 32) && g >= 2)
              p_free = mbar_test_wait(&tail->pv_done[g & 1], ((g >> 1) - 1) & 1);
            bool m_there = false;
            if constexpr (kTwo) {
              if (g > 0)
                m_there = mbar_test_wait(&tail->m_full[w4][(g - 1) & 1], ((g - 1) >> 1) & 1);
            }
            if (key0 + KT > lim_min) {
              if (hiding) {
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                  float sum = 0.f;
#pragma unroll
                  for (int i = 0; i < VT; ++i)  // (past n_keys lies anything)
                    sum += key0 + key_of(i) < pc.n_keys ? x[t][i] : 0.f;
                  odd |= lim[t] > 0 && !(fabsf(sum) < INFINITY);
                }
              }
#pragma unroll
              for (int i = 0; i < VT; ++i) {
                const int key = key0 + key_of(i);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                  if (key >= lim[t]) x[t][i] = -INFINITY;
              }
            }
            // the row's maximum (E4M3: of the weight p s, s by its exponent)
            float top[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              float y[VT];
#pragma unroll
              for (int i = 0; i < VT; ++i)
                // (2^23 + n as a float holds n in its low bits)
                y[i] = F8 ? fmaf(x[t][i], p.scale_log2,
                                 __uint_as_float((__float_as_uint(sc[i]) >> 23) | 0x4B000000u) -
                                     8388735.f)
                          : x[t][i];
              top[t] = fmax3(fmax3(y[0], y[1], y[2]), fmax3(y[3], y[4], y[5]), fmaxf(y[6], y[7]));
#pragma unroll
              for (int i = 8; i < VT; i += 8)
                top[t] = fmax3(top[t], fmax3(y[i], y[i + 1], fmaxf(y[i + 2], y[i + 3])),
                               fmax3(y[i + 4], y[i + 5], fmaxf(y[i + 6], y[i + 7])));
            }
#pragma unroll
            for (int o = 1; o <= kRowLanes; o <<= 1)
              if (o & kRowLanes)
#pragma unroll
              for (int t = 0; t < RT; ++t)
                top[t] = fmaxf(top[t], __shfl_xor_sync(0xffffffffu, top[t], o));
            float own[RT];                 // the reference that l is kept by
            if constexpr (kTwo) {
              // the tile before is the other group's: its warp of the same rows hands
              // over the reference (waited for across pieces too, so that neither
              // group can fall two tiles behind)
              own[0] = m[0];
              if (live && g > 0 && !__all_sync(0xffffffffu, m_there) &&
                  !(ok = wait(&tail->m_full[w4][(g - 1) & 1], (g - 1) >> 1)))
                break;
              m[0] = j > pc.k0 ? tail->m_ref[(g - 1) & 1][row[0]] : -INFINITY;
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              if (!F8) top[t] *= p.scale_log2;
              // the reference moves only when it grows by more than 2^kRescaleLog2
              // (any reference gives the same softmax)
              if (m[t] == -INFINITY) {
                m[t] = top[t];
              } else if (top[t] > m[t] + kRescaleLog2<F8>) {
                alpha[t] = ex2_ftz(m[t] - top[t]);
                m[t] = top[t];
              }
              if constexpr (kTwo) {
                if ((lane & kRowLanes) == 0) tail->m_ref[g & 1][row[0]] = m[0];
                __syncwarp();
                if (lane == 0 && live) mbar_arrive(&tail->m_full[w4][g & 1]);
              }
              const float neg = m[t] == -INFINITY ? 0.f : kTargetLog2<F8> - m[t];
              float sum[2] = {0.f, 0.f};
#pragma unroll
              for (int i = 0; i < VT; ++i) {
                x[t][i] = ex2_ftz(fmaf(x[t][i], p.scale_log2, neg));
                sum[i & 1] += x[t][i];
              }
              const float keep = !kTwo ? alpha[t] : own[t] == m[t] ? 1.f : ex2_ftz(own[t] - m[t]);
              l[t] = l[t] * keep + (sum[0] + sum[1]);
            }
          }
          if (!scores && lane == 0 && live) mbar_arrive(&tail->s_empty[buf]);
          // PV(g - 2) has read this half of P, and what was published with it
          if (g >= 2 && !__all_sync(0xffffffffu, p_free) &&
              !(ok = wait(&tail->pv_done[g & 1], (g >> 1) - 1)))
            break;
          if (scores) {
            if constexpr (F8) {
              // weights p s in three parts, a byte a key: an f16 number's high byte is
              // its E5M2 truncation, so a part is the high byte after half a step is
              // added to the magnitude, and what is left is exact in f16. (A NaN, 0x7FFF,
              // becomes zeros: a hidden key's scale may be one; a row that sees it is NaN
              // by its sum.)
              uint8_t* prow = ps + row[0] * 128 + (kWide ? 0 : (lane & 3) * 2);
              uint32_t bytes[3][VT / 4];  // wide: the codes of 4 keys each
#pragma unroll
              for (int i = 0; i < VT / 2; ++i) {
                __half2 h = __floats2half2_rn(x[0][2 * i] * sc[2 * i],
                                              x[0][2 * i + 1] * sc[2 * i + 1]);
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                  const uint32_t code =
                      (*reinterpret_cast<const uint32_t*>(&h) + 0x00800080u) & 0xFF00FF00u;
                  h = __hsub2(h, *reinterpret_cast<const __half2*>(&code));
                  if constexpr (kWide) {
                    bytes[part][i >> 1] =
                        (i & 1) ? __byte_perm(bytes[part][i >> 1], code, 0x7531) : code;
                  } else {
                    const int off = (g & 1) ? S::p_part(1, part) : S::p_part(0, part);
                    const int gran = (off >> 4 & 7) + (i >> 1);  // 16 keys a granule
                    *reinterpret_cast<uint16_t*>(prow + (off & ~127) + (i & 1) * 8 +
                                                 ((gran ^ (row[0] & 7)) << 4)) =
                        (uint16_t)__byte_perm(code, 0u, 0x4431);
                  }
                }
              }
              if constexpr (kWide) {
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const int off = (g & 1) ? S::p_part(1, part) : S::p_part(0, part);
                    const int gran = (off >> 4 & 7) + (lane >> 4) * 2 + u;
                    *reinterpret_cast<uint4*>(prow + (off & ~127) + ((gran ^ (row[0] & 7)) << 4)) =
                        make_uint4(bytes[part][4 * u], bytes[part][4 * u + 1],
                                   bytes[part][4 * u + 2], bytes[part][4 * u + 3]);
                  }
              }
            } else {
              const int mi = lane >> 3;  // the 8x8 matrix whose row this lane addresses
              const int prow = w4 * 16 + (mi & 1) * 8 + (lane & 7);
              const int off = (g & 1) ? S::p_part(1, 0) : S::p_part(0, 0);
#pragma unroll
              for (int i = 0; i < KT / 16; ++i) {
                const int gran = (off >> 4 & 7) + 2 * i + (mi >> 1);
                stmatrix_x4(ps + prow * 128 + (off & ~127) + ((gran ^ (prow & 7)) << 4),
                            pack_bf16(x[0][4 * i], x[0][4 * i + 1]),
                            pack_bf16(x[RT - 1][4 * i], x[RT - 1][4 * i + 1]),
                            pack_bf16(x[0][4 * i + 2], x[0][4 * i + 3]),
                            pack_bf16(x[RT - 1][4 * i + 2], x[RT - 1][4 * i + 3]));
              }
            }
          }
          const bool ask = __any_sync(0xffffffffu, alpha[0] < 1.f || alpha[RT - 1] < 1.f);
          // (8 rows a warp: a rescale takes the rows of two, either may have asked)
          if (scores && (ask || kWarpRows == 8) && (lane & kRowLanes) == 0) {
#pragma unroll
            for (int t = 0; t < RT; ++t) tail->alpha[g & 1][row[t]] = alpha[t];
          }
          if (lane == 0) tail->ask[g & 1][w4] = ask;
          if (__builtin_expect(hiding && __any_sync(0xffffffffu, odd), 0)) {  // rare
            // A later token's cell may not be finite, and 0 times it then a NaN: zeros
            // keep it from the rows that hide it. Its score is no number for any row. One
            // that sees it is NaN by that or, at -inf (no E4M3 code gives that), gets
            // 0 times the element when it is written (put_back). Cells before the
            // tile's first row's limit are seen by all rows and stay.
            if (live && !(ok = wait(&tail->k_full[g % kStages], g / kStages))) break;
            const int seen = pc.sees + (int)((unsigned)pc.first / (unsigned)p.Hq);
            clear_cells<F8, KT, kCols>(smem + S::kOffK + (g % kStages) * S::kStage,
                                       max(0, seen - key0));
            if (!F8 && lane == 0)
              *reinterpret_cast<volatile int32_t*>(&tail->cleared[n & 1]) = n + 1;
          }
          if (key0 + KT > pc.n_keys) {
            // the tile holds keys past the last visible one (unloaded blocks,
            // unwritten cells): zero them, so that P = 0 never meets a NaN (S of
            // this tile has read them)
            // the thread's chunk is (tid / 8) % kCols
            uint8_t* ks = smem + S::kOffK + (g % kStages) * S::kStage +
                          ((tid >> 3) & (kCols - 1)) * kChunk + (tid & 7) * 16;
            for (int i = pc.n_keys - key0 + tid / (8 * kCols); i < KT; i += 16 / kCols)
              *reinterpret_cast<uint4*>(ks + i * 128) = make_uint4(0, 0, 0, 0);
          }
          if (!kTwo && j == pc.k1 - 1 && scores) {
            // the piece's sums, before the arrival that its output waits behind
#pragma unroll
            for (int t = 0; t < RT; ++t) {
              float u = l[t];
#pragma unroll
              for (int o = 1; o <= kRowLanes; o <<= 1)
                if (o & kRowLanes) u += __shfl_xor_sync(0xffffffffu, u, o);
              if ((lane & kRowLanes) == 0) {
                // (a row whose scores are all -inf has a sum of 0 and O 0 or NaN: NaN)
                tail->l[n & 1][row[t]] = 1.f / u;
                if (pc.slot >= 0)
                  p.part_ml[(int64_t)(2 * cta + pc.slot) * NR + row[t]] =
                      make_float2(m[t], lim[t] > pc.k0 * KT ? u : kNoKey);
              }
            }
          }
          if (!live) break;
          tc::fence_proxy_async_smem();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->p_full[g & 1]);
          ++g;
        }
        if (!ok) break;
        if (!live) {
          g = 0;
          continue;
        }
        if constexpr (kTwo) {
          // the groups' sums of the piece, joined by the first
          float u = l[0];
#pragma unroll
          for (int o = 1; o <= kRowLanes; o <<= 1)
            if (o & kRowLanes) u += __shfl_xor_sync(0xffffffffu, u, o);
          if (second) {
            if (scores && (lane & kRowLanes) == 0)
              tail->sums[n % kPieces][row[0]] = make_float2(m[0], u);
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&tail->sum_full[w4][n % kPieces]);
              release(n);
            }
            continue;
          }
          // (released pieces bound how far the second group runs ahead)
          if (!(ok = wait(&tail->sum_full[w4][n % kPieces], n / kPieces))) break;
          if (scores) {
            const float2 o = tail->sums[n % kPieces][row[0]];
            const float top = fmaxf(m[0], o.x);
            u = u * (m[0] == top ? 1.f : ex2_ftz(m[0] - top)) +
                o.y * (o.x == top ? 1.f : ex2_ftz(o.x - top));
            if ((lane & kRowLanes) == 0) {
              tail->l[n & 1][row[0]] = 1.f / u;
              if (pc.slot >= 0)
                p.part_ml[(int64_t)(2 * cta + pc.slot) * NR + row[0]] =
                    make_float2(top, lim[0] > pc.k0 * KT ? u : kNoKey);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tail->l_full);
          if (!(ok = wait(&tail->l_full, n))) break;
        }

        // ---- the piece's rows: normalised to out, or a partial
        if (!(ok = wait(&tail->pv_done[(g - 1) & 1], (g - 1) >> 1))) break;
        tc::fence_after_sync();
        if constexpr (!F8) {
          if (__builtin_expect(
                  *reinterpret_cast<volatile int32_t*>(&tail->cleared[n & 1]) == n + 1, 0))
            put_back<L, NR>(tmem + lanes, p.latent, p.block_tables + (int64_t)pc.r * p.max_blocks,
                            p.b_shift, p.num_blocks, w4 * 32 + lane,
                            max(pc.k0 * KT, pc.sees + (int)((unsigned)pc.first / (unsigned)p.Hq)),
                            min(pc.k1 * KT, pc.n_keys), pc.first, pc.sees, p.Hq);
        }
        if (pc.slot < 0) {
          // lane = dim, register = row: three exchanges between lanes whose
          // numbers differ in one bit leave 8 dims of two rows in each lane
          __nv_bfloat16* orow = p.out + (int64_t)pc.row * L + w4 * 32 + (lane >> 3) * 8;
#pragma unroll 1
          for (int c = 0; c < NR; c += 16) {
            if (c >= pc.rows) break;
            uint32_t o[kBlocks][16];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) tmem_ld16(tmem + lanes + b * NR + c, o[b]);
            float inv[16];
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(inv + i) =
                  *reinterpret_cast<const float4*>(&tail->l[n & 1][c + i]);
            tc::tmem_wait_ld();
            // row of the lane's first output: bit 0, 1, 2 of the lane pick bits
            // 3, 2, 1 of the row
            const int r0 = c + (lane & 1) * 8 + (lane & 2) * 2 + ((lane & 4) >> 1);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // lane pairs: bf16 of two dims, 8 rows each
                const float u = __uint_as_float(o[b][i]) * inv[i];
                const float v = __uint_as_float(o[b][i + 8]) * inv[i + 8];
                const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? u : v, 1);
                w[i] = (lane & 1) ? pack_bf16(got, v) : pack_bf16(u, got);
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
                if (r0 + i < pc.rows)
                  *reinterpret_cast<uint4*>(orow + (int64_t)(r0 + i) * L + b * 128) =
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
            uint32_t o[kBlocks][16];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) tmem_ld16(tmem + lanes + b * NR + c, o[b]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int i = 0; i < 16; ++i)  // (rows past the tile's are scratch)
                prow[(c + i) * L + b * 128] = __uint_as_float(o[b][i]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tail->o_empty);
          release(n);
        }
      }
      if (!ok) tail->abort = 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  // the join may be scheduled where this CTA leaves (not before: its CTAs would
  // wait beside this one's; 1 us slower)
  launch_dependents();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partials of the row tiles cut at group boundaries:
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// Grid (attention CTAs, NR / 8): the rows of a tile of n partials are shared out
// over the CTAs of its n - 1 cuts, a row to one warp or, of more than 8 partials, to 4
// or 8, which meet in shared memory. Bound by L2 (every partial is read back once, 2 KB
// a row at L 512) and by latency: four partials are fetched at a time, beside the
// statistics and not behind them (13 partials a row, one at a time, cost 12 us). One
// request of 60000 keys, 152 partials a row: the call takes 58 us with a warp a row,
// 36 with eight; batches of short rows pay up to 0.8 us for the larger kernel.
constexpr int kJoinWarps = 8, kJoinBatch = 4;

template <int L, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const LatentParams p) {
  __shared__ float2 part_sum[kJoinWarps];
  __shared__ alignas(16) float part_acc[kJoinWarps][L];
  grid_dependency_wait();  // the partials are complete and visible
  const LatentJoin j = p.joins[blockIdx.x];
  if (j.rows == 0) return;
  const int n = j.pieces, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = n <= 8 ? 1 : n <= 16 ? 4 : 8;  // warps of a row (<= n - 1)
  const int sub = warp & (share - 1);
  const int row = (j.cut * (int)gridDim.y + (int)blockIdx.y) * (kJoinWarps / share) + warp / share;
  const bool live = row < j.rows;
  // piece 0 is slot 1 of the CTA one group before the first cut, piece i slot 0 of
  // the CTA i - 1 groups behind it
  const int first = blockIdx.x - j.cut * p.lanes;
  auto slot = [&](int i) -> int64_t { return 2 * (first + (i - 1) * p.lanes) + (i == 0 ? 1 : 0); };
  constexpr int kV = L / 128;
  float4 acc[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = kNoKey;  // running reference and sum of the pieces so far
#pragma unroll 1
  for (int i0 = sub; live && i0 < n; i0 += kJoinBatch * share) {
    float4 x[kJoinBatch][kV];
    float2 ml[kJoinBatch];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      ml[i] = make_float2(-INFINITY, kNoKey);
      if (i0 + i * share < n) {
        const int64_t at = slot(i0 + i * share) * NR + row;
        ml[i] = __ldcg(p.part_ml + at);
        // (a piece without a visible key has no partial: what is read is not used)
#pragma unroll
        for (int v = 0; v < kV; ++v)
          x[i][v] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * L) + lane + v * 32);
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i)
      if (!(ml[i].y < 0.f)) top = fmaxf(top, ml[i].x);  // (a NaN sum counts)
    const float keep = m == -INFINITY ? 0.f : ex2_ftz(m - top);
    m = top;
    if (l > 0.f) l *= keep;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      acc[v].x *= keep;
      acc[v].y *= keep;
      acc[v].z *= keep;
      acc[v].w *= keep;
    }
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      if (ml[i].y < 0.f) continue;
      // (scores of -inf alone weigh 0, which O may make a NaN)
      const float w = ml[i].x == -INFINITY ? 0.f : ex2_ftz(ml[i].x - m);
      l = fmaf(w, ml[i].y, l < 0.f ? 0.f : l);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        acc[v].x = fmaf(w, x[i][v].x, acc[v].x);
        acc[v].y = fmaf(w, x[i][v].y, acc[v].y);
        acc[v].z = fmaf(w, x[i][v].z, acc[v].z);
        acc[v].w = fmaf(w, x[i][v].w, acc[v].w);
      }
    }
  }
  uint2* dst = reinterpret_cast<uint2*>(p.out + (j.out_row + row) * L);
  if (share == 1) {
    if (!live) return;
    const float inv = l < 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int v = 0; v < kV; ++v)
      dst[lane + v * 32] = make_uint2(pack_bf16(acc[v].x * inv, acc[v].y * inv),
                                      pack_bf16(acc[v].z * inv, acc[v].w * inv));
    return;
  }
  // the warps' shares of a row, each warp some of the dims
#pragma unroll
  for (int v = 0; v < kV; ++v)
    *reinterpret_cast<float4*>(&part_acc[warp][(lane + v * 32) * 4]) = acc[v];
  if (lane == 0) part_sum[warp] = make_float2(m, l);
  __syncthreads();
  if (!live) return;
  const int w0 = warp - sub;
  float top = -INFINITY, sum = 0.f;
  auto weight = [&](float x) { return x == -INFINITY ? 0.f : ex2_ftz(x - top); };
  for (int k = 0; k < share; ++k)
    if (!(part_sum[w0 + k].y < 0.f)) top = fmaxf(top, part_sum[w0 + k].x);
  for (int k = 0; k < share; ++k)
    if (!(part_sum[w0 + k].y < 0.f))
      sum = fmaf(weight(part_sum[w0 + k].x), part_sum[w0 + k].y, sum);
  const float inv = 1.f / sum;  // (every row sees a key)
  for (int q = sub * 32 + lane; q < L / 4; q += share * 32) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < share; ++k) {
      const float2 s = part_sum[w0 + k];
      if (s.y < 0.f) continue;
      const float w = weight(s.x);
      const float4 x = *reinterpret_cast<const float4*>(&part_acc[w0 + k][q * 4]);
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    dst[q] = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
}

// ----------------------------------------------------------------- host side

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// joins, statistics and partials of a grid of n CTAs with NR-row tiles
size_t scratch_bytes(int n, int NR, int L) {
  return align256((size_t)n * sizeof(LatentJoin)) + align256((size_t)2 * n * NR * sizeof(float2)) +
         (size_t)2 * n * NR * L * sizeof(float);
}

// Rows of `chunks` times 128 bytes (64 bf16 or 128 codes), row_bytes apart, as
// [chunk][row][128 bytes]: one box is `box_rows` rows of `box_chunks` chunks, chunk
// after chunk in shared memory, each 128-byte swizzled.
bool encode_chunks(CUtensorMap* m, const void* base, bool codes, int chunks, int64_t row_bytes,
                   int64_t rows, int box_rows, int box_chunks) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint32_t cols = codes ? 128 : 64;
  const cuuint64_t dims[3] = {cols, (cuuint64_t)rows, (cuuint64_t)chunks};
  const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, 128};
  const cuuint32_t box[3] = {cols, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <int L, int NR, bool F8>
pa_status launch(const LatentParams& p, const void* q, const pa_latent_pool* pool, int grid,
                 cudaStream_t s) {
  using S = Smem<L, NR, F8>;
  CUtensorMap tq, tc, tr;
  const int64_t cells = (int64_t)pool->num_blocks * pool->block_size;
  const int box_rows = std::min(pool->block_size, S::KT);
  // (E4M3: the queries are converted, not copied)
  if (!encode_chunks(&tq, q, false, L / 64 + 1, (L + kRope) * 2, (int64_t)p.T * p.Hq, NR,
                     L / 64 + 1) ||
      !encode_chunks(&tc, pool->latent, F8, S::kCols, S::kCols * 128, cells, box_rows,
                     box_rows == S::KT ? S::kCols : 1) ||
      !encode_rope(&tr, pool->rope, cells, box_rows))
    return PA_ERR_CUDA;
  static OncePerDevice attribute;
  if (!attribute.done([] {
        return cudaFuncSetAttribute(latent_attn_kernel<L, NR, F8>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::kAlloc) == cudaSuccess;
      }))
    return PA_ERR_CUDA;
  latent_attn_kernel<L, NR, F8><<<grid, S::kThreads, S::kAlloc, s>>>(tq, tc, tr, p);
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
  return pa::scratch_bytes(std::min(pa::num_sms(), pa::kLatentMaxCtas), pa::kLatentRows,
                           latent_dim);
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
  // rows are addressed by 32-bit tensor-map coordinates
  if ((int64_t)T * Hq > INT32_MAX - pa::kLatentRows) return PA_ERR_UNSUPPORTED;

  const int KT = pa::latent_tile_keys(L, pool->dtype == PA_KV_FP8_E4M3);
  // Row tiles: the smallest of 16, 32 and 64 rows that covers the widest
  // request in one pass over its cells; 64 past that.
  int64_t widest = 0;
  for (int r = 0; r < R; ++r)
    widest = std::max<int64_t>(widest, (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq);
  const int NR = widest <= 16 ? 16 : widest <= 32 ? 32 : 64;
  // CTAs side by side (LatentParams): two on the same keys read them from HBM once
  // and then take 0.93 of the time for a pair of row tiles, but an odd one leaves a CTA
  // idle: 32 requests x 4096 keys, 4 row tiles 116 us alone and 106 side by side, 5 132
  // and 150 (more than two would gain nothing: the products bound).
  const int sms = std::min(pa::num_sms(), pa::kLatentMaxCtas);
  int64_t W = 0, passes = 0, best = INT64_MAX;
  int G = 1;
  for (int lanes = 1; lanes <= 2; ++lanes) {
    int64_t w = 0, n = 0;
    for (int r = 0; r < R; ++r) {
      const int64_t rows = (int64_t)(qsl_host[r + 1] - qsl_host[r]) * Hq;
      if (rows == 0) continue;
      const int64_t of_r = ((rows + NR - 1) / NR + lanes - 1) / lanes;
      n += of_r;
      w += of_r * ((seq_lens_host[r] + KT - 1) / KT);
    }
    const int64_t cost = w * (lanes == 1 ? 100 : 2 * 93);
    if (lanes <= sms && cost < best) {
      best = cost;
      W = w;
      passes = n;
      G = lanes;
    }
    if (widest <= NR) break;  // one row tile each
  }
  // A pass begins with its queries and ends with its output, which stalls its CTA
  // for 2 to 4 us, 3 to 5 tiles: it counts as 4 tiles more in the shares (less where
  // shares are small). 160 decodes 58.8 -> 56.5 us, 24 x 4 drafted tokens 30.2 -> 26.7.
  const int skip = (int)std::min<int64_t>(4, W / (sms / G) / 2);
  W += passes * skip;
  // the flat space stays within 31 bits whatever the device lengths are
  const int64_t most = ((int64_t)T * Hq / NR + R) *
                       (skip + ((int64_t)max_blocks * pool->block_size + KT - 1) / KT);
  if (most >= pa::kMaxWork) return PA_ERR_UNSUPPORTED;
  const int grid = G * (int)std::min<int64_t>(W, sms / G);
  if (workspace_bytes < pa::scratch_bytes(grid, NR, L)) return PA_ERR_INVALID;

  pa::LatentParams p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.qsl = query_start_loc;
  p.seq_lens = seq_lens;
  p.block_tables = block_tables;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.latent = static_cast<const uint8_t*>(pool->latent);
  p.rope = static_cast<const uint8_t*>(pool->rope);
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
  p.skip = skip;
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
  auto go = [&](auto l, auto f8) {
    constexpr int kL = decltype(l)::value;
    constexpr bool kF8 = decltype(f8)::value;
    return NR == 16   ? pa::launch<kL, 16, kF8>(p, q, pool, grid, s)
           : NR == 32 ? pa::launch<kL, 32, kF8>(p, q, pool, grid, s)
                      : pa::launch<kL, 64, kF8>(p, q, pool, grid, s);
  };
  const auto L512 = std::integral_constant<int, 512>{};
  const auto L256 = std::integral_constant<int, 256>{};
  if (pool->dtype == PA_KV_FP8_E4M3)
    return L == 512 ? go(L512, std::true_type{}) : go(L256, std::true_type{});
  return L == 512 ? go(L512, std::false_type{}) : go(L256, std::false_type{});
}
