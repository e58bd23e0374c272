// latent_attn.h — launch interface between pa_latent_forward's planner and the
// absorbed-attention kernels (internal to libpa).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Keys per tile: 64 where that leaves several tiles of stages beside Q and P, else 32.
constexpr int latent_tile_keys(int latent_dim, bool e4m3) {
  return latent_dim == 512 && !e4m3 ? 32 : 64;
}
constexpr int kLatentRows = 64;     // most query rows (token, head) per row tile
constexpr int kLatentMaxCtas = 1024;

// The work of one call is laid out as one sequence of key tiles, the "flat
// space". The grid is NG groups of G CTAs (G 1 or 2) that walk it side by
// side: a pass (request r, row tiles i G .. i G + G - 1 of NR query rows, one to
// each CTA of the group) takes the C_r = ceil(seq_len / KT) key tiles of the
// request, behind S places without a tile (what a pass costs besides its tiles), at
// pref[r] + i (S + C_r), pref the exclusive running sum of passes_r (S + C_r).
// Group b takes the tiles [b Q, b Q + Q), Q = ceil(W / NG): equal shares whatever
// the lengths, and a cell that several row tiles need is read from HBM once,
// by the first of the group's CTAs that comes to it. A CTA's pieces are the parts
// of passes inside its group's range; a piece that is a whole pass writes its
// rows, the others (at most the first and the last) write partials, joined by
// log-sum-exp:
//   slot 2 c      the piece of CTA c that begins inside a pass
//   slot 2 c + 1  the piece that begins a pass and does not end it
// so the partials of a row tile cut at group boundaries b0 + 1 .. b1 are slot
// 2 c + 1 of its CTA in group b0 and the slots 2 c of those in b0 + 1 .. b1, and
// the scratch depends on the grid alone, not on the batch. Everything is
// computed from the device arrays at every launch, so a captured call follows
// lengths that change.
struct LatentJoin {       // what the join needs of a CTA's first piece
  int32_t rows;           // query rows of the tile cut at its start; 0: none
  int32_t pieces;         // partials of that tile
  int32_t cut;            // which of its cuts this is
  int64_t out_row;        // its first row in out
};

struct LatentParams {
  const __nv_bfloat16* q;      // [T * Hq][L + 64]
  const uint8_t* latent;       // the pool's cells
  const uint8_t* rope;
  __nv_bfloat16* out;          // [T * Hq][L]
  const int32_t* qsl;          // [R+1]
  const int32_t* seq_lens;     // [R]
  const int32_t* block_tables; // [R][max_blocks]
  const float* scales;         // E4M3 pools: [num_blocks][B]
  int32_t T, R, Hq, max_blocks, num_blocks, B, b_shift;  // B = 1 << b_shift
  int32_t causal;
  int32_t lanes;               // G
  int32_t skip;                // S of the flat space
  float scale_log2;            // softmax scale * log2(e)
  LatentJoin* joins;           // [grid]
  float2* part_ml;             // [2 grid][NR] (max in log2 units, sum)
  float* part_o;               // [2 grid][NR][L], unnormalised
  unsigned* err;
};

}  // namespace pa
