// latent_attn.h — launch interface between pa_latent_forward's planner and the
// absorbed-attention kernels (internal to libpa).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

constexpr int kLatentKeys = 32;     // keys per tile
constexpr int kLatentRows = 64;     // most query rows (token, head) per row tile
constexpr int kLatentMaxCtas = 1024;

// The work of one call is laid out as one sequence of 32-key tiles, the "flat
// space": unit (request r, row tile i) holds the C_r = ceil(seq_len / 32) key
// tiles that the NR query rows i NR .. of the request are scored against, at
// pref[r] + i C_r, pref the exclusive running sum of tiles_r C_r. CTA b of the
// grid takes the tiles [b Q, b Q + Q), Q = ceil(W / grid): equal shares
// whatever the lengths. Its pieces are the parts of units inside that range; a
// piece that is a whole unit writes its rows, the others (at most the first
// and the last of a CTA) write partials, joined by log-sum-exp:
//   slot 2 b      the piece that begins inside a unit
//   slot 2 b + 1  the piece that begins a unit and does not end it
// so the partials of a unit cut at CTA boundaries c0 + 1 .. c1 are slot
// 2 c0 + 1 and the slots 2 c of c = c0 + 1 .. c1, and the scratch depends on the
// grid alone, not on the batch. Everything is computed from the device arrays
// at every launch, so a captured call follows lengths that change.
struct LatentJoin {       // what the join needs of CTA b's first piece
  int32_t rows;           // query rows of the unit cut at b Q; 0: none, or joined at an earlier cut
  int32_t last;           // c1
  int64_t out_row;        // first row of the unit in out
};

struct LatentParams {
  __nv_bfloat16* out;          // [T * Hq][L]
  const int32_t* qsl;          // [R+1]
  const int32_t* seq_lens;     // [R]
  const int32_t* block_tables; // [R][max_blocks]
  const float* scales;         // E4M3 pools: [num_blocks][B]
  int32_t T, R, Hq, max_blocks, num_blocks, B;
  int32_t causal;
  float scale_log2;            // softmax scale * log2(e)
  LatentJoin* joins;           // [grid]
  float2* part_ml;             // [2 grid][NR] (max in log2 units, sum)
  float* part_o;               // [2 grid][NR][L], unnormalised
  unsigned* err;
};

}  // namespace pa
