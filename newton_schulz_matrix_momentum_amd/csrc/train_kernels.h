// Kernel argument blocks and launchers of the training operators (internal):
// 8-bit activation checkpoints, weight gradients out of them, and routing to
// experts.  Declared in include/muon.h; host side in train_host.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"
#include "muon_kernels.h"

namespace muon {

// n / d for 0 <= n < 2^31 by one multiply-high (Granlund & Montgomery 1994,
// the round-up multiplier with a 33-bit value split as 2^32 + mul).
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv make_fastdiv(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.shift = 0;
  while (((uint64_t)1 << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - d)) / d + 1);
  return f;
}

// ------------------------------------------------------------ checkpoints
constexpr int kCkptBlock = MUON_CKPT_BLOCK;
constexpr int kCkptVec = 8;                              // columns a thread handles at once
constexpr int kCkptLanes = kCkptBlock / kCkptVec;        // threads that share a block
constexpr int kCkptThreads = 256;

struct CkptMat {
  uint8_t *codes;
  uint8_t *scales;
  int64_t codes_ld, scales_ld;
};

// One launch over rows x ceil(cols / 32) blocks; units = blocks * kCkptLanes
// threads' worth of work, row = unit / units_per_row.
struct CkptArgs {
  const void *a;           // pack: x; swiglu: gate; backward: grad_h
  const void *b;           // swiglu: up
  void *out;               // unpack: x; swiglu: h; backward: h or NULL
  void *out_g, *out_u;     // backward: grad_gate, grad_up
  int64_t ld_a, ld_b, ld_out, ld_g, ld_u;   // elements
  CkptMat m[2];
  int64_t cols;
  uint32_t units;
  FastDiv per_row;
};

hipError_t launch_ckpt_pack(const CkptArgs &args, int dtype, int format, hipStream_t s);
hipError_t launch_ckpt_unpack(const CkptArgs &args, int dtype, int format, hipStream_t s);
hipError_t launch_ckpt_swiglu(const CkptArgs &args, int dtype, int format, hipStream_t s);
hipError_t launch_ckpt_swiglu_backward(const CkptArgs &args, int dtype, int format, hipStream_t s);

// -------------------------------------------------------- weight gradients
struct WgradArgs {
  const void *dy;
  const uint8_t *codes;
  const uint8_t *scales;
  const int32_t *offsets;
  const int32_t *rows_of;
  void *out;               // final matrices
  float *part;             // fp32 partials (splits > 1) of tiles, by part, expert and tile
  int64_t ld_dy, codes_ld, scales_ld;
  int64_t slots, ckpt_rows;
  int32_t outs, cols;
  int32_t experts;
  int32_t splits;          // parts of the token range, or (64 x 64 tiles) of each expert's slots
  int64_t split_len;       // tokens of one part without offsets, a multiple of the k step
  int32_t tiles_n, tiles_d;
  int32_t out_dtype;
  int32_t accumulate;
  int32_t transposed;
  int32_t wide;            // 0: 64 x 64 tiles; 1: 256 outs x 128 columns; 2: 128 x 256
  int32_t blocks, items;   // wide: blocks of the launch; tiles x experts or parts, which the blocks take in turn
  FastDiv tiles, div_d;    // wide: by the tiles of a matrix, and by tiles_d
};
constexpr int kWgradK = 32;

hipError_t launch_wgrad(const WgradArgs &args, int dtype, int format, hipStream_t s);

// ---------------------------------------------------------------- routing
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 64;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteRows = 32;             // tokens of a block
constexpr int kRouteAlone = 64;            // up to so many tokens one block does everything

struct RouteArgs {
  const void *logits;
  int64_t ld;
  int64_t tokens;
  const float *bias;
  const uint8_t *token_mask;
  int32_t *ids;
  float *weights;
  int32_t *counts, *offsets, *order, *rows;
  int64_t *load;
  int32_t *hist;           // workspace [experts][blocks]: slots of a block, then slots of the blocks before
  int32_t *rank;           // workspace [tokens * top_k]: place within (block, expert)
  const float *grad_weights;   // backward
  void *grad_logits;
  int64_t ld_grad;
  int32_t experts, top_k;
  int32_t groups, top_groups, group_top;
  int32_t sigmoid, renormalize;
  int32_t lists;           // the dispatch lists are wanted
  float scale;
  int32_t rows_per_block, blocks;
};

hipError_t launch_route(const RouteArgs &args, int dtype, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs &args, int dtype, hipStream_t s);
hipError_t launch_balance(float *bias, const void *counts, int count_bytes, int64_t layers, int experts, float rate,
                          hipStream_t s);

}  // namespace muon
