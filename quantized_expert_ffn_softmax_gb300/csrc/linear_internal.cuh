// Shared by the translation units of moe_linear (linear.cu, linear_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_internal.cuh"

namespace moe {
namespace lin {

// Packed weights.  Tile (i, c) holds rows 16 i .. 16 i + 15 and inputs 128 c
// .. 128 c + 127 in kTileBytes bytes, tiles of one i contiguous in c:
//   1024 B of codes: two halves of 64 inputs (two scale blocks each); in a
//     half lane l = 4 g + t of a warp finds 16 bytes at 16 l: one word of
//     block 0 row g, block 0 row g + 8, block 1 row g, block 1 row g + 8.
//     A word holds the inputs 8 t .. 8 t + 7 of its block: input 2 i in
//     nibble i and input 2 i + 1 in nibble i + 4, so that
//     (word >> 4 i) & 0x000f000f is the pair (2 i, 2 i + 1).
//   128 B of scales: at 16 g the four block scales of row g, then of row
//     g + 8.
// The words are the A fragments of mma.m16n8k16 as they stand (two MMAs per
// scale block), and eight consecutive inputs of a row in one 16-byte store
// of the tcgen05 path's shared-memory tiles.  Rows past N and inputs past K
// have scale 0.
constexpr int kTileRows = 16;
constexpr int kTileK = 128;
constexpr int kTileCodes = 1024;
constexpr int kTileBytes = 1152;
constexpr int kMaxQ8Tokens = 32;

struct Weights {
  const uint8_t* tiles;
  const float* bias;  // [N] or null
  int K, N;
  int kc;             // tiles along K
  int nt;             // tiles along N
};

}  // namespace lin
}  // namespace moe

struct moe_linear {
  moe_linear_config cfg;
  moe::lin::Weights w;
  void* block = nullptr;
  int* err = nullptr;
  int device = 0;
  int num_sms = 0;
};
