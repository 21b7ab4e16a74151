// Shared by the FP8 product's kernels: tile constants, the packed layouts, the
// outputs' rows, and the launch of the pair kernel (proj_fp8_pair.cu).
#pragma once
#include "common.cuh"
#include "gemm_out.cuh"

namespace csa {

constexpr int kRowTile = 128;                 // output features per tile (MMA M)
constexpr int kKBlk = 128;                    // K per stage: one scale block
constexpr int kWTileBytes = kRowTile * kKBlk; // 16 KB
constexpr int kSfBytes = 512;                 // scales of 128 rows x 4 blocks, tcgen05.cp order
constexpr int kSfRing = 4;                    // scale buffers in TMEM
constexpr int kMinPartBlocks = 4;             // K blocks of the smallest part
constexpr int kMaxParts = 8;                  // parts of a weight: CTAs of the largest portable cluster
constexpr int kFuseTokens = 16;               // most tokens that the product quantises itself

// The first K block of part p of 2^lg (parts differ by at most one block; a
// shift, for a division costs the issuing threads 500 cycles).
__host__ __device__ inline int part_begin(int k_blocks, int lg, int p) { return (k_blocks * p) >> lg; }

// Where an output feature goes: element (token t) at y + t * rows.
struct OutRow {
  void* y;
  int64_t rows;
  bool bf16;
  __device__ __forceinline__ void store(int t, float v) const {
    if (bf16) static_cast<uint16_t*>(y)[t * rows] = bf16_rn(v);
    else static_cast<float*>(y)[t * rows] = v;
  }
  // Tokens t .. t + 15, the first n of them.
  __device__ __forceinline__ void store16(int t, int n, const float* v) const {
    if (bf16) {
      uint16_t* p = static_cast<uint16_t*>(y) + t * rows;
#pragma unroll
      for (int e = 0; e < 16; ++e, p += rows)
        if (e < n) *p = bf16_rn(v[e]);
    } else {
      float* p = static_cast<float*>(y) + t * rows;
#pragma unroll
      for (int e = 0; e < 16; ++e, p += rows)
        if (e < n) *p = v[e];
    }
  }
};

__device__ __forceinline__ OutRow out_row(const GemmOut& out, int o) {
  int sg = 0;
  while (sg + 1 < out.n_seg && o >= out.seg_end[sg]) ++sg;
  const int r0 = sg > 0 ? out.seg_end[sg - 1] : 0;
  const bool bf16 = (out.bf16_mask >> sg) & 1u;
  char* y = static_cast<char*>(out.y[sg]);
  return OutRow{y + (int64_t)(o - r0) * (bf16 ? 2 : 4), out.seg_end[sg] - r0, bf16};
}

// Offset of row r's 16-byte column c in a block of rows x 128 codes (no-swizzle
// K-major core matrices), and of row r's scale word in a 512-byte chunk.
__device__ __forceinline__ int code_off(int r, int c) { return (r >> 3) * 1024 + c * 128 + (r & 7) * 16; }
__device__ __forceinline__ int scale_off(int r) { return 16 * (r & 31) + 4 * ((r >> 5) & 3); }

// Features of a pair kernel's tile: the rows of a group in equal tiles of at
// most kPairFeatures, in steps of 16.
constexpr int kPairFeatures = 224;
__host__ __device__ inline int pair_tiles(int rows_per_group) { return (rows_per_group + kPairFeatures - 1) / kPairFeatures; }
__host__ __device__ inline int pair_features(int rows_per_group) {
  const int t = pair_tiles(rows_per_group);
  return ((rows_per_group + t - 1) / t + 15) / 16 * 16;
}

struct Fp8PairArgs {
  const uint8_t* w;       // packed weight: tiles [row_tiles][k_blocks][16 KB]
  const uint8_t* wsf;     // its scales by feature tile: chunks [groups * f_tiles][sup][2][512]
  const uint8_t* xp;      // packed tokens [groups][k_blocks][tok_tiles][16 KB], tiles of 128
  const uint8_t* xsf;     // their scales: chunks [groups][sup][tok_tiles][512]
  int n_out, n_tok, groups;
  int split_lg;           // 2^split_lg K parts
  int k_blocks, sup, tok_tiles;   // tok_tiles even
  int f_tiles, tile_f;    // feature tiles of a group, features of one
  int tiles;              // tiles of a call: groups * f_tiles * tok_tiles / 2
  GemmOut out;
};

cudaError_t launch_fp8_pair(const Fp8PairArgs& a, int sms, cudaStream_t st);
cudaError_t fp8_pair_read_error(int32_t w[2]);      // reads and clears the pair kernel's error word

}  // namespace csa
