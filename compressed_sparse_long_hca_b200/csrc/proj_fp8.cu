// Projection product in 8-bit floating point with one scale per block of 128
// (csa_gemm_fp8):
//     Y[t][o] = sum_b 2^(ex[t][b] + ew[o/128][b]) sum_{c in b} X8[t][c] W8[o][c]
// W8: E4M3 codes with one E8M0 (power-of-two) scale per 128 x 128 block; X8:
// the token's BF16 row quantised in the call to E4M3 with one E8M0 scale per
// 128 values; fp32 sums.
//
// Why power-of-two scales.  The block-scaled tensor-core instruction
// (tcgen05.mma kind::mxf8f6f4) multiplies one E8M0 scale per row and 32 values
// into the product; a block of 128 is four of its steps with the same scale
// byte.  The scaling is then exact and costs no pass over the accumulators,
// and quantising multiplies by a power of two, which is exact too: the only
// rounding is that of the E4M3 code.
//
// Layout (swap AB, as the BF16 projection).  The weight's rows are the MMA's
// M (128 per tile), the tokens its N; K runs in blocks of 128, one 16 KB
// weight tile (packed once, in the no-swizzle K-major core-matrix order: one
// bulk copy) and the matching block of the packed activations per stage.
// Scales travel in 512-byte chunks (128 rows x 4 blocks) with every fourth
// block and are copied to TMEM in front of the MMAs that read them.
//
// Batch invariance.  A weight with few row tiles cuts K into S parts (at most
// 8), S from the weight's shape and the SM count alone; the parts are summed
// in fp32 in part order.  The forms of the launch add the same numbers in the
// same order:
//   spread  one thread-block cluster per (row tile, token tile), a CTA per
//           part; the CTAs leave their fp32 partials in their own shared
//           memory and each adds the parts of its share of the tokens through
//           distributed shared memory;
//   whole   one work item per (row tile, token tile) of a persistent CTA, its
//           parts one after the other into alternating TMEM accumulators,
//           summed in the epilogue's registers.
// The K order inside a part is fixed and a token's column does not enter the
// arithmetic of the others, so a token's bits depend on its row and the weight.
//
// Up to 16 tokens (a weight stream), and for small weights more in tiles of 16,
// the call is one launch without scratch:
// four or eight warps of each CTA quantise the tokens' blocks from global memory
// straight into the MMA's operand layout.  Beyond that the quantised tokens
// are worth keeping: a kernel packs them once, and the product's CTAs read
// blocks of them by bulk copies (7168 x 16384, 37 tokens: 46 us with the
// tokens quantised in every CTA, 26 us packed).
#include <cooperative_groups.h>

#include <algorithm>

#include "csa.h"
#include "proj_fp8.cuh"
#include "tc.cuh"

namespace csa {

namespace cg = cooperative_groups;

// Device error word of this product: first error wins.
__device__ int32_t g_fp8_err[2];

namespace {

struct Fp8Args {
  const uint8_t* w;       // packed weight: tiles [row_tiles][k_blocks][16 KB]
  const uint8_t* wsf;     // its scales: chunks [row_tiles][sup][512]
  const uint8_t* xp;      // packed activations [groups][k_blocks][tok_tiles][tile_n * 128]
  const uint8_t* xsf;     // their scales: chunks [groups][sup][tok_tiles][512]
  const uint16_t* x;      // fused quantisation: the BF16 tokens [n_tok][groups * kg]
  int x_aligned;          // x on 16 bytes (every block's row then is: kg is a multiple of 8)
  int kg;
  int n_out, n_tok;
  int row_tiles, k_blocks, sup;   // sup: scale chunks along K, ceil(k_blocks / 4)
  int groups, group_tiles;        // row tiles of a group
  int splits, split_lg;           // K parts, a power of two
  int tok_tiles, tile_n;          // token tiles of tile_n tokens (a multiple of 16)
  int spread;
  int tiles;                      // row_tiles * tok_tiles
  int quant_groups;               // fused: groups of quantising warps, 1 or 2
  GemmOut out;
};

// NT: most tokens of a tile.  FUSE: the tokens are quantised by this kernel.
// ONE: one accumulator, for CTAs that work on one part of one tile (spread);
// two CTAs of 128 tokens then share an SM's TMEM.
template <int NT, bool FUSE, bool ONE>
struct Cfg {
  static constexpr int kSets = NT >= 128 ? 2 : 1;          // sets of 4 epilogue warps, each a share of the columns
  static constexpr int kCols = NT / kSets;                 // accumulator columns of a set
  static constexpr int kEpi = 128 * kSets;
  static constexpr int kThreads = 64 + kEpi + (FUSE ? 256 : 0);
  static constexpr int kAccs = ONE ? 1 : 2;
  static constexpr int kPerSm = NT <= 64 || ONE ? 2 : 1;   // CTAs per SM
  // Fused: the tokens' blocks have slots of their own beside the ring, filled
  // a batch at a time (the loads of a batch, 32 registers a thread, are in
  // flight at once) by four warps, so that the quantiser works ahead of the
  // weight.  Long parts get a second group of four warps, whose loads are under
  // way while the first's batch is quantised (quant_groups).
  static constexpr int kBatch = 4, kBatches = 2;
  static constexpr int kSlotBytes = NT * kKBlk + kSfBytes;
  static constexpr int kSlots = FUSE ? kBatch * kBatches * kSlotBytes : 0;
  static constexpr int kStageBytes = kWTileBytes + kSfBytes + (FUSE ? 0 : NT * kKBlk + kSfBytes);
  static constexpr int kStagesFit = ((kPerSm == 2 ? 110 : 224) * 1024 - kSlots) / kStageBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  // TMEM: the accumulators, the weight's scale ring, the tokens' scale ring
  static constexpr uint32_t kXsfRing = FUSE ? 8 : kSfRing;
  static constexpr uint32_t kWsfBase = kAccs * NT, kXsfBase = kWsfBase + 4 * kSfRing;
  static constexpr uint32_t kColsNeeded = kXsfBase + 4 * kXsfRing;
  static constexpr uint32_t kTmemCols = kColsNeeded <= 128 ? 128 : kColsNeeded <= 256 ? 256 : 512;
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kSlots + 256 + 128;   // ring, barriers, alignment
  static_assert(NT <= 128, "a token tile's scales are one chunk");
  static_assert(kColsNeeded <= 512 && kTmemCols * kPerSm <= 512, "TMEM");
  static_assert(kStages >= 3 && kStages <= 8, "stages");
  static_assert(kBatches == 2, "one batch of slots for each group of quantising warps");
  static_assert(!FUSE || NT == kFuseTokens, "a quantising thread takes one unit of a block");
  static_assert(kRowTile * NT * 4 <= kStages * kStageBytes, "a part's sums fit in the ring");
};

}  // namespace

// The least e >= -127 with amax <= 448 * 2^e of the BF16 magnitude with bits
// `top` (finite); 0 for an empty block.  448 = 1.75 * 2^8, so e follows from
// the exponent field and whether the mantissa exceeds 1.75; subnormals and
// what else is below 2^-127 * 448 end at -127.
__device__ __forceinline__ int fp8_exponent(uint32_t top) {
  const int e = (int)(top >> 7) - 135 + ((top & 0x7Fu) > 96u ? 1 : 0);
  return top == 0 ? 0 : (e < -127 ? -127 : e);
}

// 16 BF16 values of one row's block as loaded (columns beyond kg are zero).
struct Unit {
  uint32_t w[8];
};

__device__ __forceinline__ Unit load_unit(const uint16_t* p, int cols, bool aligned) {
  Unit u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {                          // kg is a multiple of 8: a half is whole or absent
    uint4 v = make_uint4(0, 0, 0, 0);
    if (8 * h < cols) {
      if (aligned) {
        v = *reinterpret_cast<const uint4*>(p + 8 * h);
      } else {
        const uint16_t* s = p + 8 * h;
        v.x = (uint32_t)s[0] | ((uint32_t)s[1] << 16);
        v.y = (uint32_t)s[2] | ((uint32_t)s[3] << 16);
        v.z = (uint32_t)s[4] | ((uint32_t)s[5] << 16);
        v.w = (uint32_t)s[6] | ((uint32_t)s[7] << 16);
      }
    }
    u.w[4 * h] = v.x; u.w[4 * h + 1] = v.y; u.w[4 * h + 2] = v.z; u.w[4 * h + 3] = v.w;
  }
  return u;
}

// Quantise a unit; the 8 lanes that differ in lane bits 2-4 hold one block of
// a row and share its scale.  `codes`: the 16 E4M3 codes.  Returns the scale
// byte: 255 (NaN, codes 0) for a block that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t quant_unit(const Unit& u, uint4& codes) {
  // the largest magnitude: BF16 bits without the sign order as integers
  // (infinity 0x7F80, NaN above it)
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = __vmaxu2(top, u.w[q] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool finite = top < 0x7F80u;
  const int e = finite ? fp8_exponent(top) : 0;
  const float inv = exp2i(-e);                           // -e in [-120, 127]: a normal fp32, the product exact or below half a code
  uint32_t pk[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t r = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = u.w[2 * q + h];
      const float2 f = make_float2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
      r |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * h);
    }
    pk[q] = finite ? r : 0u;
  }
  codes = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  return (uint32_t)(finite ? e + 127 : 255);
}

// Quantise X (BF16 [n_tok][groups * kg]) into the B operand's blocks: a thread
// block takes 32 rows (8 threads each) of the K blocks blockIdx.y, blockIdx.y +
// gridDim.y, ... of a group, two at a time.  Rows beyond n_tok of the last tile
// and columns beyond kg of the last block are zero; scales nothing reads are
// left as they are.
__global__ void __launch_bounds__(256) fp8_quant_x_kernel(const uint16_t* x, int n_tok, int kg, int64_t row_len,
                                                          int k_blocks, int sup, int tok_tiles, int tile_n,
                                                          bool aligned, uint8_t* xp, uint8_t* xsf) {
  tc::griddep_launch_dependents();                       // the product's blocks may start on their weights
  const int g = blockIdx.z, n_pad = tok_tiles * tile_n;  // a multiple of 16
  // a warp: 4 rows, the row in lane bits 0-1, the column in bits 2-4
  const int c = (threadIdx.x >> 2) & 7, t = blockIdx.x * 32 + (threadIdx.x >> 5) * 4 + (threadIdx.x & 3);
  if (t >= n_pad) return;                                // (whole warps)
  const int j = t / tile_n, r = t - j * tile_n;
  const uint16_t* row = x + (t < n_tok ? (int64_t)t * row_len : 0) + (int64_t)g * kg + c * 16;
  const int cols = t < n_tok ? kg - c * 16 : 0;
  const int64_t block = (int64_t)tok_tiles * tile_n * kKBlk;
  uint8_t* xd = xp + (int64_t)g * k_blocks * block + (int64_t)j * tile_n * kKBlk + code_off(r, c);
  uint8_t* sd = xsf + ((int64_t)g * sup * tok_tiles + j) * kSfBytes + scale_off(r);
  const int64_t sf_step = (int64_t)tok_tiles * kSfBytes;
  for (int b0 = blockIdx.y; b0 < k_blocks; b0 += 2 * gridDim.y) {
    const int b1 = b0 + gridDim.y;
    const bool two = b1 < k_blocks;
    const Unit u0 = load_unit(row + (int64_t)b0 * kKBlk, cols - b0 * kKBlk, aligned);
    const Unit u1 = load_unit(row + (two ? (int64_t)b1 * kKBlk : 0), two ? cols - b1 * kKBlk : 0, aligned);
    uint4 q0, q1;
    const uint32_t s0 = quant_unit(u0, q0), s1 = quant_unit(u1, q1);
    *reinterpret_cast<uint4*>(xd + b0 * block) = q0;
    if (c == 0) sd[(b0 >> 2) * sf_step + (b0 & 3)] = (uint8_t)s0;
    if (two) {
      *reinterpret_cast<uint4*>(xd + b1 * block) = q1;
      if (c == 0) sd[(b1 >> 2) * sf_step + (b1 & 3)] = (uint8_t)s1;
    }
  }
}

// Warp 0 issues the bulk copies, warp 1 the scale copies and MMAs, the next 4
// or 8 read the accumulators (a thread = one output feature, its columns =
// tokens), the last 4 or 8 (FUSE) quantise the tokens.  TILED: there may be
// more than one tile of tokens.
template <int NT, bool FUSE, bool ONE, bool TILED>
__global__ void __launch_bounds__(Cfg<NT, FUSE, ONE>::kThreads, Cfg<NT, FUSE, ONE>::kPerSm)
    fp8_gemm_kernel(const __grid_constant__ Fp8Args a) {
  using C = Cfg<NT, FUSE, ONE>;
  constexpr uint32_t kAccMask = C::kAccs - 1;
  constexpr int S = C::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint8_t* slots = sm + (size_t)S * C::kStageBytes;    // fused: the tokens' blocks
  uint64_t* full = reinterpret_cast<uint64_t*>(slots + C::kSlots);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* x_full = drain + 1;                        // fused: a batch of slots is filled, is read
  uint64_t* x_empty = x_full + C::kBatches;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(x_empty + C::kBatches);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_slot = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);   // stages the producer filled
  // (broadcast: the role and the TMEM base are then known to be warp-uniform,
  // and the MMAs' operands need no move between register files)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr uint64_t kLimit = 1000000000ull;
  constexpr int kXOff = kWTileBytes, kWsfOff = kXOff + (FUSE ? 0 : NT * kKBlk), kXsfOff = kWsfOff + kSfBytes;   // in a stage

  tc::griddep_launch_dependents();
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], 1); }
    for (int x = 0; x < 2; ++x) { tc::mbar_init(&acc_full[x], 1); tc::mbar_init(&acc_empty[x], C::kEpi); }
    tc::mbar_init(drain, 1);
    for (int b = 0; b < C::kBatches; ++b) { tc::mbar_init(&x_full[b], 4); tc::mbar_init(&x_empty[b], 1); }
    *abort_flag = 0;
    *issued_slot = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint32_t lg = (uint32_t)a.split_lg;
  const int xb = a.tile_n * kKBlk;                      // bytes of one packed activation block

  // Spread: this CTA's part of one tile.  Whole: every part of the tiles
  // blockIdx.x, blockIdx.x + gridDim.x, ...
  const int part = a.spread ? (int)(blockIdx.x & (a.splits - 1)) : 0;
  const int it0 = a.spread ? (int)(blockIdx.x >> lg) : (int)blockIdx.x;
  const int it_step = a.spread ? a.tiles : (int)gridDim.x;
  const int k0 = a.spread ? part_begin(a.k_blocks, lg, part) : 0;
  const int k1 = a.spread ? part_begin(a.k_blocks, lg, part + 1) : a.k_blocks;
  const int q0 = part, q1 = a.spread ? part + 1 : a.splits;
  auto row_tile = [&](int it) { return !TILED || a.tok_tiles == 1 ? it : it / a.tok_tiles; };
  auto group = [&](int rt) { return a.groups == 1 ? 0 : rt / a.group_tiles; };
  bool ok = true;
  if (warp == 0) {
    // ---- producer (one thread).  The weight does not depend on the kernels
    //      ahead (the packing ends with a kernel of its own): its first stages
    //      are issued before waiting for them.
    if (tc::elect_one()) {
      // (every instruction between two blocks counts: addresses run along)
      const uint32_t sm0 = tc::smem_u32(sm), full0 = tc::smem_u32(full);
      const uint32_t bytes = (uint32_t)(kWTileBytes + (FUSE ? 0 : xb)), sf_bytes = kSfBytes + (FUSE ? 0 : kSfBytes);
      const int64_t xp_step = (int64_t)a.tok_tiles * xb, xsf_step = (int64_t)a.tok_tiles * kSfBytes;
      uint32_t x = 0, st = 0, ph = 1;                   // stages filled; the stage and its last release's phase
      const int pre = k1 - k0 < S ? k1 - k0 : S;        // blocks whose weight copies are issued ahead
      {
        const int rt = row_tile(it0);
        const uint8_t* w = a.w + ((int64_t)rt * a.k_blocks + k0) * kWTileBytes;
        const uint8_t* wsf = a.wsf + ((int64_t)rt * a.sup + (k0 >> 2)) * kSfBytes;
        for (int i = 0; i < pre; ++i, w += kWTileBytes) {
          const uint32_t at = sm0 + i * C::kStageBytes, bar = full0 + i * 8;
          const bool sf = i == 0 || ((k0 + i) & 3) == 0;
          tc::mbar_expect_tx_at(bar, bytes + (sf ? sf_bytes : 0u));
          tc::bulk_g2s_at(at, w, kWTileBytes, bar);
          if (sf) {
            tc::bulk_g2s_at(at + kWsfOff, wsf, kSfBytes, bar);
            wsf += kSfBytes;
          }
        }
      }
      if (!FUSE) tc::griddep_wait();
      for (int it = it0; it < a.tiles && ok; it += it_step) {
        const int rt = row_tile(it), tt = it - rt * a.tok_tiles;
        const int64_t grp = group(rt);
        const uint8_t* w = a.w + ((int64_t)rt * a.k_blocks + k0) * kWTileBytes;
        const uint8_t* wsf = a.wsf + ((int64_t)rt * a.sup + (k0 >> 2)) * kSfBytes;
        const uint8_t* xp = a.xp + ((grp * a.k_blocks + k0) * a.tok_tiles + tt) * xb;
        const uint8_t* xsf = a.xsf + ((grp * a.sup + (k0 >> 2)) * a.tok_tiles + tt) * kSfBytes;
        for (int kb = k0; kb < k1; ++kb) {
          ok = tc::mbar_wait(&empty[st], ph, kLimit);   // (a fresh barrier's wait for phase 1 passes)
          if (!ok) break;
          const uint32_t at = sm0 + st * C::kStageBytes, bar = full0 + st * 8;
          const bool ahead = (int)x < pre;              // its weight copies are issued
          if (kb == k0 || (kb & 3) == 0) {
            if (!ahead) {
              tc::mbar_expect_tx_at(bar, bytes + sf_bytes);
              tc::bulk_g2s_at(at + kWsfOff, wsf, kSfBytes, bar);
            }
            if (!FUSE) tc::bulk_g2s_at(at + kXsfOff, xsf, kSfBytes, bar);
            wsf += kSfBytes;
            xsf += xsf_step;
          } else if (!ahead) {
            tc::mbar_expect_tx_at(bar, bytes);
          }
          if (!ahead) tc::bulk_g2s_at(at, w, kWTileBytes, bar);
          if (!FUSE) tc::bulk_g2s_at(at + kXOff, xp, (uint32_t)xb, bar);
          w += kWTileBytes;
          xp += xp_step;
          ++x;
          if (++st == S) { st = 0; ph ^= 1; }
        }
      }
      *issued_slot = x;
      if (!ok) *abort_flag = 1;
      for (; (int)x < pre; ++x) tc::mbar_wait(&full[x], 0, 1000ull);   // (an abort before) weight copies without their tokens
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- scale copies and MMAs (one thread).  Issuing a block's four MMAs
    //      bounds narrow tiles: 680 cycles a block with descriptors built from
    //      their fields in a warp-wide loop, about 300 with one thread's loop
    //      over uniform values, where base values plus multiples of the stage
    //      and block are counted along (four MMAs themselves: 180 cycles or
    //      less up to 64 tokens, 256 at 128).
    if (tc::elect_one()) {
      const uint32_t desc_hi = tc::smem_desc_hi(1024), sf_hi = tc::smem_desc_hi(128);
      const uint32_t lo0 = tc::smem_desc_lo(tc::smem_u32(sm), 128);
      const uint32_t idesc0 = tc::idesc_mxf8(kRowTile, a.tile_n, 0, 0);
      constexpr uint32_t kIdStep = (1u << 29) | (FUSE ? 0u : 1u << 4);   // the scale byte of the next block
      uint32_t st = 0, ph = 0;                          // stage and its phase
      uint32_t u = 0;                                   // accumulators used
      uint32_t wr = kSfRing - 1, xr = FUSE ? 0 : kSfRing - 1;   // scale buffers in use
      uint32_t xbatch = 0, xi = 0, xph = 0;             // fused: the tokens' batch, the block in it, its phase
      const uint32_t slot0 = tc::smem_desc_lo(tc::smem_u32(slots), 128);
      for (int it = it0; it < a.tiles && ok; it += it_step) {
        int kb = k0;
        for (int q = q0; q < q1 && ok; ++q, ++u) {
          const int b1 = part_begin(a.k_blocks, lg, q + 1);
          const uint32_t acc = tmem + (u & kAccMask) * NT;
          if (!ONE && u >= 2) ok = tc::mbar_wait(&acc_empty[u & 1], ((u >> 1) - 1) & 1, kLimit);
          uint32_t more = 0;                            // 0: the part's first block
          while (kb < b1 && ok) {
            // the blocks of one scale chunk, the scale byte a constant of each copy of the code
            const int first = kb & 3, last = min(b1 - (kb - first), 4);
#pragma unroll
            for (int id = 0; id < 4; ++id) {
              if (id < first || id >= last || !ok) continue;
              ok = tc::mbar_wait(&full[st], ph, kLimit);
              if (FUSE && xi == 0) ok = ok && tc::mbar_wait(&x_full[xbatch], xph, kLimit);
              if (!ok) continue;
              tc::tc_fence_after();
              // A scale buffer of four blocks is rewritten four loads after its
              // own: by then the MMAs that read it are complete, for the stage
              // just waited for was free (S <= 8 blocks back), or the
              // accumulator two tiles back was.  The tokens' buffers of one
              // block (FUSE) are rewritten 8 >= S blocks later.
              const bool sf = id == 0 || kb == k0;
              if (sf) {
                wr = (wr + 1) & (kSfRing - 1);
                if (!FUSE) xr = wr;
              }
              const uint32_t lo = lo0 + st * (C::kStageBytes / 16);
              const uint32_t xlo = FUSE ? slot0 + (xbatch * C::kBatch + xi) * (C::kSlotBytes / 16) : lo + kXOff / 16;
              const uint32_t wsf = tmem + C::kWsfBase + wr * 4, xsf = tmem + C::kXsfBase + xr * 4;
              const uint32_t wsf_id = wsf + ((uint32_t)id << 30), xsf_id = FUSE ? xsf : xsf + ((uint32_t)id << 30);
              const uint32_t idesc = idesc0 + id * kIdStep;
              if (sf) tc::tmem_cp_32x128b_x4(wsf, tc::desc64(lo + kWsfOff / 16, sf_hi));
              if (FUSE || sf)
                tc::tmem_cp_32x128b_x4(xsf, tc::desc64(FUSE ? xlo + NT * kKBlk / 16 : lo + kXsfOff / 16, sf_hi));
              tc::mma_mxf8(acc, tc::desc64(lo, desc_hi), tc::desc64(xlo, desc_hi), idesc, wsf_id, xsf_id, more);
#pragma unroll
              for (int m = 1; m < 4; ++m)
                tc::mma_mxf8(acc, tc::desc64(lo + m * 16, desc_hi), tc::desc64(xlo + m * 16, desc_hi), idesc, wsf_id, xsf_id, 1u);
              tc::mma_commit(&empty[st]);
              more = 1;
              ++kb;
              if (kb == b1) tc::mma_commit(&acc_full[u & kAccMask]);
              if (FUSE) {
                xr = (xr + 1) & (C::kXsfRing - 1);
                // (The batch is counted, not derived from a slot number.  With
                // x_empty[slot / 4] under slot % 4 == 3 this commit faulted on
                // a misaligned address, though by the source that address is
                // aligned for every slot: the cause is not known, and that
                // form is not used.)
                if (++xi == C::kBatch) {
                  tc::mma_commit(&x_empty[xbatch]);
                  xi = 0;
                  if (++xbatch == C::kBatches) { xbatch = 0; xph ^= 1; }
                }
              }
              if (++st == S) { st = 0; ph ^= 1; }
            }
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (FUSE && warp >= 2 + C::kEpi / 32) {
    // ---- token quantiser: the blocks of this CTA's tiles, kBatch at a time: all
    //      their loads in flight together, one proxy fence for all (a fence
    //      waits for the loads in flight, so that loading ahead across it
    //      gains nothing)
    tc::griddep_wait();
    int batch = (tid - 64 - C::kEpi) >> 7;              // the slots of this group's (next) batch
    const int qt = (tid - 64 - C::kEpi) & 127;          // row (qt >> 5) * 4 + (qt & 3), column (qt >> 2) & 7
    const int r = (qt >> 5) * 4 + (qt & 3), c = (qt >> 2) & 7;
    const int64_t row_len = (int64_t)a.groups * a.kg;
    const int n_it = it0 < a.tiles ? (a.tiles - 1 - it0) / it_step + 1 : 0;
    const int total = n_it * (k1 - k0);
    int lit = it0, lkb = k0;                            // the next block to load
    Unit v[C::kBatch];
    auto load = [&](Unit& dst) {
      const int rt = row_tile(lit), t = TILED ? (lit - rt * a.tok_tiles) * kFuseTokens + r : r;
      const int64_t grp = group(rt);
      const int col = lkb * kKBlk + c * 16;
      const bool there = lit < a.tiles && t < a.n_tok;
      dst = load_unit(a.x + (there ? t : 0) * row_len + grp * a.kg + col, there ? a.kg - col : 0, a.x_aligned != 0);
    };
    auto step = [&]() {
      if (++lkb == k1) { lkb = k0; lit += it_step; }
    };
    const bool both = a.quant_groups == 1;              // one group fills both batches of slots in turn
    for (int d = 0; d < batch * C::kBatch; ++d) step();
    uint32_t ph = 1;                                     // (a fresh barrier's wait for phase 1 passes)
    for (int j0 = batch * C::kBatch; j0 < total && ok; j0 += a.quant_groups * C::kBatch) {
#pragma unroll
      for (int d = 0; d < C::kBatch; ++d, step()) load(v[d]);   // (past the last block: zeros, not used)
      if (!both)
        for (int d = 0; d < C::kBatch; ++d) step();
      ok = tc::mbar_wait(&x_empty[batch], ph, kLimit) && !*abort_flag;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* at = slots + batch * C::kBatch * C::kSlotBytes;
#pragma unroll
      for (int d = 0; d < C::kBatch; ++d, at += C::kSlotBytes) {
        uint4 codes;
        const uint32_t sf = quant_unit(v[d], codes);
        *reinterpret_cast<uint4*>(at + code_off(r, c)) = codes;
        if (c == 0) *reinterpret_cast<uint32_t*>(at + NT * kKBlk + scale_off(r)) = sf;
      }
      tc::fence_proxy_async_smem();                     // (the MMA reads them through the async proxy)
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&x_full[batch]);
      if (both) batch ^= 1;
      if (!both || batch == 0) ph ^= 1;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ---- epilogue
    tc::griddep_wait();                                 // outputs may be written
    const int q4 = warp & 3, set = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    // this set's columns: with two sets the first or second half, in steps of 16
    const int c_half = C::kSets == 1 ? a.tile_n : (a.tile_n / 16 + 1) / 2 * 16;
    const int c_lo = set * c_half;
    uint32_t u = 0;
    for (int it = it0; it < a.tiles; it += it_step) {
      const int rt = row_tile(it), tt = it - rt * a.tok_tiles;
      const int o = rt * kRowTile + q4 * 32 + lane;
      const int t0 = tt * a.tile_n;
      const int n_here = min(min(a.tile_n, a.n_tok - t0) - c_lo, c_half);   // this set's tokens (may be <= 0)
      // The columns go out 16 at a time: to the outputs, or (spread) as this
      // part's sums to the ring's memory, where nothing is in flight any
      // more, as [token][feature].
      float* pw = reinterpret_cast<float*>(sm) + c_lo * kRowTile + q4 * 32 + lane;
      const OutRow y = out_row(a.out, o < a.n_out ? o : 0);
      auto emit = [&](int c0, const float* v) {
        if (a.spread) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c0 + e < n_here) pw[(c0 + e) * kRowTile] = v[e];
        } else if (o < a.n_out) {
          y.store16(t0 + c_lo + c0, n_here - c0, v);
        }
      };
      if (FUSE || ONE || q1 - q0 == 1) {
        ok = ok && tc::mbar_wait(&acc_full[u & kAccMask], ONE ? 0 : (u >> 1) & 1, kLimit) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc::tc_fence_after();
        for (int c0 = 0; c0 < C::kCols && c0 < n_here; c0 += 16) {
          uint32_t v[16];
          tc::tmem_ld_x16(tmem + lane_base + (u & kAccMask) * NT + c_lo + c0, v);
          tc::tmem_wait_ld();
          emit(c0, reinterpret_cast<const float*>(v));
        }
        tc::tc_fence_before();
        if (!ONE) tc::mbar_arrive(&acc_empty[u & 1]);
        ++u;
      } else {
        float acc[C::kCols];
        for (int q = q0; q < q1; ++q, ++u) {
          ok = ok && tc::mbar_wait(&acc_full[u & 1], (u >> 1) & 1, kLimit) && !*abort_flag;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          tc::tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < C::kCols; c0 += 16) {
            if (c0 < n_here) {
              uint32_t v[16];
              tc::tmem_ld_x16(tmem + lane_base + (u & 1) * NT + c_lo + c0, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                acc[c0 + e] = q == q0 ? __uint_as_float(v[e]) : acc[c0 + e] + __uint_as_float(v[e]);
            }
          }
          tc::tc_fence_before();
          tc::mbar_arrive(&acc_empty[u & 1]);
        }
        if (!ok) continue;
#pragma unroll
        for (int c0 = 0; c0 < C::kCols; c0 += 16)
          if (c0 < n_here) emit(c0, acc + c0);
      }
    }
    if (!ok) *abort_flag = 1;
  }
  if (a.spread) {
    // Every CTA of the cluster adds the parts, in part order, of the tokens
    // part, part + S, ...: a thread a feature, kAtOnce tokens in flight (a
    // thread with four features of a token, in 16-byte loads, was slower).
    constexpr int kAtOnce = NT <= 16 ? 1 : 4;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int et = tid - 64;
    const int rt = row_tile(it0), t0 = (it0 - rt * a.tok_tiles) * a.tile_n;
    const int f = et & (kRowTile - 1), o = rt * kRowTile + f;
    if (et >= 0 && et < C::kEpi && o < a.n_out && !*abort_flag) {
      const int n_here = min(a.tile_n, a.n_tok - t0);
      const OutRow y = out_row(a.out, o);
      const float* src[kMaxParts];
#pragma unroll
      for (int p = 0; p < kMaxParts; ++p)
        src[p] = cluster.map_shared_rank(reinterpret_cast<float*>(sm), p < a.splits ? p : 0) + f;
      const int step = a.splits * C::kSets;
      for (int e = part + a.splits * (et / kRowTile); e < n_here; e += step * kAtOnce) {
        float v[kAtOnce][kMaxParts];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int p = 0; p < kMaxParts; ++p)
            v[k][p] = p < a.splits && e + k * step < n_here ? src[p][(e + k * step) * kRowTile] : 0.f;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          float s = v[k][0];
#pragma unroll
          for (int p = 1; p < kMaxParts; ++p)
            if (p < a.splits) s += v[k][p];
          if (e + k * step < n_here) y.store(t0 + e + k * step, s);
        }
      }
    }
    cluster.sync();                                     // a CTA's memory stays until every other has read it
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    if (atomicCAS(&g_fp8_err[0], 0, (int32_t)kErrTimeout) == 0) g_fp8_err[1] = (int32_t)blockIdx.x;
    // let the copies already issued land before the shared memory goes away
    const uint32_t issued = *issued_slot;
    for (uint32_t x = issued > (uint32_t)S ? issued - S : 0; x < issued; ++x)
      tc::mbar_wait(&full[x % S], (x / S) & 1, 200000000ull);
  }
  if (warp == 1) {
    // no tcgen05 operation of this CTA is in flight when TMEM is released
    if (tc::elect_one()) tc::mma_commit(drain);
    __syncwarp();
    tc::mbar_wait(drain, 0, 200000000ull);
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// E4M3 codes [n_out][kg] and E8M0 scales [ceil(n_out/128)][k_blocks] -> packed
// tiles and scale chunks (missing rows and columns zero with scale 1).  The
// block rows of the scales are those of the whole weight; with groups, n_out /
// groups is a multiple of 128, so a tile never spans two groups.
__global__ void __launch_bounds__(256) fp8_pack_w_kernel(const uint8_t* codes, const uint8_t* scales, int n_out, int kg,
                                                         int k_blocks, int sup, bool aligned, uint8_t* w, uint8_t* wsf) {
  const int rt = blockIdx.y, kb = blockIdx.x;
  uint8_t* tile = w + ((int64_t)rt * k_blocks + kb) * kWTileBytes;
  for (int u = threadIdx.x; u < kRowTile * 8; u += blockDim.x) {
    const int r = u >> 3, c = u & 7;
    const int o = rt * kRowTile + r, k0 = kb * kKBlk + c * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (o < n_out && k0 < kg) {
      const uint8_t* p = codes + (int64_t)o * kg + k0;
      if (aligned && k0 + 16 <= kg) {
        v = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t q[4] = {0, 0, 0, 0};
        for (int e = 0; e < 16 && k0 + e < kg; ++e) q[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
        v = make_uint4(q[0], q[1], q[2], q[3]);
      }
    }
    *reinterpret_cast<uint4*>(tile + (r >> 3) * 1024 + c * 128 + (r & 7) * 16) = v;
  }
  uint8_t* sf = wsf + ((int64_t)rt * sup + (kb >> 2)) * kSfBytes;
  const uint8_t s = scales[(int64_t)rt * k_blocks + kb];
  for (int r = threadIdx.x; r < kRowTile; r += blockDim.x) {
    uint8_t* at = sf + 16 * (r & 31) + 4 * (r >> 5);
    at[kb & 3] = s;
    if (kb == k_blocks - 1)
      for (int j = (kb & 3) + 1; j < 4; ++j) at[j] = 127;
  }
}

// The scales once more by feature tile of the pair kernel: chunks [groups *
// f_tiles][sup][2][512], row r of a tile's chunk r / 128 with the four bytes of
// its feature's row block (features beyond the tile: the last block's).
__global__ void __launch_bounds__(256) fp8_pack_pair_scales_kernel(const uint8_t* scales, int row_tiles, int rpg, int f_tiles,
                                                                   int tile_f, int k_blocks, int sup, uint8_t* out) {
  const int ft = blockIdx.x, r = threadIdx.x;
  const int f = min((ft / f_tiles) * rpg + (ft % f_tiles) * tile_f + r, row_tiles * kRowTile - 1);
  const uint8_t* s = scales + (int64_t)(f / kRowTile) * k_blocks;
  for (int c = blockIdx.y; c < sup; c += gridDim.y) {
    uint32_t w = 0;
    for (int j = 0; j < 4; ++j) w |= (uint32_t)(4 * c + j < k_blocks ? s[4 * c + j] : 127) << (8 * j);
    *reinterpret_cast<uint32_t*>(out + (((int64_t)ft * sup + c) * 2 + (r >> 7)) * kSfBytes + scale_off(r & 127)) = w;
  }
}

__global__ void fp8_pack_end_kernel() {}

// BF16 weight [n_out][kg] -> E4M3 codes and one E8M0 scale per 128 x 128
// block, by the rule of fp8_exponent; a block that holds an infinity or a NaN
// gets the NaN scale.
__global__ void __launch_bounds__(256) fp8_quant_w_kernel(const uint16_t* w, int n_out, int kg, int k_blocks,
                                                          uint8_t* codes, uint8_t* scales) {
  __shared__ uint32_t s_top;
  const int rt = blockIdx.y, kb = blockIdx.x;
  if (threadIdx.x == 0) s_top = 0;
  __syncthreads();
  uint32_t top = 0;
  for (int u = threadIdx.x; u < kRowTile * kKBlk; u += blockDim.x) {
    const int o = rt * kRowTile + u / kKBlk, k = kb * kKBlk + u % kKBlk;
    if (o < n_out && k < kg) top = max(top, (uint32_t)(w[(int64_t)o * kg + k] & 0x7FFFu));
  }
  atomicMax(&s_top, top);
  __syncthreads();
  top = s_top;
  const bool finite = top < 0x7F80u;
  const int e = finite ? fp8_exponent(top) : 0;
  for (int u = threadIdx.x; u < kRowTile * kKBlk; u += blockDim.x) {
    const int o = rt * kRowTile + u / kKBlk, k = kb * kKBlk + u % kKBlk;
    if (o < n_out && k < kg)
      codes[(int64_t)o * kg + k] = finite ? e4m3_rn(scale_pow2(bf16_val(w[(int64_t)o * kg + k]), e)) : 0;
  }
  if (threadIdx.x == 0) scales[(int64_t)rt * k_blocks + kb] = (uint8_t)(finite ? e + 127 : 255);
}

// ---- host side

namespace {

struct Plan {
  int row_tiles, k_blocks, sup, splits, nt, tok_tiles, tile_n, tiles;
  bool fuse, spread, pair;
  size_t xsf;                 // workspace offset of the tokens' scales (their codes come first)
};

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// K parts of a weight: a function of its shape and the device alone.  The
// power of two that gives the SMs two CTAs each, every part at least
// kMinPartBlocks blocks long; 7/8 of the places count, for a cluster lies
// within a group of 16 to 20 SMs and those are not filled to the last place
// (7168 x 16384, 37 tokens: 56 clusters of 5 ran as two waves, 40 us; clusters of
// 4 take 26).
int fp8_splits(int row_tiles, int k_blocks, int sms) {
  int s = 1;
  while (2 * s <= kMaxParts && 16 * s * row_tiles <= 14 * sms && 2 * s * kMinPartBlocks <= k_blocks) s *= 2;
  return s;
}

// One launch that quantises in the product's CTAs: up to 16 tokens, and more in
// tiles of 16 while all their CTAs fit the SMs at once, two on an SM (clusters
// fill 7/8 of the places), and have no more than 8 blocks each.  It saves the
// quantiser's launch, about 5 us of host time, and the workspace; on the GPU 76
// tokens x 58 x 64 take 3.2 us instead of 4.7, 1000 x 64 x 256 3.7 instead of
// 5.9, 64 x 2048 x 8192 in 16 groups 4.6 instead of 6.8, but 128 x 1024 x 1024
// 7.5 instead of 6.5 and, 16 blocks a CTA, 20 x 1000 x 16384 10.5 instead of 8.6.
bool fp8_fused(int row_tiles, int k_blocks, int splits, int n_tok, int sms) {
  const int64_t ctas = (n_tok + kFuseTokens - 1LL) / kFuseTokens * row_tiles * splits;
  return n_tok <= kFuseTokens || (8 * ctas <= 14LL * sms && k_blocks <= 8 * splits);
}

// The form of more than 64 tokens: pairs of SMs, whole tiles of one SM or a
// CTA per part of a tile, and the tokens of a tile.  Each has an estimated time,
// waves x (K blocks x time of a block + time of a tile's end), and the least is
// taken; the constants (microseconds) are fits to measured calls:
//   639 x 750 x 8496      whole, 32 tokens a tile 22.3   parts, 128 tokens 16.8
//   140 x 1624 x 5320     whole, 80 tokens 16.4          parts, 96 tokens 10.9
//   905 x 89 x 12512      whole, 32 tokens 30.0          parts, 64 tokens 15.5
//   128 x 9000 x 2048     parts, 128 tokens 15.6         whole, 64 tokens 9.4
//   160 x 7168 x 16384    pairs 41.9                     whole, 80 tokens 36.0
//   256 x 24576 x 1536    whole, 128 tokens 17.1         pairs 16.0
//   2754 x 2564 x 488     whole, 128 tokens 15.5         pairs 12.6
//   595 x 8875 x 1224     pairs 21.9                     whole, 128 tokens 15.5
// A pair stores output rows that are not on 32 bytes more slowly, and odd ones
// more slowly still; the plan, which does not know the outputs, takes the row
// length for that.
void choose_form(Plan& p, int n_out, int groups, int n_tok, int sms) {
  double best = 1e30;
  const int t16 = (n_tok + 15) / 16;
  auto waves = [](int64_t n, int at_once) { return (double)((n + at_once - 1) / at_once); };
  for (int most = 128; most >= 32; most -= 16) {
    const int tok_tiles = (16 * t16 + most - 1) / most;
    const int tile_n = (t16 + tok_tiles - 1) / tok_tiles * 16;
    const int64_t tiles = (int64_t)p.row_tiles * ((n_tok + tile_n - 1) / tile_n);
    const double block = 0.215 + 0.0004 * tile_n;
    for (int spread = 0; spread <= (p.splits > 1 ? 1 : 0); ++spread) {
      double cost;
      if (spread) {
        // two CTAs share an SM (clusters fill 7/8 of the places)
        const int64_t ctas = tiles * p.splits;
        cost = waves(8 * ctas, 14 * sms) * ((ctas > sms ? 2.0 : 1.0) * p.k_blocks / p.splits * block + 2.3 + 0.02 * tile_n);
      } else {
        cost = waves(tiles, sms) * (p.k_blocks * block + 0.4 + 0.01 * tile_n);
      }
      if (cost < best && tiles <= 0x7FFFFFFF / kMaxParts) {
        best = cost;
        p.nt = 128;
        p.tile_n = tile_n;
        p.tok_tiles = (n_tok + tile_n - 1) / tile_n;
        p.spread = spread;
      }
    }
  }
  if (n_tok <= kRowTile) return;
  const int m_tiles = (n_tok + 2 * kRowTile - 1) / (2 * kRowTile), f_tiles = pair_tiles(n_out / groups);
  const int tile_f = pair_features(n_out / groups);
  const double end = (n_out % 16 == 0 ? 0.009 : n_out % 2 == 0 ? 0.017 : 0.024) * tile_f;
  if (waves((int64_t)groups * f_tiles * m_tiles, sms / 2) * (p.k_blocks * (0.13 + 0.0007 * tile_f) + end) < best) {
    p.pair = true;
    p.spread = false;
    p.nt = p.tile_n = kRowTile;
    p.tok_tiles = 2 * m_tiles;
  }
}

Plan fp8_plan(int n_out, int k_in, int groups, int n_tok, int sms) {
  Plan p{};
  p.row_tiles = (n_out + kRowTile - 1) / kRowTile;
  p.k_blocks = (k_in / groups + kKBlk - 1) / kKBlk;
  p.sup = (p.k_blocks + 3) / 4;
  p.splits = fp8_splits(p.row_tiles, p.k_blocks, sms);
  p.fuse = fp8_fused(p.row_tiles, p.k_blocks, p.splits, n_tok, sms);
  if (p.fuse) {
    p.nt = p.tile_n = kFuseTokens;
    p.tok_tiles = (n_tok + kFuseTokens - 1) / kFuseTokens;
    p.spread = p.splits > 1;
  } else {
    if (n_tok <= 64) {
      p.nt = n_tok <= 32 ? 32 : 64;
      p.tok_tiles = 1;
      p.tile_n = (n_tok + 15) / 16 * 16;
      p.spread = p.splits > 1 && 2 * p.row_tiles <= sms;
    } else {
      choose_form(p, n_out, groups, n_tok, sms);
    }
  }
  p.tiles = p.row_tiles * p.tok_tiles;
  p.xsf = al256((size_t)groups * p.k_blocks * p.tok_tiles * p.tile_n * kKBlk);
  return p;
}

template <int NT, bool FUSE, bool ONE, bool TILED = true>
cudaError_t launch_nt(const Fp8Args& a, int sms, cudaStream_t st) {
  using C = Cfg<NT, FUSE, ONE>;
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (setup_needed(attr_set, dev)) {
    e = cudaFuncSetAttribute(fp8_gemm_kernel<NT, FUSE, ONE, TILED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fp8_gemm_kernel<NT, FUSE, ONE, TILED>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    setup_done(attr_set, dev);
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(a.spread ? a.tiles * a.splits : std::min(a.tiles, sms * C::kPerSm)));
  lc.blockDim = dim3(FUSE ? C::kThreads - 128 * (2 - a.quant_groups) : C::kThreads);
  lc.dynamicSmemBytes = C::kSmem;
  lc.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)a.splits;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = a.spread ? 2 : 1;
  e = cudaLaunchKernelEx(&lc, fp8_gemm_kernel<NT, FUSE, ONE, TILED>, a);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

namespace {

// A packed weight: row tiles, their scale chunks, and the scales by feature
// tile of the pair kernel.
struct WeightLayout {
  int row_tiles, k_blocks, sup, f_tiles, tile_f;
  size_t sf, pair_sf, total;
};

WeightLayout weight_layout(int n_out, int k_in, int groups) {
  WeightLayout l{};
  l.row_tiles = (n_out + kRowTile - 1) / kRowTile;
  l.k_blocks = (k_in / groups + kKBlk - 1) / kKBlk;
  l.sup = (l.k_blocks + 3) / 4;
  l.f_tiles = pair_tiles(n_out / groups);
  l.tile_f = pair_features(n_out / groups);
  l.sf = (size_t)l.row_tiles * l.k_blocks * kWTileBytes;
  l.pair_sf = l.sf + (size_t)l.row_tiles * l.sup * kSfBytes;
  l.total = l.pair_sf + (size_t)groups * l.f_tiles * l.sup * 2 * kSfBytes;
  return l;
}

}  // namespace

size_t fp8_weight_bytes(int n_out, int k_in, int groups) { return weight_layout(n_out, k_in, groups).total; }

// The kernel that a call takes (csa_debug_fp8_form).
int fp8_form(int n_out, int k_in, int groups, int n_tok, int sms) {
  const Plan p = fp8_plan(n_out, k_in, groups, n_tok, sms);
  return p.pair ? 256 : p.nt | (p.spread ? CSA_FP8_FORM_CLUSTER : 0) | (p.tok_tiles > 1 ? CSA_FP8_FORM_TILES : 0);
}

// Room for the quantised tokens in every form of n_tok tokens, so that a
// workspace for many tokens serves fewer, too: a form's last tile reaches at
// most 255 rows beyond the tokens, and beyond 64 tokens tiles have at least 32.
size_t fp8_workspace_bytes(int n_out, int k_in, int groups, int n_tok, int sms) {
  const int row_tiles = (n_out + kRowTile - 1) / kRowTile, kb = (k_in / groups + kKBlk - 1) / kKBlk;
  if (fp8_fused(row_tiles, kb, fp8_splits(row_tiles, kb, sms), n_tok, sms)) return 0;
  const size_t k_blocks = kb, sup = (k_blocks + 3) / 4;
  const size_t rows = n_tok <= 64 ? (n_tok + 15) / 16 * 16 : n_tok + 255, tiles = n_tok <= 64 ? 1 : (n_tok + 31) / 32;
  return al256(groups * k_blocks * rows * kKBlk) + al256(groups * sup * tiles * kSfBytes);
}

cudaError_t launch_fp8_pack_weight(const uint8_t* codes, const uint8_t* scales, int n_out, int k_in, int groups,
                                   uint8_t* w, cudaStream_t st) {
  const WeightLayout l = weight_layout(n_out, k_in, groups);
  const int kg = k_in / groups;
  const bool aligned = kg % 16 == 0 && reinterpret_cast<uintptr_t>(codes) % 16 == 0;
  fp8_pack_w_kernel<<<dim3(l.k_blocks, l.row_tiles), 256, 0, st>>>(codes, scales, n_out, kg, l.k_blocks, l.sup, aligned, w,
                                                                   w + l.sf);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fp8_pack_pair_scales_kernel<<<dim3(groups * l.f_tiles, std::min(l.sup, 64)), 256, 0, st>>>(
      scales, l.row_tiles, n_out / groups, l.f_tiles, l.tile_f, l.k_blocks, l.sup, w + l.pair_sf);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // The product reads the weight before it waits for the kernel ahead of it
  // on the stream: that kernel must not be the packing itself.
  fp8_pack_end_kernel<<<1, 32, 0, st>>>();
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_fp8_quant_weight(const uint16_t* w, int n_out, int k_in, int groups, uint8_t* codes, uint8_t* scales,
                                    cudaStream_t st) {
  const int kg = k_in / groups, rt = (n_out + kRowTile - 1) / kRowTile, kb = (kg + kKBlk - 1) / kKBlk;
  fp8_quant_w_kernel<<<dim3(kb, rt), 256, 0, st>>>(w, n_out, kg, kb, codes, scales);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_gemm_fp8(const void* w_packed, int n_out, int k_in, int groups, const uint16_t* x, int n_tok,
                            const GemmOut& out, void* ws, int sms, cudaStream_t st) {
  const Plan p = fp8_plan(n_out, k_in, groups, n_tok, sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const uint8_t* w = static_cast<const uint8_t*>(w_packed);
  const int kg = k_in / groups;
  // every row of every group starts on 16 bytes (kg is a multiple of 8)
  const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0;
  Fp8Args a{};
  a.w = w;
  const WeightLayout l = weight_layout(n_out, k_in, groups);
  a.wsf = w + l.sf;
  a.x = x;
  a.x_aligned = aligned;
  a.kg = kg;
  a.n_out = n_out; a.n_tok = n_tok;
  a.row_tiles = p.row_tiles; a.k_blocks = p.k_blocks; a.sup = p.sup;
  a.groups = groups; a.group_tiles = groups > 1 ? n_out / groups / kRowTile : p.row_tiles;
  a.splits = p.splits;
  while (1 << a.split_lg < p.splits) ++a.split_lg;
  a.tok_tiles = p.tok_tiles; a.tile_n = p.tile_n;
  a.spread = p.spread; a.tiles = p.tiles;
  a.out = out;
  if (p.fuse) {
    // (7168 x 16384, 32 blocks a CTA: 20.8 us with two groups, 24.5 with one;
    // 16 groups of 1024 x 4096, 16 blocks: 14.6 and 15.1 us;
    // 2368 x 7168, 7 blocks: 7.0 and 6.3 us)
    a.quant_groups = (p.spread ? p.k_blocks / p.splits : p.k_blocks) >= 16 ? 2 : 1;
    // (one token tile goes without the division ahead of the first loads: 6.6
    // us instead of 7.1 at 4 tokens x 2368 x 7168)
    return p.tok_tiles > 1 ? launch_nt<kFuseTokens, true, false>(a, sms, st)
                           : launch_nt<kFuseTokens, true, false, false>(a, sms, st);
  }
  a.xp = base;
  a.xsf = base + p.xsf;
  // (An ordinary launch: with programmatic serialization its blocks were
  // resident, waiting, beside the kernel ahead, and 512 tokens x 2368 x 4096
  // took 17.8 us instead of 15.1, 200 tokens 16.4 instead of 13.2.)
  cudaLaunchConfig_t lc{};
  const int row_blocks = (p.tok_tiles * p.tile_n + 31) / 32;
  const int64_t per_group = std::max<int64_t>(1, 8LL * sms / ((int64_t)row_blocks * groups));   // 8 blocks of threads an SM
  lc.gridDim = dim3((unsigned)row_blocks, (unsigned)std::min<int64_t>(per_group, (p.k_blocks + 1) / 2), (unsigned)groups);
  lc.blockDim = dim3(256);
  lc.stream = st;
  cudaError_t e = cudaLaunchKernelEx(&lc, fp8_quant_x_kernel, x, n_tok, kg, (int64_t)k_in, p.k_blocks, p.sup, p.tok_tiles,
                                     p.tile_n, aligned, base, base + p.xsf);
  note_launch();
  if (e != cudaSuccess) return e;
  if (p.pair) {
    Fp8PairArgs b{};
    b.w = w;
    b.wsf = w + l.pair_sf;
    b.xp = a.xp;
    b.xsf = a.xsf;
    b.n_out = n_out; b.n_tok = n_tok; b.groups = groups; b.split_lg = a.split_lg;
    b.k_blocks = p.k_blocks; b.sup = p.sup; b.tok_tiles = p.tok_tiles;
    b.f_tiles = l.f_tiles; b.tile_f = l.tile_f;
    b.tiles = groups * l.f_tiles * (p.tok_tiles / 2);
    b.out = out;
    return launch_fp8_pair(b, sms, st);
  }
  switch (p.nt) {
    case 32: return launch_nt<32, false, false>(a, sms, st);
    case 64: return launch_nt<64, false, false>(a, sms, st);
    default: return p.spread ? launch_nt<128, false, true>(a, sms, st) : launch_nt<128, false, false>(a, sms, st);
  }
}

// Read and clear the device error words (the caller has synchronised).
cudaError_t fp8_read_error(int32_t* code, int32_t* detail) {
  int32_t w[2] = {0, 0};
  cudaError_t e = cudaMemcpyFromSymbol(w, g_fp8_err, sizeof w);
  if (e != cudaSuccess) return e;
  if (w[0] != 0) {
    const int32_t z[2] = {0, 0};
    e = cudaMemcpyToSymbol(g_fp8_err, z, sizeof z);
  } else {
    e = fp8_pair_read_error(w);
  }
  *code = w[0];
  *detail = w[1];
  return e;
}

}  // namespace csa
