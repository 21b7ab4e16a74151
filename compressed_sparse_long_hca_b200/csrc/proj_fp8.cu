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
// Batch invariance.  A weight with few row tiles cuts K into S parts, S from
// the weight's shape and the SM count alone; the parts are summed in fp32 in
// part order.  Two forms of the launch add the same numbers in the same order:
//   spread  (few tokens): one work item per (row tile, token tile, part); each
//           writes its fp32 partial, the item that finishes a tile last adds
//           the parts in order;
//   whole   (many tokens): one work item per (row tile, token tile), its parts
//           one after the other into alternating TMEM accumulators, summed in
//           the epilogue's registers.
// The K order inside a part is fixed and a token's column does not enter the
// arithmetic of the others, so a token's bits depend on its row and the weight.
#include <algorithm>

#include "common.cuh"
#include "gemm_out.cuh"
#include "tc.cuh"

namespace csa {

// Device error word of this product: first error wins.
__device__ int32_t g_fp8_err[2];

namespace {

constexpr int kRowTile = 128;                 // output features per tile (MMA M)
constexpr int kKBlk = 128;                    // K per stage: one scale block
constexpr int kWTileBytes = kRowTile * kKBlk; // 16 KB
constexpr int kSfBytes = 512;                 // scales of 128 rows x 4 blocks, tcgen05.cp order
constexpr int kSfRing = 4;                    // scale buffers in TMEM
constexpr int kMinPartBlocks = 4;             // K blocks of the smallest part

struct Fp8Args {
  const uint8_t* w;       // packed weight: tiles [row_tiles][k_blocks][16 KB]
  const uint8_t* wsf;     // its scales: chunks [row_tiles][sup][512]
  const uint8_t* xp;      // packed activations [groups][k_blocks][tok_tiles][tile_n * 128]
  const uint8_t* xsf;     // their scales: chunks [groups][sup][tok_tiles][chunks][512]
  int n_out, n_tok;
  int row_tiles, k_blocks, sup;   // sup: scale chunks along K, ceil(k_blocks / 4)
  int groups, splits;
  int tok_tiles, tile_n;          // token tiles of tile_n tokens (a multiple of 32)
  int spread;
  int items;
  GemmOut out;
  float* part;            // spread, splits > 1: [splits][n_tok][n_out] fp32 partials
  int32_t* done;          // spread, splits > 1: [row_tiles][tok_tiles] parts finished
};

// NT: most tokens of a tile.
template <int NT>
struct Cfg {
  static constexpr int kSets = NT >= 128 ? 2 : 1;          // sets of 4 epilogue warps, each a share of the columns
  static constexpr int kCols = NT / kSets;                 // accumulator columns of a set
  static constexpr int kThreads = 64 + 128 * kSets;
  static constexpr int kPerSm = NT <= 64 ? 2 : 1;          // CTAs per SM
  static constexpr int kChunks = (NT + 127) / 128;         // scale chunks of a token tile
  static constexpr int kStageBytes = kWTileBytes + NT * kKBlk + kSfBytes * (1 + kChunks);
  static constexpr int kStagesFit = (kPerSm == 2 ? 110 : 224) * 1024 / kStageBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr uint32_t kSfCols = 4 * (1 + kChunks);   // TMEM columns of one scale buffer
  static constexpr uint32_t kSfBase = 2 * NT;
  static constexpr uint32_t kColsNeeded = 2 * NT + kSfRing * kSfCols;
  static constexpr uint32_t kTmemCols = kColsNeeded <= 128 ? 128 : kColsNeeded <= 256 ? 256 : 512;
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 256 + 128;
  static_assert(kColsNeeded <= 512 && kTmemCols * kPerSm <= 512, "TMEM");
  static_assert(kStages >= 3 && kStages <= 8, "stages");
};

// The first K block of part p (parts differ by at most one block).
__host__ __device__ inline int part_begin(int k_blocks, int splits, int p) {
  return (int)((int64_t)k_blocks * p / splits);
}

__device__ __forceinline__ void g_store(void* base, int64_t at, bool bf16, float v) {
  if (bf16) static_cast<uint16_t*>(base)[at] = bf16_rn(v);
  else static_cast<float*>(base)[at] = v;
}

}  // namespace

// The least e with amax <= 448 * 2^e, clamped to E8M0's range; 0 for an empty
// block.  448 = 1.75 * 2^8, so e follows from amax's exponent and mantissa.
__device__ __forceinline__ int fp8_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int e = ilogbf(amax);
  const float m = scale_pow2(amax, e);               // [1, 2)
  e = e - 8 + (m > 1.75f ? 1 : 0);
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// Quantise X (BF16 [n_tok][groups * kg]) into the B operand's blocks: a thread
// takes 16 values, the 8 threads of a (token, block) share its scale.  A block
// that holds an infinity or a NaN gets the NaN scale: every output of that
// token is then NaN.  Rows beyond n_tok of the last tile and columns beyond kg
// of the last block are zero; scales nothing reads are left as they are.
// Also clears the row tiles' part counters.
__global__ void __launch_bounds__(256) fp8_quant_x_kernel(const uint16_t* x, int n_tok, int kg, int64_t row_len,
                                                          int k_blocks, int sup, int tok_tiles, int tile_n, int chunks,
                                                          bool aligned, uint8_t* xp, uint8_t* xsf, int32_t* done,
                                                          int n_done) {
  tc::griddep_launch_dependents();
  if (done != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    for (int u = threadIdx.x; u < n_done; u += blockDim.x) done[u] = 0;
  const int g = blockIdx.y;
  x += (int64_t)g * kg;
  xp += (int64_t)g * k_blocks * tok_tiles * tile_n * kKBlk;
  xsf += (int64_t)g * sup * tok_tiles * chunks * kSfBytes;
  const int n_pad = tok_tiles * tile_n;
  const int64_t total = (int64_t)k_blocks * n_pad * 8;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < total; u += (int64_t)gridDim.x * blockDim.x) {
    const int c = (int)(u & 7);
    const int t = (int)((u >> 3) % n_pad);
    const int b = (int)((u >> 3) / n_pad);
    const int k0 = b * kKBlk + c * 16;
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t < n_tok) {
      const uint16_t* p = x + (int64_t)t * row_len + k0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {                  // kg is a multiple of 8: a half is whole or absent
        if (k0 + 8 * h >= kg) break;
        if (aligned) {
          const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * h);
          w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
        } else {
          for (int q = 0; q < 4; ++q) w[4 * h + q] = (uint32_t)p[8 * h + 2 * q] | ((uint32_t)p[8 * h + 2 * q + 1] << 16);
        }
      }
    }
    // the largest magnitude: BF16 bits without the sign order as integers
    // (infinity 0x7F80, NaN above it)
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) top = __vmaxu2(top, w[q] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F80u;
    const int e = finite ? fp8_exponent(bf16_val((uint16_t)top)) : 0;
    uint32_t pk[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t r = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = w[2 * q + h];
        const float lo = scale_pow2(bf16_val((uint16_t)(v & 0xFFFFu)), e), hi = scale_pow2(bf16_val((uint16_t)(v >> 16)), e);
        r |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3) << (16 * h);
      }
      pk[q] = finite ? r : 0u;
    }
    const int j = t / tile_n, r = t % tile_n;
    uint8_t* dst = xp + ((int64_t)b * tok_tiles + j) * tile_n * kKBlk + (r >> 3) * 1024 + c * 128 + (r & 7) * 16;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    if (c == 0)
      xsf[(((int64_t)(b >> 2) * tok_tiles + j) * chunks + (r >> 7)) * kSfBytes + 16 * (r & 31) + 4 * ((r >> 5) & 3) + (b & 3)] =
          (uint8_t)(finite ? e + 127 : 255);
  }
}

// Persistent CTAs over the work items.  Warp 0 issues the bulk copies, warp 1
// the scale copies and MMAs (one elected lane each), the others read the
// accumulators (a thread = one output feature, its columns = tokens).
template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kPerSm) fp8_gemm_kernel(Fp8Args a) {
  using C = Cfg<NT>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + (size_t)S * C::kStageBytes);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr uint64_t kLimit = 1000000000ull;

  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], 1); }
    for (int x = 0; x < 2; ++x) { tc::mbar_init(&acc_full[x], 1); tc::mbar_init(&acc_empty[x], 128 * C::kSets); }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int rows_per_group = a.n_out / a.groups;
  const int xb = a.tile_n * kKBlk;                      // bytes of one packed activation block
  const int n_sfb = (a.tile_n + 127) / 128;             // its scale chunks
  const uint32_t sf_bytes = (uint32_t)(kSfBytes * (1 + n_sfb));
  const int n_parts = a.spread ? a.splits : 1;          // work items per tile

  // work item -> row tile, token tile, K blocks [k0, k1)
  auto item_tile = [&](int it, int& rt, int& tt, int& p) {
    p = it % n_parts;
    it /= n_parts;
    tt = it % a.tok_tiles;
    rt = it / a.tok_tiles;
  };
  auto item_k = [&](int p, int& k0, int& k1) {
    k0 = a.spread ? part_begin(a.k_blocks, a.splits, p) : 0;
    k1 = a.spread ? part_begin(a.k_blocks, a.splits, p + 1) : a.k_blocks;
  };
  bool ok = true;
  uint32_t issued = 0;                                  // producer: stages filled
  if (warp == 0) {
    // ---- producer.  The weight does not depend on the quantising kernel
    //      ahead: the first stages' weight copies are issued before waiting
    //      for it.
    bool waited = false;
    uint32_t pre = 0;                                   // stages whose weight copies are already issued
    auto put_w = [&](uint32_t x, int rt, int kb, bool sf) {
      uint8_t* st = sm + (size_t)(x % S) * C::kStageBytes;
      tc::mbar_arrive_expect_tx(&full[x % S], (uint32_t)(kWTileBytes + xb) + (sf ? sf_bytes : 0u));
      tc::bulk_g2s(st, a.w + ((int64_t)rt * a.k_blocks + kb) * kWTileBytes, kWTileBytes, &full[x % S]);
      if (sf)
        tc::bulk_g2s(st + kWTileBytes + NT * kKBlk, a.wsf + ((int64_t)rt * a.sup + (kb >> 2)) * kSfBytes, kSfBytes,
                     &full[x % S]);
    };
    auto put_x = [&](uint32_t x, int rt, int tt, int kb, bool sf) {
      uint8_t* st = sm + (size_t)(x % S) * C::kStageBytes;
      const int64_t grp = (rt * kRowTile) / rows_per_group;
      tc::bulk_g2s(st + kWTileBytes, a.xp + ((grp * a.k_blocks + kb) * a.tok_tiles + tt) * xb, (uint32_t)xb, &full[x % S]);
      if (sf)
        tc::bulk_g2s(st + kWTileBytes + NT * kKBlk + kSfBytes,
                     a.xsf + ((grp * a.sup + (kb >> 2)) * a.tok_tiles + tt) * n_sfb * kSfBytes,
                     (uint32_t)(kSfBytes * n_sfb), &full[x % S]);
    };
    {
      int rt, tt, p, k0, k1;
      item_tile(blockIdx.x, rt, tt, p);
      item_k(p, k0, k1);
      pre = (uint32_t)(k1 - k0 < S ? k1 - k0 : S);
      if (tc::elect_one())
        for (uint32_t x = 0; x < pre; ++x) put_w(x, rt, k0 + (int)x, x == 0 || ((k0 + (int)x) & 3) == 0);
      __syncwarp();
    }
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      int rt, tt, p, k0, k1;
      item_tile(it, rt, tt, p);
      item_k(p, k0, k1);
      if (!waited) { tc::griddep_wait(); waited = true; }
      for (int kb = k0; kb < k1; ++kb) {
        const uint32_t x = issued;
        if (x >= (uint32_t)S) ok = tc::mbar_wait(&empty[x % S], ((x / S) - 1) & 1, kLimit) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool sf = kb == k0 || (kb & 3) == 0;
        if (tc::elect_one()) {
          if (x >= pre) put_w(x, rt, kb, sf);
          put_x(x, rt, tt, kb, sf);
        }
        __syncwarp();
        issued = x + 1;
      }
    }
    if (!ok) *abort_flag = 1;
    if (issued < pre) {       // (an abort in between) the stages whose weight copies are in flight without their tokens
      if (tc::elect_one())
        for (uint32_t x = issued; x < pre; ++x) tc::mbar_wait(&full[x % S], 0, 1000ull);
      __syncwarp();
    }
  } else if (warp == 1) {
    // ---- scale copies and MMAs
    uint32_t x = 0, u = 0, nsf = 0;                     // stage, accumulator and scale-buffer counters
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      int rt, tt, p, k0, k1;
      item_tile(it, rt, tt, p);
      item_k(p, k0, k1);
      const int q0 = a.spread ? p : 0, q1 = a.spread ? p + 1 : a.splits;
      for (int q = q0; q < q1 && ok; ++q, ++u) {
        const int b0 = part_begin(a.k_blocks, a.splits, q), b1 = part_begin(a.k_blocks, a.splits, q + 1);
        const uint32_t acc = tmem + (u & 1) * NT;
        if (u >= 2) ok = tc::mbar_wait(&acc_empty[u & 1], ((u >> 1) - 1) & 1, kLimit);
        for (int kb = b0; kb < b1; ++kb, ++x) {
          ok = ok && tc::mbar_wait(&full[x % S], (x / S) & 1, kLimit) && !*abort_flag;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::tc_fence_after();
          const bool sf = kb == k0 || (kb & 3) == 0;
          if (sf) ++nsf;
          // A scale buffer is rewritten three loads after its own: by then the
          // MMAs that read it are complete, for the stage just waited for was
          // free (S <= 8 blocks back), or the accumulator two tiles back was.
          const uint32_t sfc = tmem + C::kSfBase + ((nsf - 1) % kSfRing) * C::kSfCols;
          const uint32_t wb = tc::smem_u32(sm + (size_t)(x % S) * C::kStageBytes), xbase = wb + kWTileBytes;
          if (tc::elect_one()) {
            if (sf) {
              const uint32_t sb = wb + kWTileBytes + NT * kKBlk;
              tc::tmem_cp_32x128b_x4(sfc, tc::smem_desc(sb, 128, 128));
              for (int ch = 0; ch < n_sfb; ++ch)
                tc::tmem_cp_32x128b_x4(sfc + 4 + 4 * ch, tc::smem_desc(sb + kSfBytes * (1 + ch), 128, 128));
            }
            const uint32_t id = kb & 3;
            const uint32_t idesc = tc::idesc_mxf8(kRowTile, a.tile_n, id, id);
#pragma unroll
            for (int m = 0; m < 4; ++m)
              tc::mma_mxf8(acc, tc::smem_desc(wb + m * 256, 128, 1024), tc::smem_desc(xbase + m * 256, 128, 1024), idesc,
                           sfc | (id << 30), (sfc + 4) | (id << 30), (kb > b0 || m > 0) ? 1u : 0u);
            tc::mma_commit(&empty[x % S]);
            if (kb == b1 - 1) tc::mma_commit(&acc_full[u & 1]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ---- epilogue.  After an abort the warps still walk every item and reach
    //      every named barrier (the work is skipped), so that none is left
    //      waiting at a barrier another has left.
    tc::griddep_wait();                                 // the part counters are cleared; outputs may be written
    const int q4 = warp & 3, set = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const int c_lo = set * C::kCols;
    const int et = tid - 64;
    uint32_t u = 0;
    for (int it = blockIdx.x; it < a.items; it += gridDim.x) {
      int rt, tt, p;
      item_tile(it, rt, tt, p);
      const int q0 = a.spread ? p : 0, q1 = a.spread ? p + 1 : a.splits;
      const int o = rt * kRowTile + q4 * 32 + lane;
      const int t0 = tt * a.tile_n;
      const int n_here = min(a.tile_n, a.n_tok - t0) - c_lo;      // this set's tokens (may be <= 0)
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
      int sg = 0;
      while (sg + 1 < a.out.n_seg && o >= a.out.seg_end[sg]) ++sg;
      const int r0 = sg > 0 ? a.out.seg_end[sg - 1] : 0;
      const int64_t rows = a.out.seg_end[sg] - r0;
      const bool bf = (a.out.bf16_mask >> sg) & 1u;
      void* y = a.out.y[sg];
      const int64_t y0 = (int64_t)(t0 + c_lo) * rows + (o - r0);
      const bool partial = a.spread && a.splits > 1;
      if (ok && o < a.n_out) {
        float* pw = partial ? a.part + ((int64_t)p * a.n_tok + t0 + c_lo) * a.n_out + o : nullptr;
#pragma unroll
        for (int e = 0; e < C::kCols; ++e) {
          if (e < n_here) {
            if (partial) pw[(int64_t)e * a.n_out] = acc[e];
            else g_store(y, y0 + (int64_t)e * rows, bf, acc[e]);
          }
        }
      }
      if (partial) {
        // the item that finishes the tile last adds the parts in part order
        __threadfence();
        tc::named_bar_sync(1, 128 * C::kSets);
        if (et == 0) last_flag[0] = atomicAdd(&a.done[rt * a.tok_tiles + tt], 1) == a.splits - 1 ? 1 : 0;
        tc::named_bar_sync(1, 128 * C::kSets);
        const bool last = last_flag[0] != 0;
        tc::named_bar_sync(1, 128 * C::kSets);          // (the flag is read before the next item writes it)
        if (last && ok && o < a.n_out) {
          __threadfence();
          const int64_t n = (int64_t)a.n_tok * a.n_out;
          const int n_mine = min(n_here, C::kCols);
          for (int e = 0; e < n_mine; ++e) {
            const float* pr = a.part + (int64_t)(t0 + c_lo + e) * a.n_out + o;
            float s = 0.f;
            for (int p0 = 0; p0 < a.splits; p0 += 16) {
              float v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = p0 + j < a.splits ? __ldcg(pr + (p0 + j) * n) : 0.f;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (p0 + j < a.splits) s = p0 + j == 0 ? v[j] : s + v[j];
            }
            g_store(y, y0 + (int64_t)e * rows, bf, s);
          }
        }
      }
    }
    if (!ok) *abort_flag = 1;
  }
  tc::tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    if (atomicCAS(&g_fp8_err[0], 0, (int32_t)kErrTimeout) == 0) g_fp8_err[1] = (int32_t)blockIdx.x;
    // let the copies already issued land before the shared memory goes away
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
  const int e = finite ? fp8_exponent(bf16_val((uint16_t)top)) : 0;
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
  int row_tiles, k_blocks, sup, splits, nt, tok_tiles, tile_n, chunks, spread, items;
  size_t xp, xsf, part, done, total;      // workspace offsets and size
};

// K parts of a weight: a function of its shape and the device alone.  As many
// as give every SM two work items of a few-token call, each at least
// kMinPartBlocks blocks long.
int fp8_splits(int row_tiles, int k_blocks, int sms) {
  int s = 2 * sms / row_tiles;
  if (s > k_blocks / kMinPartBlocks) s = k_blocks / kMinPartBlocks;
  return s < 1 ? 1 : s;
}

Plan fp8_plan(int n_out, int k_in, int groups, int n_tok, int sms) {
  Plan p{};
  p.row_tiles = (n_out + kRowTile - 1) / kRowTile;
  p.k_blocks = (k_in / groups + kKBlk - 1) / kKBlk;
  p.sup = (p.k_blocks + 3) / 4;
  p.splits = fp8_splits(p.row_tiles, p.k_blocks, sms);
  p.nt = n_tok <= 32 ? 32 : n_tok <= 64 ? 64 : n_tok <= 128 ? 128 : 224;
  p.tok_tiles = (n_tok + p.nt - 1) / p.nt;
  // equal tiles, in steps of 32 tokens
  p.tile_n = ((n_tok + p.tok_tiles - 1) / p.tok_tiles + 31) / 32 * 32;
  p.chunks = (p.tile_n + 127) / 128;
  p.spread = p.row_tiles * (int64_t)p.tok_tiles < sms ? 1 : 0;
  p.items = p.row_tiles * p.tok_tiles * (p.spread ? p.splits : 1);
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t o = 0;
  p.xp = o;   o += al((size_t)groups * p.k_blocks * p.tok_tiles * p.tile_n * kKBlk);
  p.xsf = o;  o += al((size_t)groups * p.sup * p.tok_tiles * p.chunks * kSfBytes);
  const bool partial = p.spread && p.splits > 1;
  p.part = o; o += al(partial ? (size_t)p.splits * n_tok * n_out * 4 : 0);
  p.done = o; o += al(partial ? (size_t)p.row_tiles * p.tok_tiles * 4 : 0);
  p.total = o;
  return p;
}

template <int NT>
cudaError_t launch_nt(const Fp8Args& a, int sms, cudaStream_t st) {
  using C = Cfg<NT>;
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (setup_needed(attr_set, dev)) {
    e = cudaFuncSetAttribute(fp8_gemm_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fp8_gemm_kernel<NT>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    setup_done(attr_set, dev);
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(a.items < sms * C::kPerSm ? a.items : sms * C::kPerSm));
  lc.blockDim = dim3(C::kThreads);
  lc.dynamicSmemBytes = C::kSmem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, fp8_gemm_kernel<NT>, a);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

size_t fp8_weight_bytes(int n_out, int k_in, int groups) {
  const size_t rt = (n_out + kRowTile - 1) / kRowTile, kb = (k_in / groups + kKBlk - 1) / kKBlk;
  return rt * kb * kWTileBytes + rt * ((kb + 3) / 4) * kSfBytes;
}

size_t fp8_workspace_bytes(int n_out, int k_in, int groups, int n_tok, int sms) {
  return fp8_plan(n_out, k_in, groups, n_tok, sms).total;
}

cudaError_t launch_fp8_pack_weight(const uint8_t* codes, const uint8_t* scales, int n_out, int k_in, int groups,
                                   uint8_t* w, cudaStream_t st) {
  const int kg = k_in / groups, rt = (n_out + kRowTile - 1) / kRowTile, kb = (kg + kKBlk - 1) / kKBlk;
  const bool aligned = kg % 16 == 0 && reinterpret_cast<uintptr_t>(codes) % 16 == 0;
  fp8_pack_w_kernel<<<dim3(kb, rt), 256, 0, st>>>(codes, scales, n_out, kg, kb, (kb + 3) / 4, aligned, w,
                                                  w + (size_t)rt * kb * kWTileBytes);
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
  const bool partial = p.spread && p.splits > 1;
  int32_t* done = partial ? reinterpret_cast<int32_t*>(base + p.done) : nullptr;
  const int kg = k_in / groups;
  const int64_t units = (int64_t)p.k_blocks * p.tok_tiles * p.tile_n * 8;
  const int blocks = (int)std::min<int64_t>((units + 255) / 256, 8 * sms);
  // aligned: every row of every group starts on 16 bytes (kg is a multiple of 8)
  const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0;
  fp8_quant_x_kernel<<<dim3(blocks, groups), 256, 0, st>>>(x, n_tok, kg, (int64_t)k_in, p.k_blocks, p.sup, p.tok_tiles,
                                                           p.tile_n, p.chunks, aligned, base + p.xp, base + p.xsf, done,
                                                           p.row_tiles * p.tok_tiles);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  Fp8Args a{};
  a.w = w;
  a.wsf = w + (size_t)p.row_tiles * p.k_blocks * kWTileBytes;
  a.xp = base + p.xp;
  a.xsf = base + p.xsf;
  a.n_out = n_out; a.n_tok = n_tok;
  a.row_tiles = p.row_tiles; a.k_blocks = p.k_blocks; a.sup = p.sup;
  a.groups = groups; a.splits = p.splits;
  a.tok_tiles = p.tok_tiles; a.tile_n = p.tile_n;
  a.spread = p.spread; a.items = p.items;
  a.out = out;
  a.part = partial ? reinterpret_cast<float*>(base + p.part) : nullptr;
  a.done = done;
  switch (p.nt) {
    case 32: return launch_nt<32>(a, sms, st);
    case 64: return launch_nt<64>(a, sms, st);
    case 128: return launch_nt<128>(a, sms, st);
    default: return launch_nt<224>(a, sms, st);
  }
}

// Read and clear the device error word (the caller has synchronised).
cudaError_t fp8_read_error(int32_t* code, int32_t* detail) {
  int32_t w[2] = {0, 0};
  cudaError_t e = cudaMemcpyFromSymbol(w, g_fp8_err, sizeof w);
  if (e != cudaSuccess) return e;
  *code = w[0];
  *detail = w[1];
  if (w[0] != 0) {
    const int32_t z[2] = {0, 0};
    e = cudaMemcpyToSymbol(g_fp8_err, z, sizeof z);
  }
  return e;
}

}  // namespace csa
