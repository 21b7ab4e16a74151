// The FP8 product (proj_fp8.cu) of many tokens, by pairs of SMs.
//
// What bounds it.  A 128 x 224 tile of one SM moves 84 KB through its shared
// memory for every block of 128 columns (42 KB copied in, 42 KB read by the
// MMAs), 656 cycles at 128 bytes a cycle, where the MMAs take 448.  Two SMs that
// work on one 256 x 224 tile (tcgen05 cta_group::2) each hold 128 tokens and half
// of the features and read 60 KB a block, 470 cycles.
//
// Tokens are the MMA's M here and features its N, so that a thread holds a
// token's consecutive features and stores them 32 bytes at a time (features as
// M left a thread one 2-byte store per token and feature: 9000 cycles a tile,
// twice the MMAs' time at K = 1024).  Rows that are not on 32 bytes are exchanged
// within the warp first (4096 x 1000 x 2048 by this kernel: 22 us, value by
// value 52; 3000 tokens x 5000 fp32 and 15000 BF16 features x 232: 54, exchanged
// as single features 91).  An element is the same sum of the same
// products in the same order as with the operands exchanged.
//
// Roles: in both CTAs warp 0 copies its own tokens and its half of the features;
// the second CTA's warp 1 passes the completion of its copies on to the first,
// whose warp 1 issues the scale copies and MMAs for both; warps 2-9 read the
// accumulators (two, so that the next tile's MMAs run meanwhile).
#include <cooperative_groups.h>

#include <algorithm>

#include "proj_fp8.cuh"
#include "tc.cuh"

namespace csa {

namespace cg = cooperative_groups;

// Device error word of this kernel: first error wins.
__device__ int32_t g_pair_err[2];

namespace {

constexpr int kPairThreads = 64 + 256;
constexpr int kHalfBytes = kPairFeatures / 2 * kKBlk;           // most bytes of a CTA's half of the features
constexpr int kPairSf = 3 * kSfBytes;                           // scales: own tokens, all features
constexpr int kPairStage = kWTileBytes + kHalfBytes + kPairSf;
constexpr int kPairStages = 224 * 1024 / kPairStage;
constexpr size_t kPairSmem = (size_t)kPairStages * kPairStage + 256 + 128;
constexpr uint32_t kPairASf = 2 * kPairFeatures, kPairBSf = kPairASf + 4 * kSfRing;   // TMEM columns
constexpr int kSetCols = kPairFeatures / 2;                     // accumulator columns of four warps
static_assert(kPairBSf + 8 * kSfRing <= 512, "TMEM");
static_assert(kPairStages >= 4 && kPairStages <= 8, "stages");

// Of N words a lane, word i of lane l of a group of N goes to word l of lane i.
template <int N>
__device__ __forceinline__ void exchange(uint32_t (&w)[N]) {
#pragma unroll
  for (int s = N / 2; s > 0; s >>= 1) {
    const bool up = threadIdx.x & s;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & s)) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + s], s);
        w[i] = up ? got : w[i];
        w[i + s] = up ? w[i + s] : got;
      }
  }
}

// Stores of a warp's tokens (t0 + lane, below n_tok), features f, f + 1, ...,
// f + n - 1 (of the weight), 16 at a time.  Where they lie in one segment, and
// every token's on 32 bytes, a lane stores its token's 16 in one or two stores.
// Else lanes exchange values first, so that a store is neighbouring features
// of few tokens: in one segment pairs of features within 8 lanes (a store is 8
// pairs of four tokens; two of single features where pairs are not aligned),
// across segments single features within 16.
struct TokenOut {
  const GemmOut* out;
  int t0, n_tok, f, n;
  char* row;             // token t0's feature f
  int64_t step;          // bytes of a token's row
  bool bf16, one, wide, even;   // one: one segment; wide, even: every token on 32 bytes, on a pair of values

  __device__ __forceinline__ TokenOut(const GemmOut& o, int t0_, int n_tok_, int f_, int n_)
      : out(&o), t0(t0_), n_tok(n_tok_), f(f_), n(n_), row(nullptr), step(0), bf16(false), one(false), wide(false), even(false) {
    if (n <= 0) return;
    int sg = 0;
    while (sg + 1 < o.n_seg && f >= o.seg_end[sg]) ++sg;
    const int r0 = sg > 0 ? o.seg_end[sg - 1] : 0, el = (o.bf16_mask >> sg) & 1u ? 2 : 4;
    bf16 = el == 2;
    step = (int64_t)(o.seg_end[sg] - r0) * el;
    row = static_cast<char*>(o.y[sg]) + t0 * step + (int64_t)(f - r0) * el;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row) | (n_tok - t0 > 1 ? step : 0);
    one = f + n <= o.seg_end[sg];
    wide = one && at % 32 == 0;
    even = at % (2 * el) == 0;
  }
  __device__ __forceinline__ void put(int c, const uint32_t* v) const {       // features f + c .. f + c + 15
    if (c >= n) return;
    const int lane = threadIdx.x & 31;
    if (one && c + 16 <= n) {
      if (bf16) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (wide) {
          if (t0 + lane < n_tok) tc::st_global_32b(row + lane * step + 2 * c, w);
        } else {
          exchange(w);
          char* q = row + (lane & 24) * step + 2 * c + 4 * (lane & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i, q += step)
            if (t0 + (lane & 24) + i < n_tok) {
              if (even) {
                *reinterpret_cast<uint32_t*>(q) = w[i];
              } else {
                reinterpret_cast<uint16_t*>(q)[0] = (uint16_t)w[i];
                reinterpret_cast<uint16_t*>(q)[1] = (uint16_t)(w[i] >> 16);
              }
            }
        }
      } else if (wide) {
        if (t0 + lane < n_tok) {
          tc::st_global_32b(row + lane * step + 4 * c, v);
          tc::st_global_32b(row + lane * step + 4 * c + 32, v + 8);
        }
      } else {
        uint32_t a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) { a[e] = v[2 * e]; b[e] = v[2 * e + 1]; }
        exchange(a);
        exchange(b);
        char* q = row + (lane & 24) * step + 4 * c + 8 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i, q += step)
          if (t0 + (lane & 24) + i < n_tok) {
            if (even) {
              *reinterpret_cast<uint2*>(q) = make_uint2(a[i], b[i]);
            } else {
              reinterpret_cast<uint32_t*>(q)[0] = a[i];
              reinterpret_cast<uint32_t*>(q)[1] = b[i];
            }
          }
      }
    } else {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = v[e];
      exchange(w);
      const int fe = lane & 15, t = t0 + (lane & 16);
      if (c + fe < n) {                                  // w[i]: this feature of token t + i
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(w[e]);
        out_row(*out, f + c + fe).store16(t, n_tok - t, x);
      }
    }
    __syncwarp();
  }
};

}  // namespace

__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const __grid_constant__ Fp8PairArgs a) {
  constexpr int S = kPairStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + (size_t)S * kPairStage);   // first CTA: both CTAs' copies; second: its own
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;                  // used in the first CTA
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_slot = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  constexpr uint64_t kLimit = 1000000000ull;
  constexpr int kBOff = kWTileBytes, kASfOff = kBOff + kHalfBytes, kBSfOff = kASfOff + kSfBytes;   // in a stage
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)(blockIdx.x & 1);              // in the cluster (two consecutive blocks)

  tc::griddep_launch_dependents();
  if (warp == 1) {
    tc::pair_tmem_alloc(tmem_slot, 512);
    tc::pair_tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) { tc::mbar_init(&full[s], rank == 0 ? 2 : 1); tc::mbar_init(&empty[s], 1); }
    for (int x = 0; x < 2; ++x) { tc::mbar_init(&acc_full[x], 1); tc::mbar_init(&acc_empty[x], 16); }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    *issued_slot = 0;
    tc::fence_mbar_init();
  }
  tc::tc_fence_before();
  cluster.sync();                                      // both CTAs' barriers are set up
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int rpg = a.n_out / a.groups;
  const int m_tiles = a.tok_tiles / 2;
  const int it0 = blockIdx.x / 2, it_step = gridDim.x / 2;
  // The tiles of this pair: token pair m and feature tile ft, stepped without
  // divisions; group, first feature f0 (of the weight), features n (a multiple
  // of 16).
  struct Walk {
    int it, m, ft, dm, dft;
  };
  Walk wk{it0, it0 % m_tiles, it0 / m_tiles, it_step % m_tiles, it_step / m_tiles};
  auto next = [&]() {
    wk.it += it_step;
    wk.m += wk.dm;
    wk.ft += wk.dft;
    if (wk.m >= m_tiles) { wk.m -= m_tiles; ++wk.ft; }
  };
  auto tile = [&](int& grp, int& f0, int& n) {
    grp = a.groups == 1 ? 0 : wk.ft / a.f_tiles;
    f0 = (wk.ft - grp * a.f_tiles) * a.tile_f;
    n = min(a.tile_f, (rpg - f0 + 15) / 16 * 16);
    f0 += grp * rpg;
  };
  bool ok = true;
  if (warp == 0) {
    // ---- producer of this CTA (one thread)
    if (tc::elect_one()) {
      // (every instruction between two blocks counts: addresses run along)
      uint32_t x = 0, st = 0, ph = 1;                  // (a fresh barrier's wait for phase 1 passes)
      const int64_t xp_step = (int64_t)a.tok_tiles * kWTileBytes, xsf_step = (int64_t)a.tok_tiles * kSfBytes;
      const uint32_t sm0 = tc::smem_u32(sm), full0 = tc::smem_u32(full);
      tc::griddep_wait();
      for (; wk.it < a.tiles && ok; next()) {
        int grp, f0, n;
        tile(grp, f0, n);
        const int m = wk.m;
        const int half = n / 2, f = f0 + rank * half;
        const int rt = f / kRowTile, r0 = f % kRowTile;
        const uint32_t b1 = (uint32_t)min(half, kRowTile - r0) * kKBlk, b2 = (uint32_t)half * kKBlk - b1;
        const uint8_t* w1 = a.w + (int64_t)rt * a.k_blocks * kWTileBytes + r0 * kKBlk;
        const uint8_t* w2 = a.w + (int64_t)(rt + 1) * a.k_blocks * kWTileBytes;
        const uint8_t* xp = a.xp + ((int64_t)grp * a.k_blocks * a.tok_tiles + 2 * m + rank) * kWTileBytes;
        const uint8_t* xsf = a.xsf + ((int64_t)grp * a.sup * a.tok_tiles + 2 * m + rank) * kSfBytes;
        const uint8_t* wsf = a.wsf + (int64_t)wk.ft * a.sup * 2 * kSfBytes;
        const uint32_t bytes = (uint32_t)kWTileBytes + b1 + b2;
        for (int kb = 0; kb < a.k_blocks; ++kb) {
          ok = tc::mbar_wait(&empty[st], ph, kLimit);
          if (!ok) break;
          const uint32_t at = sm0 + st * kPairStage, bar = full0 + st * 8;
          if ((kb & 3) == 0) {
            tc::mbar_expect_tx_at(bar, bytes + kPairSf);
            tc::bulk_g2s_at(at + kASfOff, xsf, kSfBytes, bar);
            tc::bulk_g2s_at(at + kBSfOff, wsf, 2 * kSfBytes, bar);
            xsf += xsf_step;
            wsf += 2 * kSfBytes;
          } else {
            tc::mbar_expect_tx_at(bar, bytes);
          }
          tc::bulk_g2s_at(at, xp, kWTileBytes, bar);
          tc::bulk_g2s_at(at + kBOff, w1, b1, bar);
          if (b2) tc::bulk_g2s_at(at + kBOff + b1, w2, b2, bar);
          xp += xp_step;
          w1 += kWTileBytes;
          w2 += kWTileBytes;
          ++x;
          if (++st == S) { st = 0; ph ^= 1; }
        }
      }
      *issued_slot = x;
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp == 1 && rank == 1) {
    // ---- this CTA's copies of a stage have landed: tell the first CTA
    if (tc::elect_one()) {
      uint32_t st = 0, ph = 0;
      for (int it = it0; it < a.tiles && ok; it += it_step)
        for (int kb = 0; kb < a.k_blocks; ++kb) {
          ok = tc::mbar_wait(&full[st], ph, kLimit);
          if (!ok) break;
          tc::mbar_arrive_cluster(&full[st], 0);
          if (++st == S) { st = 0; ph ^= 1; }
        }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- scale copies and MMAs of both CTAs (one thread)
    if (tc::elect_one()) {
      const uint32_t desc_hi = tc::smem_desc_hi(1024), sf_hi = tc::smem_desc_hi(128);
      const uint32_t lo0 = tc::smem_desc_lo(tc::smem_u32(sm), 128);
      constexpr uint32_t kIdStep = (1u << 29) | (1u << 4);
      uint32_t st = 0, ph = 0, u = 0, r = kSfRing - 1;
      for (; wk.it < a.tiles && ok; next()) {
        int grp, f0, n;
        tile(grp, f0, n);
        const uint32_t idesc0 = tc::idesc_mxf8(2 * kRowTile, n, 0, 0);
        int kb = 0;
        for (int q = 0; q < 1 << a.split_lg && ok; ++q, ++u) {
          const int b1 = part_begin(a.k_blocks, a.split_lg, q + 1);
          const uint32_t acc = tmem + (u & 1) * kPairFeatures;
          if (u >= 2) ok = tc::mbar_wait_cluster(&acc_empty[u & 1], ((u >> 1) - 1) & 1, kLimit);
          for (uint32_t more = 0; kb < b1; ++kb, more = 1) {
            ok = ok && tc::mbar_wait_cluster(&full[st], ph, kLimit);
            if (!ok) break;
            tc::tc_fence_after();
            // (a scale buffer is rewritten 16 blocks or two tiles after its
            // load, when the MMAs that read it are complete)
            const bool sf = (kb & 3) == 0;
            if (sf) r = (r + 1) & (kSfRing - 1);
            const uint32_t id = kb & 3, lo = lo0 + st * (kPairStage / 16);
            const uint32_t asf = tmem + kPairASf + r * 4, bsf = tmem + kPairBSf + r * 8;
            const uint32_t asf_id = asf | (id << 30), bsf_id = bsf | (id << 30);
            const uint32_t idesc = idesc0 + id * kIdStep;
            if (sf) {
              tc::pair_tmem_cp(asf, tc::desc64(lo + kASfOff / 16, sf_hi));
              tc::pair_tmem_cp(bsf, tc::desc64(lo + kBSfOff / 16, sf_hi));
              tc::pair_tmem_cp(bsf + 4, tc::desc64(lo + (kBSfOff + kSfBytes) / 16, sf_hi));
            }
            tc::pair_mma_mxf8(acc, tc::desc64(lo, desc_hi), tc::desc64(lo + kBOff / 16, desc_hi), idesc, asf_id, bsf_id, more);
#pragma unroll
            for (int k = 1; k < 4; ++k)
              tc::pair_mma_mxf8(acc, tc::desc64(lo + k * 16, desc_hi), tc::desc64(lo + kBOff / 16 + k * 16, desc_hi), idesc,
                                asf_id, bsf_id, 1u);
            tc::pair_commit(&empty[st]);
            if (kb + 1 == b1) tc::pair_commit(&acc_full[u & 1]);
            if (++st == S) { st = 0; ph ^= 1; }
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ---- epilogue: a thread is a token of this CTA, set 0 or 1 the features' halves
    tc::griddep_wait();
    const int q4 = warp & 3, set = (warp - 2) >> 2;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    uint32_t u = 0;
    for (; wk.it < a.tiles; next()) {
      int grp, f0, n;
      tile(grp, f0, n);
      const int t0 = (2 * wk.m + rank) * kRowTile + q4 * 32;
      // this set's columns: the first or second half in steps of 16
      const int c_lo = set == 0 ? 0 : (n / 16 + 1) / 2 * 16, c_n = (set == 0 ? (n / 16 + 1) / 2 * 16 : n) - c_lo;
      const int f_end = grp * rpg + min(rpg, f0 - grp * rpg + n);
      const TokenOut y(a.out, t0, a.n_tok, f0 + c_lo, min(c_n, f_end - f0 - c_lo));
      if (a.split_lg == 0) {
        ok = ok && tc::mbar_wait(&acc_full[u & 1], (u >> 1) & 1, kLimit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc::tc_fence_after();
        // the accumulator is free once its last columns have been read
        const uint32_t base = tmem + lane_base + (u & 1) * kPairFeatures + c_lo;
        for (int c = 0; c < c_n; c += 16) {
          uint32_t v[16];
          tc::tmem_ld_x16(base + c, v);
          tc::tmem_wait_ld();
          if (c + 16 >= c_n) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(&acc_empty[u & 1], 0);
          }
          y.put(c, v);
        }
        if (c_n <= 0 && lane == 0) tc::mbar_arrive_cluster(&acc_empty[u & 1], 0);
        ++u;
      } else {
        float acc[kSetCols];
        for (int q = 0; q < 1 << a.split_lg; ++q, ++u) {
          ok = ok && tc::mbar_wait(&acc_full[u & 1], (u >> 1) & 1, kLimit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < kSetCols; c += 16)
            if (c < c_n) {
              uint32_t v[16];
              tc::tmem_ld_x16(tmem + lane_base + (u & 1) * kPairFeatures + c_lo + c, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[c + e] = q == 0 ? __uint_as_float(v[e]) : acc[c + e] + __uint_as_float(v[e]);
            }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(&acc_empty[u & 1], 0);
        }
        if (!ok) continue;
#pragma unroll
        for (int c = 0; c < kSetCols; c += 16)
          if (c < c_n) y.put(c, reinterpret_cast<const uint32_t*>(acc) + c);
      }
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  if (warp == 1 && rank == 0) {
    // no MMA of the pair is in flight when either CTA's memory is released
    if (tc::elect_one()) tc::pair_commit_own(drain);
    __syncwarp();
    tc::mbar_wait(drain, 0, 200000000ull);
  }
  if (*abort_flag && tid == 0) {
    if (atomicCAS(&g_pair_err[0], 0, (int32_t)kErrTimeout) == 0) g_pair_err[1] = (int32_t)blockIdx.x;
    // let the copies already issued land before the shared memory goes away
    const uint32_t issued = *issued_slot;
    for (uint32_t x = issued > (uint32_t)S ? issued - S : 0; x < issued; ++x)
      tc::mbar_wait(&full[x % S], (x / S) & 1, 200000000ull);
  }
  tc::tc_fence_before();
  cluster.sync();
  if (warp == 1) tc::pair_tmem_dealloc(tmem, 512);
  cluster.sync();
}

cudaError_t launch_fp8_pair(const Fp8PairArgs& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (setup_needed(attr_set, dev)) {
    e = cudaFuncSetAttribute(fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    setup_done(attr_set, dev);
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(2 * std::min(a.tiles, sms / 2)));
  lc.blockDim = dim3(kPairThreads);
  lc.dynamicSmemBytes = kPairSmem;
  lc.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = 2;
  e = cudaLaunchKernelEx(&lc, fp8_pair_kernel, a);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t fp8_pair_read_error(int32_t w[2]) {
  cudaError_t e = cudaMemcpyFromSymbol(w, g_pair_err, 2 * sizeof(int32_t));
  if (e != cudaSuccess || w[0] == 0) return e;
  const int32_t z[2] = {0, 0};
  return cudaMemcpyToSymbol(g_pair_err, z, sizeof z);
}

}  // namespace csa
