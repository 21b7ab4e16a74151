// RMS norm of every query and key head with the partial RoPE, one launch
// (csa_head_norm):
//     y = w * x / sqrt(mean(x^2) + eps),  then the pairs (2i, 2i+1) of the last
//     R dims rotated by pos * base^(-2i/R)
// The sum of squares, the scale and the rotation are fp32, angles fp64 (as in
// every kernel here: positions reach 2^20); a result is rounded once, to its
// type.
//
// Bound: one read and one write of the heads.  A head stays in the registers
// of the lanes that loaded it (8 values a lane and step; the 2^n lanes that
// cover the head, so a warp takes four heads of 64 dims, one of 512), so each
// value moves once each way.  A block works on heads of one token: it loads
// its first heads, then computes the token's cosines and sines once (fp64, in
// the shadow of the loads), and every further head reuses them.
#include "common.cuh"
#include "head_norm.cuh"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kHnThreads = 128;
constexpr int kHnMaxDim = 1024;

template <typename T>
struct Raw;                            // 8 values as loaded
template <>
struct Raw<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void set(int e, uint16_t b) {
    uint32_t& w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    w |= (uint32_t)b << (16 * (e & 1));
  }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return bf16_val((uint16_t)(e & 1 ? w >> 16 : w & 0xFFFFu));
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void set(int e, float f) {
    float4& q = e < 4 ? a : b;
    ((e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w) = f;
  }
  __device__ __forceinline__ float get(int e) const {
    const float4& q = e < 4 ? a : b;
    return (e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w;
  }
};

__device__ __forceinline__ void put8(uint16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (uint32_t)bf16_rn(v[2 * e]) | ((uint32_t)bf16_rn(v[2 * e + 1]) << 16);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = bf16_rn(v); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }

// Heads [h0, h1) of token t.  NC: steps of 8 values a lane takes; U: heads
// whose loads are in flight at once.
template <typename T, int NC, int U>
__device__ __forceinline__ void norm_heads(const HeadNormArgs& a, const HeadNormPart& p, int64_t t, int h0, int h1,
                                           float2* cs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lph = a.lanes, l = lane & (lph - 1);
  const int per_warp = 32 / lph, slots = (kHnThreads / 32) * per_warp;
  const int slot = warp * per_warp + lane / lph;
  const int D = a.dim, rot0 = p.rotate ? D - a.rope : D;
  const T* x = static_cast<const T*>(p.x) + t * p.x_tok;
  T* y = static_cast<T*>(p.y) + t * p.y_tok;
  float w[NC][8];
  bool first = true;
  for (int hb = h0; hb < h1; hb += slots * U) {
    Raw<T> raw[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * slots + slot;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d0 = (c * lph + l) * 8;
        raw[u][c].zero();
        if (h < h1 && d0 < D) {
          const T* px = x + h * p.x_head + d0;
          if (p.vec) {
            raw[u][c].load(px);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (d0 + e < D) raw[u][c].set(e, px[e]);
          }
        }
      }
    }
    if (first) {
      first = false;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = (c * lph + l) * 8 + e;
          w[c][e] = p.weight != nullptr && d < D ? __ldg(p.weight + d) : 1.f;
        }
      if (p.rotate) {
        const int64_t pos = a.positions[t];
        for (int i = threadIdx.x; i < a.rope / 2; i += kHnThreads) {
          float c = 1.f, s = 0.f;
          rope_pair(c, s, a.theta[i], pos);            // rotating (1, 0) gives (cos, sin)
          cs[i] = make_float2(c, s);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * slots + slot;
      float v[NC][8], ss = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[c][e] = raw[u][c].get(e);
          ss = fmaf(v[c][e], v[c][e], ss);
        }
      for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      // Squares beyond fp32's range (a sum that overflowed, or one that may
      // have lost its small squares while eps does not cover them): the sum
      // and the scale again, in fp64.
      const bool wide = !(ss <= 3.0e38f) || (ss < 1e-30f && a.eps < 1e-20);
      if (__any_sync(0xffffffffu, wide)) {
        double s2 = 0.0;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) s2 += (double)v[c][e] * v[c][e];
        for (int o = lph >> 1; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        const double r = 1.0 / sqrt(s2 / D + a.eps), r32 = (double)__frcp_rn(sqrtf(ss / (float)D + (float)a.eps));
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] = wide ? (float)(v[c][e] * r) : v[c][e] * (float)r32;
      } else {
        const float r = __frcp_rn(sqrtf(ss / (float)D + (float)a.eps));
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] *= r;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d0 = (c * lph + l) * 8;
        if (h >= h1 || d0 >= D) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] *= w[c][e];
        if (d0 + 8 > rot0) {
#pragma unroll
          for (int e = 0; e < 8; e += 2)
            if (d0 + e >= rot0 && d0 + e < D) {        // D and rot0 are even: a pair never straddles
              const float2 q = cs[(d0 + e - rot0) >> 1];
              const float x0 = v[c][e], x1 = v[c][e + 1];
              v[c][e] = fmaf(x0, q.x, -(x1 * q.y));
              v[c][e + 1] = fmaf(x0, q.y, x1 * q.x);
            }
        }
        T* py = y + h * p.y_head + d0;
        if (p.vec) {
          put8(py, v[c]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (d0 + e < D) put1(py + e, v[c][e]);
        }
      }
    }
  }
}

template <int NC>
__global__ void __launch_bounds__(kHnThreads) head_norm_kernel(const __grid_constant__ HeadNormArgs a) {
  __shared__ float2 cs[kHnMaxDim / 2];
  const int per_tok = a.part[0].blocks + a.part[1].blocks;
  const int64_t t = blockIdx.x / per_tok;
  int b = blockIdx.x % per_tok;
  const int which = b >= a.part[0].blocks ? 1 : 0;
  const HeadNormPart& p = a.part[which];
  if (which) b -= a.part[0].blocks;
  const int h0 = b * p.block_heads, h1 = min(p.heads, h0 + p.block_heads);
  constexpr int U = NC == 1 ? 4 : NC == 2 ? 2 : 1;
  if (p.f32) norm_heads<float, NC, U>(a, p, t, h0, h1, cs);
  else norm_heads<uint16_t, NC, U>(a, p, t, h0, h1, cs);
}

}  // namespace

int head_norm_max_dim() { return kHnMaxDim; }

cudaError_t launch_head_norm(HeadNormArgs a, int sms, cudaStream_t st) {
  const int steps = (a.dim + 7) / 8;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < steps) a.lanes *= 2;
  const int nc = (steps + 31) / 32;
  const int slots = (kHnThreads / 32) * (32 / a.lanes);
  int64_t per_tok = 0;
  for (HeadNormPart& p : a.part) {
    if (p.heads == 0) { p.blocks = 0; p.block_heads = 1; continue; }
    const int esz = p.f32 ? 4 : 2, al = 16 / esz;
    p.vec = a.dim % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 &&
            p.x_tok % al == 0 && p.x_head % al == 0 && p.y_tok % al == 0 && p.y_head % al == 0;
    // A token's heads in one block once the tokens alone give every SM 8
    // blocks; for fewer tokens the heads are spread over blocks of one pass.
    const int64_t want = (8LL * sms + a.n_tok - 1) / a.n_tok;
    int64_t bh = (p.heads + want - 1) / want;
    bh = (bh + slots - 1) / slots * slots;
    p.block_heads = (int)bh;
    p.blocks = (int)((p.heads + bh - 1) / bh);
    per_tok += p.blocks;
  }
  const int64_t grid = per_tok * a.n_tok;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (grid == 0) return cudaSuccess;
  const dim3 g((unsigned)grid);
  if (nc == 1) head_norm_kernel<1><<<g, kHnThreads, 0, st>>>(a);
  else if (nc == 2) head_norm_kernel<2><<<g, kHnThreads, 0, st>>>(a);
  else head_norm_kernel<4><<<g, kHnThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace csa
