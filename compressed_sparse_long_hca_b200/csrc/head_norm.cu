// RMS norm of every query and key head with the partial RoPE, one launch
// (csa_head_norm):
//     y = w * x / sqrt(mean(x^2) + eps),  then the pairs (2i, 2i+1) of the last
//     R dims rotated by pos * base^(-2i/R)
// The sum of squares, the scale and the rotation are fp32, angles are reduced
// in fp64 (positions reach 2^20); a result is rounded once, to its type.
//
// Bound: one read and one write of the heads.  A head stays in the registers
// of the lanes that loaded it (8 values a lane and step; the 2^n lanes that
// cover the head, so a warp takes four heads of 64 dims, one of 512), so each
// value moves once each way.  A block works on heads of one token: it loads
// its first heads, then computes the token's cosines and sines once, in the
// shadow of the loads, and every further head reuses them; the next heads'
// loads are issued before the present ones are worked on (4 blocks of 128
// threads an SM: the registers that the loads in flight take are worth more
// than more blocks).  Where many tokens have few heads each, a block takes a
// run of tokens instead.  4096 tokens x (128 BF16 + 1 fp32) heads of 512 on one
// B200: 190 us, 5.75 TB/s or 0.88 of a device copy; without the loads ahead
// 214 us at best (7 blocks), with one value at a time instead of packed fp32
// pairs and fp64 sines 351 us.
#include <algorithm>

#include "common.cuh"
#include "head_norm.cuh"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kHnThreads = 128;
constexpr int kHnMaxDim = 1024;

// Two fp32 values in one 64-bit register pair, and their packed arithmetic.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Cosine and sine of an angle, each within a few fp32 half steps: the angle in
// half turns and its reduction in fp64, its fp32 value by sincospif, what that
// rounding left by the first-order term.
__device__ __forceinline__ float2 cos_sin(double angle) {
  const double turns = angle * 0.15915494309189535;      // 1 / (2 pi)
  const double half = 2.0 * (turns - rint(turns));
  const float hi = (float)half, lo = (float)((half - (double)hi) * 3.141592653589793);
  float s, c;
  sincospif(hi, &s, &c);
  return make_float2(fmaf(-lo, s, c), fmaf(lo, c, s));
}

// 8 values of a head as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load(const uint16_t* p, int n) {          // the first n, the others zero
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint64_t get(int i) const {                    // values 2 i, 2 i + 1
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void store(uint16_t* p, const uint64_t (&y)[4], int n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(y[i]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (n < 0) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = (uint16_t)(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    }
  }
};
template <>
struct Raw<float> {
  uint64_t v[4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0;
  }
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = pair(a.x, a.y); v[1] = pair(a.z, a.w); v[2] = pair(b.x, b.y); v[3] = pair(b.z, b.w);
  }
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(2 * i < n ? p[2 * i] : 0.f, 2 * i + 1 < n ? p[2 * i + 1] : 0.f);
  }
  __device__ __forceinline__ uint64_t get(int i) const { return v[i]; }
  static __device__ __forceinline__ void store(float* p, const uint64_t (&y)[4], int n) {
    const float2 a = unpair(y[0]), b = unpair(y[1]), c = unpair(y[2]), d = unpair(y[3]);
    if (n < 0) {
      reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
      reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
    } else {
      const float f[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = f[e];
    }
  }
};

// A head (`wide`) whose squares leave fp32's range: its sum overflowed, or may
// have lost small squares that eps does not cover.  Its values are scaled by a
// power of two and summed again, the scale `r` follows in fp64; the warp's
// other heads stay as they are.  All lanes of the warp call it.
template <int NC>
__device__ __forceinline__ void wide_head(uint64_t (&v)[NC][4], float& r, bool wide, int lanes, int dim, double eps) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(v[c][i]);
      top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
  for (int o = lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = wide && top > 0.f && top <= 3.4028235e38f ? ilogbf(top) : 0;
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(v[c][i]);
      const float x0 = scale_pow2(f.x, e), x1 = scale_pow2(f.y, e);
      ss = fmaf(x1, x1, fmaf(x0, x0, ss));
      v[c][i] = pair(x0, x1);
    }
  for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (wide) r = (float)(ldexp(1.0, e) / sqrt(ldexp((double)ss / dim, 2 * e) + eps));
}

// One head as loaded: normalised, times the weight, rotated, and stored if
// there is one.
template <typename T, int NC, bool kVec>
__device__ __forceinline__ void norm_head(const Raw<T> (&raw)[NC], const uint64_t (&w)[NC][4], int lph, int l, int D, int rot0,
                                          float inv_d, float eps, double eps64, bool tiny_eps, const float2* turn, bool there,
                                          T* y) {
  uint64_t v[NC][4], s2 = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[c][i] = raw[c].get(i);
      s2 = fma2(v[c][i], v[c][i], s2);
    }
  const float2 s = unpair(s2);
  float ss = s.x + s.y;
  for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  float r = __frcp_rn(sqrtf(fmaf(ss, inv_d, eps)));
  const bool wide = !(ss <= 3.0e38f) || (tiny_eps && ss < 1e-30f);
  if (__any_sync(0xffffffffu, wide)) wide_head<NC>(v, r, wide, lph, D, eps64);
  const uint64_t rr = pair(r, r);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int d0 = (c * lph + l) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[c][i] = mul2(mul2(v[c][i], rr), w[c][i]);
    if (d0 + 8 > rot0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = d0 + 2 * i;                    // D and rot0 are even: a pair never straddles
        if (d >= rot0 && d < D) {
          const float2 q = turn[(d - rot0) >> 1], f = unpair(v[c][i]);
          v[c][i] = pair(fmaf(f.x, q.x, -(f.y * q.y)), fmaf(f.x, q.y, f.y * q.x));
        }
      }
    }
    if (there && d0 < D) Raw<T>::store(y + c * lph * 8, v[c], kVec ? -1 : D - d0);
  }
}

// Heads h0 + slot, h0 + slot + slots, ... below h1 of token t.  NC: steps of
// 8 values a lane takes; U: heads whose loads are in flight at once.  kVec:
// 16-byte accesses.  `table`: the block's cosines and sines still have to be
// computed (by every warp of the block together).
template <typename T, int NC, int U, bool kVec>
__device__ __forceinline__ void norm_heads(const HeadNormArgs& a, const HeadNormPart& p, int64_t t, int h0, int h1,
                                           float2* cs, bool table) {
  const int lane = threadIdx.x & 31, lph = a.lanes, l = lane & (lph - 1);
  const int per_warp = 32 / lph, slots = (kHnThreads / 32) * per_warp;
  const int D = a.dim, rot0 = p.rotate ? D - a.rope : D;
  int h = h0 + (int)(threadIdx.x >> 5) * per_warp + lane / lph;
  const T* x = static_cast<const T*>(p.x) + t * p.x_tok + h * p.x_head + l * 8;
  T* y = static_cast<T*>(p.y) + t * p.y_tok + h * p.y_head + l * 8;
  const int64_t x_step = slots * p.x_head, y_step = slots * p.y_head;
  const float inv_d = 1.f / (float)D, eps = (float)a.eps;
  const bool tiny_eps = a.eps < 1e-20;
  uint64_t w[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = (c * lph + l) * 8 + 2 * i;
      w[c][i] = p.weight != nullptr && d < D ? pair(__ldg(p.weight + d), __ldg(p.weight + d + 1)) : pair(1.f, 1.f);
    }
  Raw<T> next[U][NC];
  auto fetch = [&](int at) {                             // heads at, at + slots, ...
#pragma unroll
    for (int u = 0; u < U; ++u, x += x_step) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int left = D - (c * lph + l) * 8;
        next[u][c].zero();
        if (at + u * slots < h1 && left > 0) {
          if (kVec) next[u][c].load(x + c * lph * 8);
          else next[u][c].load(x + c * lph * 8, left);
        }
      }
    }
  };
  fetch(h);
  for (int n = (h1 - h0 + slots * U - 1) / (slots * U); n > 0; --n) {      // the same count in every warp
    Raw<T> raw[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) raw[u][c] = next[u][c];
    if (n > 1) fetch(h + U * slots);
    if (table) {       // (the first pass of the block's first heads)
      table = false;
      const int64_t pos = a.positions != nullptr ? a.positions[t] : 0;
      for (int i = threadIdx.x; i < a.rope / 2; i += kHnThreads) {
        cs[i] = cos_sin((double)pos * a.theta[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u, h += slots, y += y_step) {
      if (u == 0 || __any_sync(0xffffffffu, h < h1))
        norm_head<T, NC, kVec>(raw[u], w, lph, l, D, rot0, inv_d, eps, a.eps, tiny_eps, cs, h < h1, y);
    }
  }
}

// Items first .. total - 1, item i being head i % heads of token t0 + i / heads,
// the block's slots one item each at a time.  NC: steps of 8 values a lane
// takes; U: heads whose loads are in flight at once.  kVec: 16-byte accesses.
// `table`: the cosines and sines of tokens t0 .. t0 + nt - 1 have to be computed
// (by every warp of the block together).
template <typename T, int NC, int U, bool kVec>
__device__ __forceinline__ void norm_run(const HeadNormArgs& a, const HeadNormPart& p, int64_t t0, int nt, int first, int total,
                                         float2* cs, bool table) {
  const int lane = threadIdx.x & 31, lph = a.lanes, l = lane & (lph - 1);
  const int per_warp = 32 / lph, slots = (kHnThreads / 32) * per_warp;
  const int D = a.dim, rot0 = p.rotate ? D - a.rope : D;
  const T* x = static_cast<const T*>(p.x) + t0 * p.x_tok + l * 8;
  T* y = static_cast<T*>(p.y) + t0 * p.y_tok + l * 8;
  const float inv_d = 1.f / (float)D, eps = (float)a.eps;
  const bool tiny_eps = a.eps < 1e-20;
  const int nh = p.heads;
  // this lane group's item, its token and head; those of the next fetch, too
  int item = first + (int)(threadIdx.x >> 5) * per_warp + lane / lph;
  int tok = item / nh, h = item - tok * nh;
  const int d_tok = slots / nh, d_h = slots - d_tok * nh;
  int ftok = tok, fh = h;
  uint64_t w[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = (c * lph + l) * 8 + 2 * k;
      w[c][k] = p.weight != nullptr && d < D ? pair(__ldg(p.weight + d), __ldg(p.weight + d + 1)) : pair(1.f, 1.f);
    }
  Raw<T> next[U][NC];
  auto fetch = [&](int at) {                             // items at, at + slots, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* px = x + ftok * p.x_tok + fh * p.x_head;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int left = D - (c * lph + l) * 8;
        next[u][c].zero();
        if (at + u * slots < total && left > 0) {
          if (kVec) next[u][c].load(px + c * lph * 8);
          else next[u][c].load(px + c * lph * 8, left);
        }
      }
      ftok += d_tok;
      fh += d_h;
      if (fh >= nh) { fh -= nh; ++ftok; }
    }
  };
  fetch(item);
  for (int n = (total - first + slots * U - 1) / (slots * U); n > 0; --n) {   // the same count in every warp
    Raw<T> raw[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) raw[u][c] = next[u][c];
    if (n > 1) fetch(item + U * slots);
    if (table) {
      table = false;
      const int half = a.rope / 2;
      for (int k = threadIdx.x; k < nt * half; k += kHnThreads) {
        const int dt = k / half;
        cs[k] = cos_sin((double)(a.positions != nullptr ? a.positions[t0 + dt] : 0) * a.theta[k - dt * half]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      T* py = y + tok * p.y_tok + h * p.y_head;
      // (an item beyond the last is worked on, not stored)
      const float2* turn = cs + min(tok, nt - 1) * (a.rope / 2);
      if (u == 0 || __any_sync(0xffffffffu, item < total))
        norm_head<T, NC, kVec>(raw[u], w, lph, l, D, rot0, inv_d, eps, a.eps, tiny_eps, turn, item < total, py);
      item += slots;
      tok += d_tok;
      h += d_h;
      if (h >= nh) { h -= nh; ++tok; }
    }
  }
}

// kRun: items first .. end - 1 from token t on; else heads of token t.
template <int NC, bool kRun>
__device__ __forceinline__ void norm_part(const HeadNormArgs& a, const HeadNormPart& p, int64_t t, int nt, int first, int end,
                                          float2* cs, bool table) {
  // heads in flight a warp: as many as the registers hold twice
  constexpr int U = NC == 1 ? 2 : 1, UB = NC == 4 ? 1 : 2;
  if (p.f32) {
    if (kRun && p.vec) norm_run<float, NC, U, true>(a, p, t, nt, first, end, cs, table);
    else if (kRun) norm_run<float, NC, 1, false>(a, p, t, nt, first, end, cs, table);
    else if (p.vec) norm_heads<float, NC, U, true>(a, p, t, first, end, cs, table);
    else norm_heads<float, NC, 1, false>(a, p, t, first, end, cs, table);
  } else {
    if (kRun && p.vec) norm_run<uint16_t, NC, UB, true>(a, p, t, nt, first, end, cs, table);
    else if (kRun) norm_run<uint16_t, NC, 1, false>(a, p, t, nt, first, end, cs, table);
    else if (p.vec) norm_heads<uint16_t, NC, UB, true>(a, p, t, first, end, cs, table);
    else norm_heads<uint16_t, NC, 1, false>(a, p, t, first, end, cs, table);
  }
}

// A block works on some heads of one token.  kPerSm: blocks an SM holds.
template <int NC, int kPerSm>
__global__ void __launch_bounds__(kHnThreads, kPerSm) head_norm_kernel(const __grid_constant__ HeadNormArgs a) {
  __shared__ float2 cs[kHnMaxDim / 2];
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int64_t t = blockIdx.x / a.blocks;
  const int b = blockIdx.x % a.blocks;
  const HeadNormPart &q = a.part[0], &k = a.part[1];
  const int qb = b - q.block0, kb = b - k.block0;
  const bool has_q = qb >= 0 && qb < q.blocks, has_k = kb >= 0 && kb < k.blocks;
  const bool table = (has_q && q.rotate) || (has_k && k.rotate);
  if (has_q) norm_part<NC, false>(a, q, t, 1, qb * q.block_heads, min(q.heads, (qb + 1) * q.block_heads), cs, table);
  if (has_k) norm_part<NC, false>(a, k, t, 1, kb * k.block_heads, min(k.heads, (kb + 1) * k.block_heads), cs, table && !has_q);
}

// Blocks an SM holds of the kernel below for NC steps (168 registers a thread
// with NC = 4, at most 128 else).  The wave of runs is counted with it: 4000
// tokens x 9 heads of 576 30.3 us, counted with a block too many 43.7.
constexpr int run_per_sm(int nc) { return nc > 2 ? 3 : 4; }

// A block works on a run of tokens.  The heads of all tokens, a token's queries
// before its keys, are one list in which a head costs its values' bytes; a
// block takes `share` of the list's cost.  The tokens whose sines fit are done
// at a time, their queries and then their keys.
template <int NC>
__global__ void __launch_bounds__(kHnThreads, run_per_sm(NC)) head_norm_run_kernel(const __grid_constant__ HeadNormArgs a) {
  __shared__ float2 cs[kHnMaxDim / 2];
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const HeadNormPart &q = a.part[0], &k = a.part[1];
  const int lq = q.f32 ? 1 : 0, lk = k.f32 ? 1 : 0, cq = q.heads << lq, c = cq + (k.heads << lk);
  const int64_t lo = blockIdx.x * a.share, hi = min(lo + a.share, a.n_tok * c);
  auto token = [&](int64_t v) { return v <= 0x7FFFFFFF ? (int64_t)((uint32_t)v / (uint32_t)c) : v / c; };
  // the first query and key heads of a token that lie at its cost `v` or behind
  auto q_head = [&](int v) { return min(q.heads, (v + lq) >> lq); };
  auto k_head = [&](int v) { return min(k.heads, (max(v - cq, 0) + lk) >> lk); };
  const int64_t ta = token(lo), tb = token(hi);          // the first token, and the one at which the run ends
  const int va = (int)(lo - ta * c), vb = (int)(hi - tb * c);
  for (int64_t t = ta; t < tb + (vb > 0); t += a.group) {
    if (t > ta) __syncthreads();                         // the sines of the tokens before are read no more
    const int nt = (int)min(tb + (vb > 0) - t, (int64_t)a.group);
    const bool last = tb - t < a.group;
    const int full = last ? (int)(tb - t) : nt;          // tokens that are not cut at their end
    const int q0 = t == ta ? q_head(va) : 0, q1 = full * q.heads + (last ? q_head(vb) : 0);
    const int k0 = t == ta ? k_head(va) : 0, k1 = full * k.heads + (last ? k_head(vb) : 0);
    if (q0 < q1) norm_part<NC, true>(a, q, t, nt, q0, q1, cs, q.rotate);
    if (k0 < k1) norm_part<NC, true>(a, k, t, nt, k0, k1, cs, k.rotate && !(q0 < q1 && q.rotate));
  }
}

}  // namespace

int head_norm_max_dim() { return kHnMaxDim; }

cudaError_t launch_head_norm(HeadNormArgs a, int sms, cudaStream_t st) {
  const int steps = (a.dim + 7) / 8;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes < steps) a.lanes *= 2;
  const int nc = (steps + 31) / 32;
  const int slots = (kHnThreads / 32) * (32 / a.lanes);
  // A token's heads in one block once the tokens alone give every SM 8 blocks
  // (the sines are computed once a token, the keys follow the queries); for
  // fewer tokens the heads are spread over blocks of at least one pass, the
  // keys in blocks of their own.
  const int64_t want = (8LL * sms + a.n_tok - 1) / a.n_tok;
  int64_t blocks = 0, cost = 0;
  for (HeadNormPart& p : a.part) {
    if (p.heads == 0) { p.blocks = p.block0 = 0; p.block_heads = 1; continue; }
    const int al = p.f32 ? 4 : 8;
    p.vec = a.dim % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 &&
            p.x_tok % al == 0 && p.x_head % al == 0 && p.y_tok % al == 0 && p.y_head % al == 0;
    int64_t bh = (p.heads + want - 1) / want;
    bh = (bh + slots - 1) / slots * slots;
    p.block_heads = (int)bh;
    p.blocks = (int)((p.heads + bh - 1) / bh);
    p.block0 = want == 1 ? 0 : (int)blocks;
    blocks = std::max<int64_t>(blocks, p.block0 + p.blocks);
    cost += (a.n_tok * p.heads) << (p.f32 ? 1 : 0);
  }
  a.blocks = (int)blocks;
  int64_t grid = blocks * a.n_tok;
  if (grid == 0) return cudaSuccess;
  // Beyond two waves of such blocks, tokens of few heads leave them after a
  // pass or two, before their loads ahead gain anything: one wave of blocks
  // with runs of tokens then.  (4000 tokens x 3 heads of 64, one pass: 5.2 us
  // instead of 20; 3000 x 26 of 128, 4 passes: 18 instead of 27; 1000 x 40 BF16
  // heads of 256, 10 passes: 18 instead of 23; but 2048 x 72 heads of 128, 9
  // passes: BF16 29 instead of 25, fp32 49 instead of 41; and in less than two
  // waves, 500 x 3 of 64: 4.8 instead of 4.2.)
  const int64_t wave = (int64_t)run_per_sm(nc) * sms;
  const bool many = grid > 2 * wave;
  const int passes = (a.part[0].heads + a.part[1].heads + slots - 1) / slots;
  const bool run = many && passes <= (nc == 2 && !a.part[a.part[0].heads ? 0 : 1].f32 ? 10 : 6);
  if (run) {
    a.share = (cost + wave - 1) / wave;
    grid = (cost + a.share - 1) / a.share;
    a.group = a.rope ? kHnMaxDim / a.rope : kHnMaxDim;
  }
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(kHnThreads);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  // (Short heads take six blocks an SM where there are many: 2048 tokens x 72
  // BF16 heads of 128 25 us instead of 29; few blocks do better with four, 130
  // x 27 of 96 2.6 instead of 3.0.)
  void (*kernel)(HeadNormArgs) = nc == 1 ? (many ? head_norm_kernel<1, 6> : head_norm_kernel<1, 4>)
                                 : nc == 2 ? head_norm_kernel<2, 4> : head_norm_kernel<4, 3>;
  if (run) kernel = nc == 1 ? head_norm_run_kernel<1> : nc == 2 ? head_norm_run_kernel<2> : head_norm_run_kernel<4>;
  cudaError_t e = cudaLaunchKernelEx(&lc, kernel, a);
  note_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace csa
