// swiglu_ckpt.cu -- the experts' activation with 8-bit checkpoints.
//
// Forward, per row [g | u] of 2I bf16 values:
//   h = bf16(silu(g) * u), silu(g) = g / (1 + exp(-g)), from g and u themselves
//   q, s = e4m3 codes and fp32 scales of [g | u] per 128 columns, by the rule
//          of the block quantiser (s = amax / 448, 1 for an all-zero block;
//          q = e4m3(v / s), nearest even): 1 byte per value is kept for the
//          backward pass in place of 2.
// Backward, from the checkpoint alone (g, u = code * scale) and dh:
//   sig = 1 / (1 + exp(-g)), h = g sig u
//   dw  = <dh, h> over the row                        (weighted)
//   hw  = bf16(w h)                                   (weighted: the down product's input for its weight gradient)
//   dg  = w dh u sig (1 + g (1 - sig)),  du = w dh g sig, one rounding to bf16
// with w the pair's routing weight (1 without weights). With the weight here,
// the gradient that arrives is the unweighted dout W_dn of each pair, and the
// down product's output need not be kept to differentiate the weight.
//
// Bound by HBM: 8 bytes and 10 bytes per (row, column of I). Measured at 32768
// rows, I = 2048, of a copy's 6.56 TB/s: forward 91.7 us (90%), gradient with
// weights 115 us (89%) on warm inputs; on new ones 97 and 121 us a call (84 and
// 85%). What stood in the way was arithmetic: with IEEE divisions (one per
// code, one per sigmoid) and 8 lanes' worth of shuffles the forward took 166
// us. Codes now take a reciprocal per block and three fused multiply-adds per
// value, to the same bits (below). The sigmoid takes the fast exponential and
// division, whose relative error is at most (2 + 1.2 |g|) 2^-23 and 2^-22: far
// below the bf16 rounding that follows in h, dgu and hw. dw is not rounded to
// bf16, and keeps fp32's accuracy all the same: of the sum of its terms'
// magnitudes over 2048 columns at most 2.2e-8 off (expf and torch's fp32 sum:
// 2.1e-8), with every g near -20 1.5e-7 (1.0e-7), near -80 6.8e-7 (3.5e-7);
// expf in its place took the gradient from 117 to 123 us. A block's amax is
// taken in bf16, two values at a time, over 8 lanes of 16 values (16 lanes of 8
// values: 109 us). The register bounds are those measured fastest: forward 48
// (58 unbounded: 101 us), gradient 64 (74 unbounded: 121 us, where the bounded
// one took 115).
#include "rows.cuh"
#include "train.h"

namespace moe {

namespace {

// Where exp(-g) passes 2^126 the division gives 0 for a true value below 2^-126.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

__device__ __forceinline__ __nv_bfloat162 amax8(const uint4& v) {
  return __hmax2(__hmax2(__habs2(as_bf162(v.x)), __habs2(as_bf162(v.y))),
                 __hmax2(__habs2(as_bf162(v.z)), __habs2(as_bf162(v.w))));
}

// The largest magnitudes of the lane's g (x) and u (y), then over the 8 lanes that share a 128-column block: whole
// in bf16, two at a time. NaN values do not count.
__device__ __forceinline__ float2 block_amax(const uint4 (&g)[2], const uint4 (&u)[2]) {
  const __nv_bfloat162 mg = __hmax2(amax8(g[0]), amax8(g[1])), mu = __hmax2(amax8(u[0]), amax8(u[1]));
  __nv_bfloat162 m = __hmax2(__lows2bfloat162(mg, mu), __highs2bfloat162(mg, mu));
  m = __hmax2(m, __floats2bfloat162_rn(0.0f, 0.0f));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return __bfloat1622float2(m);
}

// v / s rounded to nearest, as IEEE division rounds it, for a bf16 v with |v| <= amax, s = RN(amax / 448) and r the
// fast reciprocal of s: one correction of v * r by its exact remainder, the step of Newton's method for the quotient
// that a fused multiply-add allows (Markstein's).
__device__ __forceinline__ float quotient(float v, float s, float r) {
  const float y = v * r;
  return fmaf(fmaf(-s, y, v), r, y);
}

// The scale of a block with this amax and a factor r for its codes (0: divide). For 2^-50 <= amax <= 2^100 the scale
// and every code below are those of IEEE division (compared over all pairs of bf16 amax and v); other blocks divide.
__device__ __forceinline__ float block_scale(float amax, float* r) {
  if (amax >= 0x1p-50f && amax <= 0x1p100f) {
    const float s = quotient(amax, 448.0f, 1.0f / 448.0f);
    *r = __fdividef(1.0f, s);
    return s;
  }
  *r = 0.0f;
  return amax == 0.0f ? 1.0f : amax / 448.0f;
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float r) {
  float y[8];
  if (r != 0.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = quotient(f[j], s, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = f[j] / s;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j], y[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Eight lanes per (row, 128-column block of I), 2 x 8 values of g and u each; rows are pairs in token order
// (row = inv[i]) or, without inv, the rows themselves.
__global__ void __launch_bounds__(256, 5) swiglu_ckpt_kernel(const uint4* __restrict__ gu,
                                                           const int32_t* __restrict__ inv, int rows, int blocks,
                                                           uint4* __restrict__ h, uint2* __restrict__ q,
                                                           float* __restrict__ s, int* status) {
  const int l = threadIdx.x & 7;
  const unsigned unit = blockIdx.x * 32u + (threadIdx.x >> 3);
  const unsigned i = unit / (unsigned)blocks;
  const int b = (int)(unit - i * blocks);
  int r = -1;
  if (i < (unsigned)rows) r = inv ? pair_row(inv, i, rows, status) : (int)i;
  const size_t hv = (size_t)(r < 0 ? 0 : r) * blocks * 16 + b * 16 + l;  // 16-byte pieces of h
  const size_t gv = (size_t)(r < 0 ? 0 : r) * blocks * 32 + b * 16 + l, uv = gv + blocks * 16;  // and of gu
  uint4 ga[2] = {}, ua[2] = {};
  if (r >= 0) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      ga[n] = __ldg(gu + gv + 8 * n);
      ua[n] = __ldg(gu + uv + 8 * n);
    }
  }
  const float2 amax = block_amax(ga, ua);  // all lanes of the warp take part
  if (r < 0) return;
  float rg, ru;
  const float sg = block_scale(amax.x, &rg), su = block_scale(amax.y, &ru);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float g[8], u[8], o[8];
    RowBf16::unpack(ga[n], g);
    RowBf16::unpack(ua[n], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * u[j];
    h[hv + 8 * n] = RowBf16::pack(o);
    q[gv + 8 * n] = encode8(g, sg, rg);
    q[uv + 8 * n] = encode8(u, su, ru);
  }
  if (l == 0) {
    s[(size_t)r * blocks * 2 + b] = sg;
    s[(size_t)r * blocks * 2 + blocks + b] = su;
  }
}

constexpr int kMaxBlocks = 64;  // of a row: I <= 8192

// kWarps warps per row; each half-warp takes every (2 kWarps)-th 128-column
// block, two blocks' loads in flight. The weight's gradient is summed per block
// and then over the blocks, in an order that does not depend on kWarps: a
// pair's bits are the same among any number of rows.
template <bool kWeighted, int kWarps>
__global__ void __launch_bounds__(256, 4) swiglu_ckpt_bwd_kernel(const uint2* __restrict__ q,
                                                               const float* __restrict__ s,
                                                               const uint4* __restrict__ dh,
                                                               const float* __restrict__ w,
                                                               const int32_t* __restrict__ inv, int rows, int blocks,
                                                               uint4* __restrict__ dgu, uint4* __restrict__ hw,
                                                               float* __restrict__ dw, int* status) {
  constexpr int kRows = 8 / kWarps;  // rows per CTA
  __shared__ float s_dot[kRows][kMaxBlocks];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15;
  const long long i = (long long)blockIdx.x * kRows + warp / kWarps;
  const bool in = i < rows;
  const int r = !in ? -1 : inv ? pair_row(inv, i, rows, status) : (int)i;
  if (r >= 0) {
    const float wk = kWeighted ? __ldg(w + i) : 1.0f;
    constexpr int kStep = 2 * kWarps;
    for (int b0 = (warp % kWarps) * 2 + (lane >> 4); b0 < blocks; b0 += 2 * kStep) {
      uint2 qg[2], qu[2];
      uint4 dv[2];
      float sg[2], su[2], dot[2] = {};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int b = b0 + n * kStep;
        if (b >= blocks) break;
        const size_t gv = (size_t)r * blocks * 32 + b * 16 + l, sv = (size_t)r * blocks * 2 + b;
        qg[n] = __ldg(q + gv);
        qu[n] = __ldg(q + gv + blocks * 16);
        dv[n] = __ldg(dh + (size_t)r * blocks * 16 + b * 16 + l);
        sg[n] = __ldg(s + sv);
        su[n] = __ldg(s + sv + blocks);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int b = b0 + n * kStep;
        if (b >= blocks) break;
        const size_t hv = (size_t)r * blocks * 16 + b * 16 + l, gv = (size_t)r * blocks * 32 + b * 16 + l;
        float g[8], u[8], d[8], o[8];
        e4m3x8(qg[n], sg[n], g);
        e4m3x8(qu[n], su[n], u);
        RowBf16::unpack(dv[n], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sig = sigmoid(g[j]), silu = g[j] * sig, hj = silu * u[j];
          if (kWeighted) dot[n] = fmaf(d[j], hj, dot[n]);
          o[j] = wk * hj;
          const float wd = wk * d[j];
          const float dgj = wd * u[j] * sig * (1.0f + g[j] * (1.0f - sig));
          u[j] = wd * silu;
          g[j] = dgj;
        }
        dgu[gv] = RowBf16::pack(g);
        dgu[gv + blocks * 16] = RowBf16::pack(u);
        if (kWeighted && hw) hw[hv] = RowBf16::pack(o);
      }
      if (kWeighted) {  // lanes 0-7 of the half-warp take the first block's sum, 8-15 the second's
        const unsigned half = 0xffffu << (lane & 16);
        const bool second = l >= 8;
        float sum = (second ? dot[1] : dot[0]) + __shfl_xor_sync(half, second ? dot[0] : dot[1], 8);
#pragma unroll
        for (int x = 4; x >= 1; x >>= 1) sum += __shfl_xor_sync(half, sum, x);
        const int b = b0 + (second ? kStep : 0);
        if ((l & 7) == 0 && b < blocks) s_dot[warp / kWarps][b] = sum;
      }
    }
  }
  if (kWeighted) {
    if (kWarps > 1) __syncthreads();
    else __syncwarp();
    if (!in || warp % kWarps) return;
    float sum = 0.0f;
    if (r >= 0)
      for (int b = lane; b < blocks; b += 32) sum += s_dot[warp / kWarps][b];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) dw[i] = sum;
  }
}

}  // namespace

cudaError_t launch_swiglu_ckpt(const void* gu, const int32_t* inv, int rows, int I, void* h, uint8_t* q, float* s,
                               int* status, cudaStream_t st) {
  const int blocks = I / 128;
  const long long units = (long long)rows * blocks;
  swiglu_ckpt_kernel<<<(unsigned)((units + 31) / 32), 256, 0, st>>>(static_cast<const uint4*>(gu), inv, rows, blocks,
                                                                     static_cast<uint4*>(h),
                                                                     reinterpret_cast<uint2*>(q), s, status);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_ckpt_bwd(const uint8_t* q, const float* s, const void* dh, const float* w,
                                   const int32_t* inv, int rows, int I, void* dgu, void* hw, float* dw, int* status,
                                   cudaStream_t st) {
  const int blocks = I / 128;
  const uint2* qv = reinterpret_cast<const uint2*>(q);
  const uint4* dv = static_cast<const uint4*>(dh);
  uint4 *o = static_cast<uint4*>(dgu), *hv = static_cast<uint4*>(hw);
  // Warps per row: as many as have a block for each half-warp, while the rows alone are too few to fill the GPU.
  int warps = 1;
  while (warps < 8 && 4 * warps <= blocks && rows * (long long)warps < 8192) warps *= 2;
  const unsigned grid = (unsigned)(((long long)rows * warps + 7) / 8);
  auto pick = [&](auto* one, auto* two, auto* four, auto* eight) {
    (warps == 1 ? one : warps == 2 ? two : warps == 4 ? four : eight)<<<grid, 256, 0, st>>>(
        qv, s, dv, w, inv, rows, blocks, o, hv, dw, status);
  };
  if (w)
    pick(swiglu_ckpt_bwd_kernel<true, 1>, swiglu_ckpt_bwd_kernel<true, 2>, swiglu_ckpt_bwd_kernel<true, 4>,
         swiglu_ckpt_bwd_kernel<true, 8>);
  else
    pick(swiglu_ckpt_bwd_kernel<false, 1>, swiglu_ckpt_bwd_kernel<false, 2>, swiglu_ckpt_bwd_kernel<false, 4>,
         swiglu_ckpt_bwd_kernel<false, 8>);
  return cudaGetLastError();
}

}  // namespace moe
