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
// Bound by HBM: 10 bytes per (row, column of I) each way. A half-warp owns a
// 128-column block: 16 lanes x 8 values, so that every access is 8 or 16 bytes
// and a block's amax needs four shuffles.
#include "internal.h"
#include "rows.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// amax over the 16 lanes that share a 128-column block; NaN values do not count.
__device__ __forceinline__ float block_amax(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(f[j] / s, __NV_SATFINITE, __NV_E4M3) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

// One half-warp per (row, 128-column block of I); rows are pairs in token
// order (row = inv[i]) or, without inv, the rows themselves.
__global__ void __launch_bounds__(256) swiglu_ckpt_kernel(const uint4* __restrict__ gu,
                                                           const int32_t* __restrict__ inv, int rows, int blocks,
                                                           uint4* __restrict__ h, uint2* __restrict__ q,
                                                           float* __restrict__ s, int* status) {
  const int l = threadIdx.x & 15;
  const long long unit = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  const long long i = unit / blocks;
  const int b = (int)(unit - i * blocks);
  int r = -1;
  if (i < rows) r = inv ? pair_row(inv, i, rows, status) : (int)i;
  const size_t gv = (size_t)(r < 0 ? 0 : r) * blocks * 32 + b * 16 + l, uv = gv + blocks * 16;  // 16-byte pieces
  uint4 ga = make_uint4(0, 0, 0, 0), ua = ga;
  if (r >= 0) {
    ga = __ldg(gu + gv);
    ua = __ldg(gu + uv);
  }
  float g[8], u[8], o[8];
  RowBf16::unpack(ga, g);
  RowBf16::unpack(ua, u);
  const float mg = block_amax(g), mu = block_amax(u);  // all lanes of the warp take part
  if (r < 0) return;
  const float sg = mg == 0.0f ? 1.0f : mg / 448.0f, su = mu == 0.0f ? 1.0f : mu / 448.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * u[j];
  h[(size_t)r * blocks * 16 + b * 16 + l] = RowBf16::pack(o);
  q[gv] = encode8(g, sg);
  q[uv] = encode8(u, su);
  if (l == 0) {
    s[(size_t)r * blocks * 2 + b] = sg;
    s[(size_t)r * blocks * 2 + blocks + b] = su;
  }
}

// One warp per row; each half-warp takes every second 128-column block.
template <bool kWeighted>
__global__ void __launch_bounds__(256) swiglu_ckpt_bwd_kernel(const uint2* __restrict__ q,
                                                               const float* __restrict__ s,
                                                               const uint4* __restrict__ dh,
                                                               const float* __restrict__ w,
                                                               const int32_t* __restrict__ inv, int rows, int blocks,
                                                               uint4* __restrict__ dgu, uint4* __restrict__ hw,
                                                               float* __restrict__ dw, int* status) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= rows) return;
  const int r = inv ? pair_row(inv, i, rows, status) : (int)i;
  if (r < 0) {
    if (kWeighted && lane == 0) dw[i] = 0.0f;
    return;
  }
  const float wk = kWeighted ? __ldg(w + i) : 1.0f;
  float dot = 0.0f;
  for (int b = lane >> 4; b < blocks; b += 2) {
    const size_t hv = (size_t)r * blocks * 16 + b * 16 + l, gv = (size_t)r * blocks * 32 + b * 16 + l,
                 uv = gv + blocks * 16, sv = (size_t)r * blocks * 2 + b;
    const uint2 qg = __ldg(q + gv), qu = __ldg(q + uv);
    const uint4 dv = __ldg(dh + hv);
    float g[8], u[8], d[8], o[8];
    e4m3x8(qg, __ldg(s + sv), g);
    e4m3x8(qu, __ldg(s + sv + blocks), u);
    RowBf16::unpack(dv, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sig = sigmoid(g[j]), silu = g[j] * sig, hj = silu * u[j];
      if (kWeighted) dot = fmaf(d[j], hj, dot);
      o[j] = wk * hj;
      const float wd = wk * d[j];
      const float dgj = wd * u[j] * sig * (1.0f + g[j] * (1.0f - sig));
      u[j] = wd * silu;
      g[j] = dgj;
    }
    dgu[gv] = RowBf16::pack(g);
    dgu[uv] = RowBf16::pack(u);
    if (kWeighted && hw) hw[hv] = RowBf16::pack(o);
  }
  if (kWeighted) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) dw[i] = dot;
  }
}

}  // namespace

cudaError_t launch_swiglu_ckpt(const void* gu, const int32_t* inv, int rows, int I, void* h, uint8_t* q, float* s,
                               int* status, cudaStream_t st) {
  const int blocks = I / 128;
  const long long units = (long long)rows * blocks;
  swiglu_ckpt_kernel<<<(unsigned)((units + 15) / 16), 256, 0, st>>>(static_cast<const uint4*>(gu), inv, rows, blocks,
                                                                     static_cast<uint4*>(h),
                                                                     reinterpret_cast<uint2*>(q), s, status);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_ckpt_bwd(const uint8_t* q, const float* s, const void* dh, const float* w,
                                   const int32_t* inv, int rows, int I, void* dgu, void* hw, float* dw, int* status,
                                   cudaStream_t st) {
  const int blocks = I / 128;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  const uint2* qv = reinterpret_cast<const uint2*>(q);
  const uint4* dv = static_cast<const uint4*>(dh);
  uint4 *o = static_cast<uint4*>(dgu), *hv = static_cast<uint4*>(hw);
  if (w)
    swiglu_ckpt_bwd_kernel<true><<<grid, 256, 0, st>>>(qv, s, dv, w, inv, rows, blocks, o, hv, dw, status);
  else
    swiglu_ckpt_bwd_kernel<false><<<grid, 256, 0, st>>>(qv, s, dv, w, inv, rows, blocks, o, hv, dw, status);
  return cudaGetLastError();
}

}  // namespace moe
