// train_rows.cu -- tokens to expert order and back in a training step, and the
// gradients of both. Pair i = t*K + k; inv[i] is its row in expert order, -1
// for a dropped pair (it takes no part). Sums run k ascending in fp32 and are
// rounded once.
//
//   dispatch              xs[inv[t,k], :] = x[t, :]
//                         (x bf16 or fp32: copied; x an e4m3 checkpoint:
//                         bf16(code * scale), scales per 1 x 128 block)
//   its gradient          dx[t, :] = sum_k dxs[inv[t,k], :] + dl[t,k] * Wr[idx[t,k], :]
//                         (the second term when the router's logits pass a gradient back)
//   weighted combine      out[t, :] = sum_k w[t,k] * y[inv[t,k], :]
//   its gradient          dy[inv[t,k], :] = w[t,k] * dout[t, :],  dw[t,k] = <dout[t, :], y[inv[t,k], :]>
//
// All are bound by HBM. Each kernel touches a token's row once and the token's
// K expert rows once: a thread owns one 16-byte piece of a token's row and
// walks the K rows (dispatch, its gradient, the combine), or a warp owns one
// pair (the combine's gradient, where each pair needs a dot product over the
// whole row and the token's row is shared by neighbouring warps).
//
// Measured at 4096 tokens, K = 8, H = 4096, bf16, of a copy's 6.56 TB/s:
// dispatch 49 us (95%), combine 44 us (104%: part of the rows is still in L2),
// its gradient 89 us (98%), dispatch gradient 44 us (104%). With the router's
// term that takes 68 us from a cold L2 (55 us without it): K fp32 router rows
// per token, 537 MB, come from L1 and L2. Expert rows are read past L1 (they
// are read once), which leaves it to the router rows of the busiest experts:
// 105 us before. A CTA that keeps 64 columns of the whole router weight in
// shared memory and passes the tokens by it took 126 to 174 us; expert rows
// requested before or together with the router rows 71 to 82 us (registers);
// paired fp32 instructions in both sums changed nothing.
#include "rows.cuh"
#include "train.h"

namespace moe {

namespace {

// Expert rows in flight per thread. Few, so that five blocks fit an SM: with eight (64 registers, four blocks) the
// combine took 53 us.
constexpr int kSlots = 4;
// 16-byte pieces of a row that the router's form takes of every token before it goes on to the next ones: the router
// rows' columns in use stay in L1.
constexpr unsigned kSlice = 64;

// The sums of gather_sum_kernel.
enum Sum { kPlain, kWeighted, kRouter };

// One thread per 16-byte piece of the output row.
template <bool kCkpt>
__global__ void __launch_bounds__(256) dispatch_kernel(const void* __restrict__ x, const float* __restrict__ scales,
                                                        const int32_t* __restrict__ inv, int T, int K, unsigned V,
                                                        uint4* __restrict__ xs, int* status) {
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  const unsigned t = i / V, v = i - t * V;
  if (t >= (unsigned)T) return;
  uint4 piece;
  if (kCkpt) {
    const uint2 q = __ldg(static_cast<const uint2*>(x) + (size_t)t * V + v);
    float f[8];
    e4m3x8(q, __ldg(scales + (size_t)t * (V / 16) + v / 16), f);
    piece = RowBf16::pack(f);
  } else {
    piece = __ldg(static_cast<const uint4*>(x) + (size_t)t * V + v);
  }
  const int P = T * K;
  for (int k = 0; k < K; ++k) {
    const int p = pair_row(inv, (long long)t * K + k, P, status);
    if (p >= 0) xs[(size_t)p * V + v] = piece;
  }
}

// A row piece that is read once: not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint2 load_once(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// acc += the sum over k of a token's rows, one 16-byte piece of them (kHalves: two 8-byte pieces, v and v + 16): f or,
// with weights, w f.
template <class R, bool kWeights, bool kHalves>
__device__ __forceinline__ void sum_rows(const uint4* __restrict__ rows, const float* __restrict__ w,
                                         const int32_t* __restrict__ inv, size_t t, int K, int P, unsigned V,
                                         unsigned v, float (&acc)[R::kN], int* status) {
  for (int k0 = 0; k0 < K; k0 += kSlots) {
    int p[kSlots];
    uint4 a[kSlots];
    float wk[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      p[u] = k0 + u < K ? pair_row(inv, (long long)t * K + k0 + u, P, status) : -1;
      wk[u] = kWeights && k0 + u < K ? __ldg(w + t * K + k0 + u) : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
      if (p[u] >= 0) {
        if (kHalves) {
          const uint2* r = reinterpret_cast<const uint2*>(rows + (size_t)p[u] * V) + v;
          const uint2 lo = load_once(r), hi = load_once(r + 16);
          a[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          a[u] = load_once(rows + (size_t)p[u] * V + v);
        }
      }
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      if (p[u] < 0) continue;
      float f[R::kN];
      R::unpack(a[u], f);
#pragma unroll
      for (int j = 0; j < R::kN; ++j) acc[j] = kWeights ? fmaf(wk[u], f[j], acc[j]) : acc[j] + f[j];
    }
  }
}

// acc += d * r for one piece's columns of a router row.
template <int kN>
__device__ __forceinline__ void add_router(float (&acc)[kN], float d, const float4 (&r)[kN / 4]) {
#pragma unroll
  for (int j = 0; j < kN / 4; ++j) {
    acc[4 * j] = fmaf(d, r[j].x, acc[4 * j]);
    acc[4 * j + 1] = fmaf(d, r[j].y, acc[4 * j + 1]);
    acc[4 * j + 2] = fmaf(d, r[j].z, acc[4 * j + 2]);
    acc[4 * j + 3] = fmaf(d, r[j].w, acc[4 * j + 3]);
  }
}

// kWeighted: out = sum_k w y (the combine). Otherwise the dispatch's gradient, kRouter: with the router's term.
//
// Router rows are fp32: where expert rows are bf16, a thread takes columns 4l..4l+3 of both halves of a 128-column
// block in place of eight neighbouring ones, so that a warp's loads of router rows are contiguous too (77.7 -> 73.3 us
// for 4096 tokens of 8 x 4096; slices and one router row at a time, which lets six blocks fit an SM: 67.7 us). Slices
// narrower than 512 columns were not measured.
template <class R, Sum kSum>
__global__ void __launch_bounds__(256, kSum == kRouter && R::kN == 8 ? 6 : 5)
    gather_sum_kernel(const uint4* __restrict__ rows, const float* __restrict__ w, const int32_t* __restrict__ inv,
                      const float* __restrict__ dl, const int32_t* __restrict__ idx, const float* __restrict__ wr,
                      int T, int K, int E, unsigned V, uint4* __restrict__ out, int* status) {
  constexpr bool kHalves = kSum == kRouter && R::kN == 8;
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  unsigned t, v;
  if (kSum == kRouter) {
    const unsigned slice = i / (kSlice * T), v0 = slice * kSlice;
    if (v0 >= V) return;
    const unsigned width = min(kSlice, V - v0), j = i - v0 * T;
    t = j / width;
    v = v0 + (j - t * width);
    if (kHalves) v = v / 16 * 32 + v % 16;  // 8-byte pieces
  } else {
    t = i / V;
    v = i - t * V;
  }
  if (t >= (unsigned)T) return;
  float acc[R::kN] = {};
  if (kSum == kRouter) {
    const size_t H = (size_t)V * R::kN;
    constexpr int kSlotsR = kHalves ? 1 : 2;  // router rows in flight
    for (int k0 = 0; k0 < K; k0 += kSlotsR) {
      int e[kSlotsR];
      float d[kSlotsR];
#pragma unroll
      for (int u = 0; u < kSlotsR; ++u) {
        const bool in = k0 + u < K;
        e[u] = in ? __ldg(idx + (size_t)t * K + k0 + u) : 0;
        d[u] = in ? __ldg(dl + (size_t)t * K + k0 + u) : 0.0f;
      }
      float4 q[kSlotsR][R::kN / 4];
#pragma unroll
      for (int u = 0; u < kSlotsR; ++u) {
        const bool good = e[u] >= 0 && e[u] < E;
        if (!good) flag_status(status, MOE_DEV_BAD_EXPERT);
        if (!good || k0 + u >= K) e[u] = -1;
#pragma unroll
        for (int j = 0; j < R::kN / 4; ++j)
          if (e[u] >= 0) q[u][j] = __ldg(reinterpret_cast<const float4*>(wr + e[u] * H) + v + 16 * j);
      }
#pragma unroll
      for (int u = 0; u < kSlotsR; ++u)
        if (e[u] >= 0) add_router(acc, d[u], q[u]);
    }
  }
  sum_rows<R, kSum == kWeighted, kHalves>(rows, w, inv, t, K, T * K, V, v, acc, status);
  const uint4 sum = R::pack(acc);
  uint4* o = out + (size_t)t * V;
  if (kHalves) {
    uint2* h = reinterpret_cast<uint2*>(o) + v;
    h[0] = make_uint2(sum.x, sum.y);
    h[16] = make_uint2(sum.z, sum.w);
  } else {
    o[v] = sum;
  }
}

// One warp per pair.
template <class R>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ inv, int T, int K, int V,
                                                           uint4* __restrict__ dy, float* __restrict__ dw,
                                                           int* status) {
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= (long long)T * K) return;
  const int p = pair_row(inv, i, T * K, status);
  if (p < 0) {
    if (lane == 0) dw[i] = 0.0f;
    return;
  }
  const int t = (int)(i / K);
  const float wk = __ldg(w + i);
  const uint4* d = dout + (size_t)t * V;
  const uint4* r = y + (size_t)p * V;
  uint4* o = dy + (size_t)p * V;
  float dot = 0.0f;
  for (int v0 = lane; v0 < V; v0 += 32 * 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v0 + 32 * u < V) {
        a[u] = __ldg(d + v0 + 32 * u);
        b[u] = __ldg(r + v0 + 32 * u);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v0 + 32 * u < V) {
        float fa[R::kN], fb[R::kN];
        R::unpack(a[u], fa);
        R::unpack(b[u], fb);
#pragma unroll
        for (int j = 0; j < R::kN; ++j) {
          dot = fmaf(fa[j], fb[j], dot);
          fa[j] *= wk;
        }
        o[v0 + 32 * u] = R::pack(fa);
      }
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
  if (lane == 0) dw[i] = dot;
}

unsigned blocks_for(long long n) { return (unsigned)((n + 255) / 256); }

}  // namespace

cudaError_t launch_dispatch(const void* x, const float* scales, int dtype, const int32_t* inv, int T, int K, int H,
                            void* xs, int* status, cudaStream_t s) {
  uint4* o = static_cast<uint4*>(xs);
  const unsigned V = (unsigned)(dtype == MOE_T_F32 ? H / 4 : H / 8);
  const unsigned blocks = blocks_for((long long)T * V);
  if (dtype == MOE_T_E4M3_B128)
    dispatch_kernel<true><<<blocks, 256, 0, s>>>(x, scales, inv, T, K, V, o, status);
  else
    dispatch_kernel<false><<<blocks, 256, 0, s>>>(x, scales, inv, T, K, V, o, status);
  return cudaGetLastError();
}

cudaError_t launch_dispatch_bwd(const void* rows, int dtype, const int32_t* inv, const float* dl, const int32_t* idx,
                                const float* wr, int T, int K, int E, int H, void* dx, int* status, cudaStream_t s) {
  const uint4* r = static_cast<const uint4*>(rows);
  uint4* o = static_cast<uint4*>(dx);
  const bool f32 = dtype == MOE_T_F32;
  const unsigned V = (unsigned)(f32 ? H / 4 : H / 8);
  const unsigned blocks = blocks_for((long long)T * V);
  auto sum = dl ? (f32 ? gather_sum_kernel<RowF32, kRouter> : gather_sum_kernel<RowBf16, kRouter>)
                : (f32 ? gather_sum_kernel<RowF32, kPlain> : gather_sum_kernel<RowBf16, kPlain>);
  sum<<<blocks, 256, 0, s>>>(r, nullptr, inv, dl, idx, wr, T, K, E, V, o, status);
  return cudaGetLastError();
}

cudaError_t launch_combine_weighted(const void* y, int dtype, const float* w, const int32_t* inv, int T, int K, int H,
                                    void* out, int* status, cudaStream_t s) {
  const uint4* r = static_cast<const uint4*>(y);
  uint4* o = static_cast<uint4*>(out);
  const unsigned V = (unsigned)(dtype == MOE_T_F32 ? H / 4 : H / 8);
  const unsigned blocks = blocks_for((long long)T * V);
  auto sum = dtype == MOE_T_F32 ? gather_sum_kernel<RowF32, kWeighted> : gather_sum_kernel<RowBf16, kWeighted>;
  sum<<<blocks, 256, 0, s>>>(r, w, inv, nullptr, nullptr, nullptr, T, K, 0, V, o, status);
  return cudaGetLastError();
}

cudaError_t launch_combine_weighted_bwd(const void* dout, const void* y, int dtype, const float* w,
                                        const int32_t* inv, int T, int K, int H, void* dy, float* dw, int* status,
                                        cudaStream_t s) {
  const int V = dtype == MOE_T_F32 ? H / 4 : H / 8;
  const unsigned blocks = (unsigned)(((long long)T * K + 7) / 8);
  const uint4 *d = static_cast<const uint4*>(dout), *r = static_cast<const uint4*>(y);
  uint4* o = static_cast<uint4*>(dy);
  if (dtype == MOE_T_F32)
    combine_bwd_kernel<RowF32><<<blocks, 256, 0, s>>>(d, r, w, inv, T, K, V, o, dw, status);
  else
    combine_bwd_kernel<RowBf16><<<blocks, 256, 0, s>>>(d, r, w, inv, T, K, V, o, dw, status);
  return cudaGetLastError();
}

}  // namespace moe
