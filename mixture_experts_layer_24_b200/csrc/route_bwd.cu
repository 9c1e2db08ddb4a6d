// route_bwd.cu -- gradient of the router. With w = softmax of a token's K
// selected logits and dw its gradient,
//   dl[t,k]   = w[t,k] * (dw[t,k] - sum_j w[t,j] dw[t,j])
//   dWr[e, :] = sum over the pairs (t,k) of expert e of dl[t,k] * x[t, :]
//   dbias[e]  = sum over the same pairs of dl[t,k]
// (logits outside the top k get no gradient). Sums are fp32.
//
// The pairs are already sorted by expert, so dWr is a segmented sum of scaled
// rows: the sorted list is cut every `chunk` pairs, a CTA takes one piece and
// 2048 columns, and adds up each expert's run inside it. A run that is its
// expert's whole list is written out at once; the first and last run of a
// piece may be parts, which go to the workspace and are added in order by a
// second kernel (it also writes the zero rows of experts without pairs). The
// order of every sum depends on the routing alone, so results repeat exactly.
#include <type_traits>

#include "internal.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kChunkMax = 64;
constexpr int kCols = 2048;  // columns per CTA: 256 threads x 8

// dl of every pair, in token order: one thread per pair.
__global__ void __launch_bounds__(256) route_dlogit_kernel(const float* __restrict__ w, const float* __restrict__ dw,
                                                            int T, int K, float* __restrict__ dl) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)T * K) return;
  const long long t = i / K;
  float dot = 0.0f;
  for (int k = 0; k < K; ++k) dot = fmaf(__ldg(w + t * K + k), __ldg(dw + t * K + k), dot);
  dl[i] = __ldg(w + i) * (__ldg(dw + i) - dot);
}

__device__ __forceinline__ int valid_pairs(const int32_t* __restrict__ offsets, int E, int P, int* status) {
  const int n = __ldg(offsets + E);
  if (n < 0 || n > P) {
    flag_status(status, MOE_DEV_BAD_INDEX);
    return 0;
  }
  return n;
}

// The expert whose rows hold sorted pair p: the last e with offsets[e] <= p.
__device__ __forceinline__ int expert_of(const int32_t* __restrict__ offsets, int E, int p) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) <= p) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kCkpt: x is an e4m3 checkpoint (codes, one scale per 128 columns).
template <bool kCkpt>
__global__ void __launch_bounds__(256) route_wgrad_kernel(const void* __restrict__ x,
                                                           const float* __restrict__ scales,
                                                           const float* __restrict__ dl,
                                                           const int32_t* __restrict__ offsets,
                                                           const int32_t* __restrict__ perm_src,
                                                           const int32_t* __restrict__ perm_k, int T, int K, int E,
                                                           int H, int chunk, float* __restrict__ dwr,
                                                           float* __restrict__ dbias, float* __restrict__ part,
                                                           float* __restrict__ part_b, int* status) {
  using Piece = typename std::conditional<kCkpt, uint2, uint4>::type;  // eight columns
  __shared__ int s_t[kChunkMax];
  __shared__ float s_d[kChunkMax];
  const int n = valid_pairs(offsets, E, T * K, status);
  const int p0 = blockIdx.x * chunk, p1 = min(n, p0 + chunk);
  if (p0 >= p1) return;
  for (int j = threadIdx.x; j < p1 - p0; j += 256) {
    int t = __ldg(perm_src + p0 + j);
    const int k = __ldg(perm_k + p0 + j);
    float d = 0.0f;
    if (t < 0 || t >= T || k < 0 || k >= K) {
      flag_status(status, MOE_DEV_BAD_INDEX);
      t = -1;
    } else {
      d = __ldg(dl + (size_t)t * K + k);
    }
    s_t[j] = t;
    s_d[j] = d;
  }
  __syncthreads();
  const int V = H / 8;
  const int v = blockIdx.y * 256 + threadIdx.x;
  const bool live = v < V;
  int e = expert_of(offsets, E, p0);
  for (int p = p0; p < p1; ++e) {
    const int first = __ldg(offsets + e), end = __ldg(offsets + e + 1);
    const int stop = min(p1, end);
    float acc[8], bias = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    if (stop <= p) {
      if (e >= E - 1) break;  // offsets that do not rise: nothing more to do
      continue;
    }
    for (; p < stop; p += 8) {
      Piece a[8];
      float sc[8];
      const int m = min(8, stop - p);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        a[u] = Piece{};
        sc[u] = 0.0f;
        const int t = u < m ? s_t[p - p0 + u] : -1;
        if (live && t >= 0) {
          a[u] = __ldg(static_cast<const Piece*>(x) + (size_t)t * V + v);
          if constexpr (kCkpt) sc[u] = __ldg(scales + (size_t)t * (V / 16) + v / 16);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u < m) {
          float f[8];
          if constexpr (kCkpt) e4m3x8(a[u], sc[u], f);
          else RowBf16::unpack(a[u], f);
          const float d = s_d[p - p0 + u];
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = fmaf(d, f[j], acc[j]);
          bias += d;
        }
      }
    }
    p = stop;
    // whole list of e: final; otherwise a part (0: runs from the piece's first pair, 1: up to its last)
    const bool whole = first >= p0 && end <= p1;
    const int half = first < p0 ? 0 : 1;
    const size_t slot = (size_t)blockIdx.x * 2 + half;
    if (live) {
      float4* o = reinterpret_cast<float4*>((whole ? dwr + (size_t)e * H : part + slot * H) + v * 8);
      o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
      if (!whole) part_b[slot] = bias;
      else if (dbias) dbias[e] = bias;
    }
  }
}

// Experts whose list spans several pieces, and experts without pairs.
__global__ void __launch_bounds__(256) route_wgrad_join_kernel(const int32_t* __restrict__ offsets, int P, int E,
                                                                int H, int chunk, const float* __restrict__ part,
                                                                const float* __restrict__ part_b,
                                                                float* __restrict__ dwr, float* __restrict__ dbias,
                                                                int* status) {
  const int e = blockIdx.x;
  const int n = valid_pairs(offsets, E, P, status);
  int first = __ldg(offsets + e), end = __ldg(offsets + e + 1);
  if (first < 0 || end < first || end > n) first = end = 0;
  const int b0 = first / chunk, b1 = end > first ? (end - 1) / chunk : b0;
  if (end > first && b0 == b1) return;  // whole inside one piece: written already
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float bias = 0.0f;
  if (end > first) {
    for (int b = b0; b <= b1; ++b) {
      // the run starts inside piece b0 (its last run: slot 1), and at the start of the others (slot 0)
      const size_t slot = (size_t)b * 2 + (b == b0 ? 1 : 0);
      if (c < H) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(part + slot * H + c));
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      bias += __ldg(part_b + slot);
    }
  }
  if (c < H) *reinterpret_cast<float4*>(dwr + (size_t)e * H + c) = acc;
  if (dbias && blockIdx.y == 0 && threadIdx.x == 0) dbias[e] = bias;
}

}  // namespace

// Pairs per piece: pieces of 64 once they fill the GPU; shorter for few pairs, where a CTA's serial walk is the time.
int route_bwd_chunk(int P) {
  int c = kChunkMax;
  while (c > 8 && P / c < 148) c >>= 1;
  return c;
}

size_t route_bwd_workspace_floats(int P, int H) {
  const size_t pieces = ((size_t)P + route_bwd_chunk(P) - 1) / route_bwd_chunk(P);
  return pieces * 2 * ((size_t)H + 1);
}

cudaError_t launch_route_bwd(const void* x, const float* scales, const float* w, const float* dw, const int32_t* offsets,
                             const int32_t* perm_src, const int32_t* perm_k, int T, int K, int E, int H, float* dl,
                             float* dwr, float* dbias, float* ws, int* status, cudaStream_t s) {
  const int P = T * K, chunk = route_bwd_chunk(P);
  const unsigned pieces = (unsigned)((P + chunk - 1) / chunk);
  float* part = ws;
  float* part_b = ws + (size_t)pieces * 2 * H;
  if (P > 0) {
    route_dlogit_kernel<<<(unsigned)((P + 255) / 256), 256, 0, s>>>(w, dw, T, K, dl);
    auto* kern = scales ? route_wgrad_kernel<true> : route_wgrad_kernel<false>;
    kern<<<dim3(pieces, (H + kCols - 1) / kCols), 256, 0, s>>>(x, scales, dl, offsets, perm_src, perm_k, T, K, E, H,
                                                               chunk, dwr, dbias, part, part_b, status);
  }
  route_wgrad_join_kernel<<<dim3((unsigned)E, (H + 1023) / 1024), 256, 0, s>>>(offsets, P, E, H, chunk, part, part_b,
                                                                              dwr, dbias, status);
  return cudaGetLastError();
}

}  // namespace moe
