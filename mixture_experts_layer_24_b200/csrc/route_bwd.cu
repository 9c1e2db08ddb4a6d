// route_bwd.cu -- gradient of the router. With w = softmax of a token's K
// selected logits and dw its gradient,
//   dl[t,k]   = w[t,k] * (dw[t,k] - sum_j w[t,j] dw[t,j])
//   dWr[e, :] = sum over the pairs (t,k) of expert e of dl[t,k] * x[t, :]
//   dbias[e]  = sum over the same pairs of dl[t,k]
// (logits outside the top k get no gradient). Sums are fp32. A pair that the
// forward dropped has dw = 0 and a dl all the same, so the sums are over every
// chosen pair: the list of pairs has to be the sort of the router's own choice
// (moe_route_bwd_topk makes it), not that of the kept pairs.
//
// The pairs come sorted by expert, so dWr is a segmented sum of scaled
// rows: the sorted list is cut every `chunk` pairs, a CTA takes one piece and
// 2048 columns, and adds up each expert's run inside it. A run that is its
// expert's whole list is written out at once; the first and last run of a
// piece may be parts, which go to the workspace and are added in order by a
// second kernel. The order of every sum depends on the routing alone, so
// results repeat exactly.
//
// Two launches, the second one starting under the first (programmatic
// dependent launch): until the parts are there it writes the zero rows of
// experts without pairs. A piece computes the dl it needs itself; CTAs behind
// the pieces write dl out for every pair, dropped ones too.
//
// x is read from L2 once per pair (K times over), 268 MB for 4096 tokens of
// 8 x 4096: 31.5 us for the two kernels on warm inputs, 35 to 37 us a call on
// new ones, where HBM needs 6.2 us for x and dWr once. What bounds it is issue
// and latency together: paired fp32 multiply-adds (one instruction, two
// columns) and four rows in flight, four blocks per SM (three or five: 37 and
// 44 us); 16 columns per thread took 36 us, eight rows in flight 42 us, rows
// through shared memory by asynchronous copies, once per pair as here, 54 us,
// and a single thread's walk over the longest expert's parts 4 us more. A block
// that keeps a few columns of all tokens in shared memory would read x once and
// have no parts to join; it has not been built.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kChunkMax = 128;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float dlogit(const float* __restrict__ w, const float* __restrict__ dw, size_t t, int k,
                                        int K) {
  float dot = 0.0f;
  for (int j = 0; j < K; ++j) dot = fmaf(__ldg(w + t * K + j), __ldg(dw + t * K + j), dot);
  return __ldg(w + t * K + k) * (__ldg(dw + t * K + k) - dot);
}

// Number of kept pairs; 0 and a report where offsets[E] is not inside [0, P].
__device__ __forceinline__ int valid_pairs(int n, int P, int* status) {
  if (n >= 0 && n <= P) return n;
  flag_status(status, MOE_DEV_BAD_INDEX);
  return 0;
}

// acc (two columns) += d * f, both lanes rounded as fmaf rounds.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t d2, float lo, float hi) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%2, %3};\n\tfma.rn.f32x2 %0, %1, t, %0;\n\t}"
      : "+l"(acc)
      : "l"(d2), "f"(lo), "f"(hi));
}

// kCkpt: x is an e4m3 checkpoint (codes, one scale per 128 columns). A thread
// owns eight columns.
template <bool kCkpt>
__global__ void __launch_bounds__(256, 4) route_wgrad_kernel(const void* __restrict__ x,
                                                           const float* __restrict__ scales,
                                                           const float* __restrict__ w, const float* __restrict__ dw,
                                                           const int32_t* __restrict__ offsets,
                                                           const int32_t* __restrict__ perm_src,
                                                           const int32_t* __restrict__ perm_k, int T, int K, int E,
                                                           int H, int chunk, int pieces, float* __restrict__ dl,
                                                           float* __restrict__ dwr, float* __restrict__ dbias,
                                                           float* __restrict__ part, float* __restrict__ part_b,
                                                           int* status) {
  using Piece = typename std::conditional<kCkpt, uint2, uint4>::type;  // eight columns
  __shared__ int s_off[kMaxExperts + 1];
  __shared__ int2 s_pair[kChunkMax];  // a pair's token (-1: none) and the bits of its dl
  __shared__ int s_e[kChunkMax];      // its expert
  pdl_trigger();
  const int tid = threadIdx.x, nt = blockDim.x;
  if ((int)blockIdx.x >= pieces) {  // dl of every pair, in token order
    const long long i = (long long)(blockIdx.x - pieces) * nt + tid;
    if (blockIdx.y == 0 && i < (long long)T * K) dl[i] = dlogit(w, dw, i / K, (int)(i % K), K);
    return;
  }
  const int p0 = blockIdx.x * chunk;
  for (int e = tid; e <= E; e += nt) s_off[e] = __ldg(offsets + e);
  // places behind the kept pairs may hold anything: taken as no pair, and reported below if they are not behind
  for (int j = tid; j < min(chunk, T * K - p0); j += nt) {
    const int t = __ldg(perm_src + p0 + j), k = __ldg(perm_k + p0 + j);
    const bool good = t >= 0 && t < T && k >= 0 && k < K;
    s_pair[j] = good ? make_int2(t, __float_as_int(dlogit(w, dw, t, k, K))) : make_int2(-1, 0);
  }
  __syncthreads();
  const int n = min(valid_pairs(s_off[E], T * K, status) - p0, chunk);  // this piece's pairs
  if (n <= 0) return;
  bool bad = false;
  for (int j = tid; j < n; j += nt) {
    bad |= s_pair[j].x < 0;
    int e = 0;  // the last expert whose rows start at or before this place
    for (int hi = E; hi - e > 1;) {
      const int mid = (e + hi) >> 1;
      if (s_off[mid] <= p0 + j) e = mid;
      else hi = mid;
    }
    s_e[j] = e;
  }
  if (bad) flag_status(status, MOE_DEV_BAD_INDEX);
  const bool clean = !__syncthreads_or(bad);
  const int V = H / 8;
  const int v = blockIdx.y * nt + tid;
  const bool live = v < V;  // idle threads load too, and store nothing
  const Piece* xv = static_cast<const Piece*>(x) + (live ? v : 0);
  const float* sv = kCkpt ? scales + (live ? v : 0) / 16 : nullptr;
  for (int j = 0; j < n;) {
    const int e = s_e[j];
    const int first = s_off[e], end = s_off[e + 1];
    // offsets that do not rise: at least this pair, so that the walk ends (the sums mean nothing then)
    const int stop = max(j + 1, min(n, end - p0));
    uint64_t acc[4] = {};
    float bias = 0.0f;
    auto add = [&](const Piece& a, float scale, float d) {
      float f[8];
      if constexpr (kCkpt) e4m3x8(a, scale, f);
      else RowBf16::unpack(a, f);
      uint64_t d2;
      asm("mov.b64 %0, {%1, %1};" : "=l"(d2) : "f"(d));
#pragma unroll
      for (int i = 0; i < 4; ++i) fma2(acc[i], d2, f[2 * i], f[2 * i + 1]);
      bias += d;
    };
    // kRows rows in flight, then the rest of the run (and any piece with an entry to leave out) with checks
    constexpr int kRows = 4;
    for (; clean && j + kRows <= stop; j += kRows) {
      Piece a[kRows];
      float sc[kRows], d[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int2 pr = s_pair[j + u];
        d[u] = __int_as_float(pr.y);
        a[u] = __ldg(xv + (size_t)pr.x * V);
        sc[u] = kCkpt ? __ldg(sv + (size_t)pr.x * (V / 16)) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) add(a[u], sc[u], d[u]);
    }
    for (; j < stop; j += kRows) {
      Piece a[kRows];
      float sc[kRows];
      int2 pr[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        pr[u] = j + u < stop ? s_pair[j + u] : make_int2(-1, 0);
        if (pr[u].x < 0) continue;
        a[u] = __ldg(xv + (size_t)pr[u].x * V);
        sc[u] = kCkpt ? __ldg(sv + (size_t)pr[u].x * (V / 16)) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (pr[u].x >= 0) add(a[u], sc[u], __int_as_float(pr[u].y));
    }
    j = stop;
    // whole list of e: final; otherwise a part (0: runs from the piece's first pair, 1: up to its last)
    const bool whole = first >= p0 && end <= p0 + n;
    const size_t slot = (size_t)blockIdx.x * 2 + (first < p0 ? 0 : 1);
    if (live) {
      ulonglong2* o = reinterpret_cast<ulonglong2*>((whole ? dwr + (size_t)e * H : part + slot * H) + v * 8);
      o[0] = make_ulonglong2(acc[0], acc[1]);
      o[1] = make_ulonglong2(acc[2], acc[3]);
    }
    if (blockIdx.y == 0 && tid == 0) {
      if (!whole) part_b[slot] = bias;
      else if (dbias) dbias[e] = bias;
    }
  }
}

// Experts whose list spans several pieces, and experts without pairs (whose
// zeros need not wait for the pieces). Four groups of 64 threads take a quarter
// of the pieces each, kJoinVec x 256 columns (512: 2 us less than 256 or 1024);
// their sums are added in order.
constexpr int kJoinVec = 2;

__global__ void __launch_bounds__(256) route_wgrad_join_kernel(const int32_t* __restrict__ offsets, int P, int E,
                                                                int H, int chunk, const float* part,
                                                                const float* part_b, float* __restrict__ dwr,
                                                                float* __restrict__ dbias, int* status) {
  __shared__ float4 s_acc[3][kJoinVec][64];
  __shared__ float s_bias[3];
  const int e = blockIdx.x, group = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int total = __ldg(offsets + E);
  int first = __ldg(offsets + e), end = __ldg(offsets + e + 1);
  const int n = valid_pairs(total, P, status);
  if (first < 0 || end < first || end > n) first = end = 0;
  const int b0 = first / chunk, b1 = end > first ? (end - 1) / chunk : b0;
  // One CTA always waits, so that this grid is not over before the pieces' (what follows on the stream waits for it).
  if (b1 > b0 || (blockIdx.x == 0 && blockIdx.y == 0)) pdl_wait();
  if (end > first && b0 == b1) return;  // whole inside one piece: written there
  float4 acc[kJoinVec] = {};
  float bias = 0.0f;
  auto column = [&](int i) { return ((blockIdx.y * kJoinVec + i) * 64 + l) * 4; };
  if (end > first) {
    // the run starts inside piece b0 (its last run: slot 1), and at the start of the others (slot 0)
    constexpr int kAhead = 8 / kJoinVec;
    const int each = (b1 - b0 + 4) / 4, lo = b0 + group * each, hi = min(b1 + 1, lo + each);
    for (int b = lo; b < hi; b += kAhead) {
      float4 v[kAhead][kJoinVec];
      float vb[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const size_t slot = (size_t)(b + u) * 2 + (b + u == b0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < kJoinVec; ++i) {
          v[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (b + u < hi && column(i) < H) v[u][i] = *reinterpret_cast<const float4*>(part + slot * H + column(i));
        }
        vb[u] = b + u < hi && blockIdx.y == 0 ? part_b[slot] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int i = 0; i < kJoinVec; ++i)
          acc[i].x += v[u][i].x, acc[i].y += v[u][i].y, acc[i].z += v[u][i].z, acc[i].w += v[u][i].w;
        bias += vb[u];
      }
    }
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < kJoinVec; ++i) s_acc[group - 1][i][l] = acc[i];
      if (l == 0) s_bias[group - 1] = bias;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 0; g < 3; ++g) {
#pragma unroll
        for (int i = 0; i < kJoinVec; ++i) {
          const float4 v = s_acc[g][i][l];
          acc[i].x += v.x, acc[i].y += v.y, acc[i].z += v.z, acc[i].w += v.w;
        }
        bias += s_bias[g];
      }
    }
  }
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < kJoinVec; ++i)
    if (column(i) < H) *reinterpret_cast<float4*>(dwr + (size_t)e * H + column(i)) = acc[i];
  if (dbias && blockIdx.y == 0 && threadIdx.x == 0) dbias[e] = bias;
}

// Pairs per piece: two pieces per SM of a B200 (at 32768 pairs of 384 experts three cost 2 us more, four 3 us: more
// parts to add), 8 at least (a CTA's serial walk is the time then) and 128 at most. The number of SMs is a constant,
// so that the order of the sums follows from the number of pairs alone, on a part of a GPU too.
constexpr int kPieces = 2 * 148;

int route_bwd_chunk(int P) {
  const int c = (P + kPieces - 1) / kPieces;
  return std::min(kChunkMax, std::max(8, (c + 3) / 4 * 4));
}

}  // namespace

size_t route_bwd_workspace_floats(int P, int H) {
  const size_t pieces = ((size_t)P + route_bwd_chunk(P) - 1) / route_bwd_chunk(P);
  return pieces * 2 * ((size_t)H + 1);
}

cudaError_t launch_route_bwd(const void* x, const float* scales, const float* w, const float* dw,
                             const int32_t* offsets, const int32_t* perm_src, const int32_t* perm_k, int T, int K,
                             int E, int H, float* dl, float* dwr, float* dbias, float* ws, int* status, cudaStream_t s,
                             bool pdl) {
  const int P = T * K, chunk = route_bwd_chunk(P);
  const int pieces = (P + chunk - 1) / chunk;
  float* part = ws;
  float* part_b = ws + (size_t)pieces * 2 * H;
  if (P > 0) {
    const int threads = std::min(256, (H / 8 + 31) / 32 * 32);
    const dim3 grid((unsigned)(pieces + (P + threads - 1) / threads), (unsigned)((H / 8 + threads - 1) / threads));
    auto* kern = scales ? route_wgrad_kernel<true> : route_wgrad_kernel<false>;
    const cudaError_t err = launch_ex(kern, grid, dim3((unsigned)threads), 0, s, false, x, scales, w, dw, offsets,
                                      perm_src, perm_k, T, K, E, H, chunk, pieces, dl, dwr, dbias, part, part_b,
                                      status);
    if (err != cudaSuccess) return err;
  }
  constexpr int kJoinCols = 256 * kJoinVec;
  return launch_ex(route_wgrad_join_kernel, dim3((unsigned)E, (unsigned)((H + kJoinCols - 1) / kJoinCols)), dim3(256),
                   0, s, pdl && P > 0, offsets, P, E, H, chunk, (const float*)part, (const float*)part_b, dwr, dbias,
                   status);
}

}  // namespace moe
