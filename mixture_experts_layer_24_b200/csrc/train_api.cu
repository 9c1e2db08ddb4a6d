// train_api.cu -- the C ABI of the training calls: argument checks, tensor maps
// and launches of train_rows.cu, swiglu_ckpt.cu, route_bwd.cu and expert_product.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <string>

#include "../../include/moe.h"
#include "ctx.h"
#include "train.h"

using namespace moe;

namespace {

constexpr int kMaxRows = 65536 * 32;  // pairs of the largest batch
constexpr int kMaxFeatures = 16384;   // 2I at the largest I

moe_status_t fail(moe_status_t st, const std::string& msg) {
  record_error(msg.c_str());
  return st;
}

// The context's device while a call runs; the caller's is put back.
struct OnDevice {
  int prev = -1;
  cudaError_t err;
  explicit OnDevice(int device) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != device) err = cudaSetDevice(device);
    else prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

moe_status_t check_tokens(const moe_ctx_t* ctx, int T) {
  if (!ctx) return fail(MOE_ERR_INVALID_ARG, "NULL context");
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (T > 65536) return fail(MOE_ERR_UNSUPPORTED, "T must be <= 65536");
  return MOE_OK;
}

moe_status_t check_rows(const moe_ctx_t* ctx, int rows) {
  if (!ctx) return fail(MOE_ERR_INVALID_ARG, "NULL context");
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "the number of rows must be >= 0");
  if (rows > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "at most 65536 * 32 rows");
  return MOE_OK;
}

moe_status_t check_row_type(int dtype) {
  if (dtype != MOE_T_BF16 && dtype != MOE_T_F32)
    return fail(MOE_ERR_INVALID_ARG, "dtype must be MOE_T_BF16 or MOE_T_F32");
  return MOE_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace of moe_route_bwd_topk: that of moe_route_bwd, the list of pairs, and the sort's scratch.
struct SortedPairs {
  size_t rank, chunk_counts, counts, offsets, perm_src, perm_k, inv, total;
};

SortedPairs sorted_pairs(size_t first, const moe_config_t& c, int T) {
  const size_t pairs = (size_t)T * c.top_k * 4, experts = (size_t)c.n_experts * 4;
  SortedPairs s{};
  size_t o = align256(first);
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  s.rank = take(pairs);
  s.chunk_counts = take(64 * experts);  // permute_chunk_tokens makes at most 64 chunks
  s.counts = take(experts);
  s.offsets = take(experts + 4);
  s.perm_src = take(pairs);
  s.perm_k = take(pairs);
  s.inv = take(pairs);
  s.total = o;
  return s;
}

moe_status_t check_route_bwd(const moe_ctx_t* ctx, const void* x, const float* topk_w, const float* dtopk_w, int T,
                             const float* dlogit, const float* dw_router, const void* ws, size_t ws_bytes,
                             size_t need) {
  if (!dw_router) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (T > 0 && (!x || !topk_w || !dtopk_w || !dlogit)) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({x, dw_router})) return fail(MOE_ERR_INVALID_ARG, "x and dw_router must be 16-byte aligned");
  if (need && (!ws || ws_bytes < need))
    return fail(MOE_ERR_INVALID_ARG,
                "workspace too small (see moe_route_bwd_workspace_size, moe_route_bwd_topk_workspace_size)");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return MOE_OK;
}

moe_status_t check_features(int n_in, int n_out) {
  if (n_in <= 0 || n_out <= 0) return fail(MOE_ERR_INVALID_ARG, "n_in and n_out must be positive");
  if (n_in % 128 || n_out % 128 || n_in > kMaxFeatures || n_out > kMaxFeatures)
    return fail(MOE_ERR_UNSUPPORTED, "n_in and n_out must be multiples of 128, at most 16384");
  return MOE_OK;
}

// bf16 or fp32 [rows, inner] with boxes of 128 bytes x box_rows rows, 128-byte swizzle.
moe_status_t encode(const moe_ctx_t* ctx, CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t rows,
                    uint32_t box_rows, bool f32 = false) {
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {inner * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 32u : 64u, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = ctx->encode_tiled(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                                 const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
  return MOE_OK;
}

// Maps of a K-major rows operand, one per box height.
moe_status_t encode_rows(const moe_ctx_t* ctx, ProductMaps* maps, const void* ptr, uint64_t inner, uint64_t rows) {
  for (int i = 0; i < 4; ++i) {
    const moe_status_t st = encode(ctx, &maps->n[i], ptr, inner, rows, 16u << i);
    if (st != MOE_OK) return st;
  }
  return MOE_OK;
}

}  // namespace

#define ON_DEVICE(ctx)                                                                                      \
  OnDevice on_device_((ctx)->device);                                                                      \
  if (on_device_.err != cudaSuccess)                                                                       \
  return fail(MOE_ERR_CUDA, std::string("cudaSetDevice: ") + cudaGetErrorString(on_device_.err))

extern "C" {

moe_status_t moe_dispatch(moe_ctx_t* ctx, const void* x, const float* x_scales, int dtype, const int32_t* inv, int T,
                          void* x_sorted, moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if (dtype != MOE_T_E4M3_B128 && (st = check_row_type(dtype)) != MOE_OK) return st;
  if ((dtype == MOE_T_E4M3_B128) != (x_scales != nullptr) && T > 0)
    return fail(MOE_ERR_INVALID_ARG, "x_scales goes with MOE_T_E4M3_B128, and only with it");
  if (T == 0) return MOE_OK;
  if (!x || !inv || !x_sorted) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({x, x_sorted})) return fail(MOE_ERR_INVALID_ARG, "x and x_sorted must be 16-byte aligned");
  ON_DEVICE(ctx);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_ROWS, s);
  MOE_CUDA(launch_dispatch(x, x_scales, dtype, inv, T, ctx->cfg.top_k, ctx->cfg.hidden, x_sorted, ctx->d_status, s));
  return MOE_OK;
}

moe_status_t moe_dispatch_bwd(moe_ctx_t* ctx, const void* dx_sorted, int dtype, const int32_t* inv,
                              const float* dlogit, const int32_t* topk_idx, const float* w_router, int T, void* dx,
                              moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if ((st = check_row_type(dtype)) != MOE_OK) return st;
  const int given = (dlogit != nullptr) + (topk_idx != nullptr) + (w_router != nullptr);
  if (T > 0 && given != 0 && given != 3)
    return fail(MOE_ERR_INVALID_ARG, "dlogit, topk_idx and w_router go together");
  if (T == 0) return MOE_OK;
  if (!dx_sorted || !inv || !dx) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({dx_sorted, dx, w_router}))
    return fail(MOE_ERR_INVALID_ARG, "dx_sorted, dx and w_router must be 16-byte aligned");
  ON_DEVICE(ctx);
  const moe_config_t& c = ctx->cfg;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_ROWS, s);
  MOE_CUDA(launch_dispatch_bwd(dx_sorted, dtype, inv, dlogit, topk_idx, w_router, T, c.top_k, c.n_experts, c.hidden,
                               dx, ctx->d_status, s));
  return MOE_OK;
}

moe_status_t moe_combine_weighted(moe_ctx_t* ctx, const void* y_sorted, int dtype, const float* topk_w,
                                  const int32_t* inv, int T, void* out, moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if ((st = check_row_type(dtype)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!y_sorted || !topk_w || !inv || !out) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({y_sorted, out})) return fail(MOE_ERR_INVALID_ARG, "y_sorted and out must be 16-byte aligned");
  ON_DEVICE(ctx);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_ROWS, s);
  MOE_CUDA(launch_combine_weighted(y_sorted, dtype, topk_w, inv, T, ctx->cfg.top_k, ctx->cfg.hidden, out,
                                   ctx->d_status, s));
  return MOE_OK;
}

moe_status_t moe_combine_weighted_bwd(moe_ctx_t* ctx, const void* dout, const void* y_sorted, int dtype,
                                      const float* topk_w, const int32_t* inv, int T, void* dy_sorted,
                                      float* dtopk_w, moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if ((st = check_row_type(dtype)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!dout || !y_sorted || !topk_w || !inv || !dy_sorted || !dtopk_w)
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({dout, y_sorted, dy_sorted}))
    return fail(MOE_ERR_INVALID_ARG, "dout, y_sorted and dy_sorted must be 16-byte aligned");
  ON_DEVICE(ctx);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_ROWS, s);
  MOE_CUDA(launch_combine_weighted_bwd(dout, y_sorted, dtype, topk_w, inv, T, ctx->cfg.top_k, ctx->cfg.hidden,
                                       dy_sorted, dtopk_w, ctx->d_status, s));
  return MOE_OK;
}

moe_status_t moe_swiglu_ckpt(moe_ctx_t* ctx, const void* gu, const int32_t* inv, int rows, void* h, uint8_t* q,
                             float* s, moe_stream_t stream) {
  moe_status_t st = check_rows(ctx, rows);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!gu || !h || !q || !s) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({gu, h, q})) return fail(MOE_ERR_INVALID_ARG, "gu, h and q must be 16-byte aligned");
  ON_DEVICE(ctx);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_SWIGLU, cs);
  MOE_CUDA(launch_swiglu_ckpt(gu, inv, rows, ctx->cfg.intermediate, h, q, s, ctx->d_status, cs));
  return MOE_OK;
}

moe_status_t moe_swiglu_ckpt_bwd(moe_ctx_t* ctx, const uint8_t* q, const float* s, const void* dh,
                                 const float* topk_w, const int32_t* inv, int rows, void* dgu, void* hw,
                                 float* dtopk_w, moe_stream_t stream) {
  moe_status_t st = check_rows(ctx, rows);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!q || !s || !dh || !dgu) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if ((topk_w != nullptr) != (dtopk_w != nullptr)) return fail(MOE_ERR_INVALID_ARG, "topk_w and dtopk_w go together");
  if (hw && !topk_w) return fail(MOE_ERR_INVALID_ARG, "hw goes with topk_w");
  if (!aligned16({q, dh, dgu, hw})) return fail(MOE_ERR_INVALID_ARG, "q, dh, dgu and hw must be 16-byte aligned");
  ON_DEVICE(ctx);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_SWIGLU, cs);
  MOE_CUDA(launch_swiglu_ckpt_bwd(q, s, dh, topk_w, inv, rows, ctx->cfg.intermediate, dgu, hw, dtopk_w,
                                  ctx->d_status, cs));
  return MOE_OK;
}

size_t moe_route_bwd_workspace_size(const moe_ctx_t* ctx, int T) {
  if (!ctx || T < 0 || T > 65536) return 0;
  return route_bwd_workspace_floats(T * ctx->cfg.top_k, ctx->cfg.hidden) * sizeof(float);
}

moe_status_t moe_route_bwd(moe_ctx_t* ctx, const void* x, const float* x_scales, const float* topk_w,
                           const float* dtopk_w, const int32_t* offsets, const int32_t* perm_src,
                           const int32_t* perm_k, int T, float* dlogit, float* dw_router, float* dlogit_bias, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if (!offsets || (T > 0 && (!perm_src || !perm_k))) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  st = check_route_bwd(ctx, x, topk_w, dtopk_w, T, dlogit, dw_router, ws, ws_bytes,
                       moe_route_bwd_workspace_size(ctx, T));
  if (st != MOE_OK) return st;
  ON_DEVICE(ctx);
  const moe_config_t& c = ctx->cfg;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_ROUTE_BWD, s);
  ctx->launches.fetch_add(T > 0 ? kRouteBwdLaunches - 1 : 0, std::memory_order_relaxed);  // Prof counts one
  MOE_CUDA(launch_route_bwd(x, x_scales, topk_w, dtopk_w, offsets, perm_src, perm_k, T, c.top_k, c.n_experts, c.hidden,
                            dlogit, dw_router, dlogit_bias, static_cast<float*>(ws), ctx->d_status, s, ctx->chain));
  return MOE_OK;
}

size_t moe_route_bwd_topk_workspace_size(const moe_ctx_t* ctx, int T) {
  if (!ctx || T < 0 || T > 65536) return 0;
  return sorted_pairs(moe_route_bwd_workspace_size(ctx, T), ctx->cfg, T).total;
}

moe_status_t moe_route_bwd_topk(moe_ctx_t* ctx, const void* x, const float* x_scales, const int32_t* topk_idx,
                                const float* topk_w, const float* dtopk_w, int T, float* dlogit, float* dw_router,
                                float* dlogit_bias, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status_t st = check_tokens(ctx, T);
  if (st != MOE_OK) return st;
  if (T > 0 && !topk_idx) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  st = check_route_bwd(ctx, x, topk_w, dtopk_w, T, dlogit, dw_router, ws, ws_bytes,
                       moe_route_bwd_topk_workspace_size(ctx, T));
  if (st != MOE_OK) return st;
  ON_DEVICE(ctx);
  const moe_config_t& c = ctx->cfg;
  const size_t own = moe_route_bwd_workspace_size(ctx, T);
  const SortedPairs w = sorted_pairs(own, c, T);
  auto at = [&](size_t o) { return reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + o); };
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int chunk = permute_chunk_tokens(T, c.top_k), n_chunks = (T + chunk - 1) / chunk;
  if (T > 0) {
    Prof p(ctx, MOE_PROF_PERMUTE, s);
    MOE_CUDA(launch_permute_rank(topk_idx, T, c.top_k, c.n_experts, chunk, at(w.rank), at(w.chunk_counts),
                                 ctx->d_status, s, false));
  }
  {
    Prof p(ctx, MOE_PROF_PERMUTE, s);
    MOE_CUDA(launch_permute_scan(at(w.chunk_counts), n_chunks, c.n_experts, at(w.counts), at(w.offsets), s,
                                 ctx->chain && T > 0));
  }
  if (T > 0) {
    Prof p(ctx, MOE_PROF_PERMUTE, s);
    MOE_CUDA(launch_permute_scatter(topk_idx, at(w.rank), at(w.chunk_counts), at(w.offsets), T, c.top_k, c.n_experts,
                                    chunk, at(w.perm_src), at(w.perm_k), at(w.inv), s, ctx->chain));
  }
  return moe_route_bwd(ctx, x, x_scales, topk_w, dtopk_w, at(w.offsets), at(w.perm_src), at(w.perm_k), T, dlogit,
                       dw_router, dlogit_bias, ws, own, stream);
}

moe_status_t moe_expert_product(moe_ctx_t* ctx, const void* a, const void* w, const int32_t* offsets, int P, int n_in,
                                int n_out, int transposed, void* out, moe_stream_t stream) {
  moe_status_t st = check_rows(ctx, P);
  if (st != MOE_OK) return st;
  if ((st = check_features(n_in, n_out)) != MOE_OK) return st;
  if (P == 0) return MOE_OK;
  if (!a || !w || !offsets || !out) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({a, w, out})) return fail(MOE_ERR_INVALID_ARG, "a, w and out must be 16-byte aligned");
  ON_DEVICE(ctx);
  const int E = ctx->cfg.n_experts;
  const int k = transposed ? n_out : n_in, m = transposed ? n_in : n_out;
  ProductMaps maps;
  if ((st = encode(ctx, &maps.m, w, n_in, (uint64_t)E * n_out, transposed ? 64 : 128)) != MOE_OK) return st;
  if ((st = encode_rows(ctx, &maps, a, k, P)) != MOE_OK) return st;
  maps.out = maps.m;  // this form writes its rows itself
  ProductArgs args{offsets, E, P, m, 0, k, out, 0, 0, ctx->d_status};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof p(ctx, MOE_PROF_PRODUCT, s);
  MOE_CUDA(launch_expert_product(transposed ? 1 : 0, maps, args, ctx->num_sms, s));
  return MOE_OK;
}

moe_status_t moe_expert_wgrad(moe_ctx_t* ctx, const void* dy, const void* a, const int32_t* offsets, int P, int n_in,
                              int n_out, int dtype, int accumulate, void* dw, moe_stream_t stream) {
  moe_status_t st = check_rows(ctx, P);
  if (st != MOE_OK) return st;
  if ((st = check_features(n_in, n_out)) != MOE_OK) return st;
  if ((st = check_row_type(dtype)) != MOE_OK) return st;
  if (accumulate && dtype != MOE_T_F32) return fail(MOE_ERR_UNSUPPORTED, "accumulate needs an fp32 gradient");
  if (!dw || !offsets || (P > 0 && (!dy || !a))) return fail(MOE_ERR_INVALID_ARG, "NULL tensor");
  if (!aligned16({dy, a, dw})) return fail(MOE_ERR_INVALID_ARG, "dy, a and dw must be 16-byte aligned");
  ON_DEVICE(ctx);
  const int E = ctx->cfg.n_experts;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P == 0) {
    if (!accumulate)
      MOE_CUDA(cudaMemsetAsync(dw, 0, (size_t)E * n_out * n_in * (dtype == MOE_T_F32 ? 4 : 2), s));
    return MOE_OK;
  }
  ProductMaps maps;
  if ((st = encode(ctx, &maps.m, dy, n_out, P, 64)) != MOE_OK) return st;
  if ((st = encode(ctx, &maps.n[0], a, n_in, P, 64)) != MOE_OK) return st;
  if ((st = encode(ctx, &maps.n[1], a, n_in, P, 16)) != MOE_OK) return st;
  if ((st = encode(ctx, &maps.n[2], dy, n_out, P, 16)) != MOE_OK) return st;
  maps.n[3] = maps.n[2];  // not used in this form
  if ((st = encode(ctx, &maps.out, dw, n_in, (uint64_t)E * n_out, 32, dtype == MOE_T_F32)) != MOE_OK) return st;
  ProductArgs args{offsets, E, P, n_out, n_in, 0, dw, dtype == MOE_T_F32, accumulate, ctx->d_status};
  Prof p(ctx, MOE_PROF_PRODUCT, s);
  MOE_CUDA(launch_expert_product(2, maps, args, ctx->num_sms, s));
  return MOE_OK;
}

}  // extern "C"
