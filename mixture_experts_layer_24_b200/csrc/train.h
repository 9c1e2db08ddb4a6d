// train.h -- declarations shared between the training kernels' files and
// train_api.cu (not part of the public ABI).
#pragma once

#include "internal.h"

namespace moe {

cudaError_t launch_dispatch(const void* x, const float* scales, int dtype, const int32_t* inv, int T, int K, int H,
                            void* xs, int* status, cudaStream_t s);
cudaError_t launch_dispatch_bwd(const void* rows, int dtype, const int32_t* inv, const float* dl, const int32_t* idx,
                                const float* wr, int T, int K, int E, int H, void* dx, int* status, cudaStream_t s);
cudaError_t launch_combine_weighted(const void* y, int dtype, const float* w, const int32_t* inv, int T, int K, int H,
                                    void* out, int* status, cudaStream_t s);
cudaError_t launch_combine_weighted_bwd(const void* dout, const void* y, int dtype, const float* w,
                                        const int32_t* inv, int T, int K, int H, void* dy, float* dw, int* status,
                                        cudaStream_t s);
cudaError_t launch_swiglu_ckpt(const void* gu, const int32_t* inv, int rows, int I, void* h, uint8_t* q, float* s,
                               int* status, cudaStream_t st);
cudaError_t launch_swiglu_ckpt_bwd(const uint8_t* q, const float* s, const void* dh, const float* w,
                                   const int32_t* inv, int rows, int I, void* dgu, void* hw, float* dw, int* status,
                                   cudaStream_t st);
size_t route_bwd_workspace_floats(int P, int H);
constexpr int kRouteBwdLaunches = 2;
cudaError_t launch_route_bwd(const void* x, const float* scales, const float* w, const float* dw,
                             const int32_t* offsets, const int32_t* perm_src, const int32_t* perm_k, int T, int K,
                             int E, int H, float* dl, float* dwr, float* dbias, float* ws, int* status, cudaStream_t s,
                             bool pdl);

// Tensor maps of one expert product: the M operand (weights, or dy), the N
// operand (rows) and the output of the weights' gradient. A K-major N operand
// has one map per box height 16 << i; in the weights' gradient n[0] is the N
// operand in boxes of 64 rows, n[1] and n[2] the N and the M operand in boxes
// of 16.
struct alignas(64) ProductMaps {
  CUtensorMap m;
  CUtensorMap n[4];
  CUtensorMap out;  // weights' gradient: boxes of 32 rows x 128 bytes
};

struct ProductArgs {
  const int32_t* offsets;
  int E, P;
  int m_total;  // features on the M axis: n_out, or n_in in the rows' gradient
  int n_total;  // weights' gradient: n_in
  int k_total;  // K length of the first two forms
  void* out;
  int out_f32, accumulate;  // weights' gradient
  int* status;
};

// form: 0 forward, 1 rows' gradient, 2 weights' gradient
cudaError_t launch_expert_product(int form, const ProductMaps& maps, const ProductArgs& a, int num_sms,
                                  cudaStream_t s);

}  // namespace moe
