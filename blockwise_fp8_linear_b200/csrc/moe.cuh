// moe.cuh -- launchers of the mixture-of-experts and few-token kernels (internal to
// libfp8bw).  Arguments already validated by the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8bw {

// Router: k largest logits of each row and their softmax weights; gradient.
cudaError_t launch_moe_route(const void *logits, bool bf16, int64_t T, int E, int k, bool renorm,
                             float *weights, int32_t *ids, cudaStream_t stream, int num_sms);
cudaError_t launch_moe_route_bwd(const float *dweights, const float *weights, const int32_t *ids,
                                 const void *logits, bool bf16, int64_t T, int E, int k,
                                 bool renorm, void *dlogits, cudaStream_t stream, int num_sms);

// Plan: the (token, choice) pairs laid out by expert in blocks of 128 rows.
int64_t moe_plan_rows(int64_t T, int k, int E);
size_t moe_plan_workspace(int E);
cudaError_t launch_moe_plan(const int32_t *ids, int64_t T, int k, int E, int32_t *seg,
                            int32_t *row, int32_t *src, void *workspace, cudaStream_t stream);

// Few-token linear and the two kernels of the few-token expert layer.
constexpr int kFewMaxTokens = 64;
cudaError_t launch_linear_few(const void *x, int T, const uint8_t *qw, const float *sw, void *y,
                              int64_t N, int64_t K, void *workspace, cudaStream_t stream,
                              int num_sms);
size_t linear_few_workspace(int T, int64_t K);
size_t moe_few_workspace(int T, int k, int64_t H, int64_t I);
cudaError_t launch_moe_few(const void *x, int T, const uint8_t *w1, const float *s1,
                           const uint8_t *w2, const float *s2, const int32_t *ids,
                           const float *weights, int k, int E, int64_t H, int64_t I, void *y,
                           void *workspace, cudaStream_t stream, int num_sms);

// Error word of the few-token kernels' bounded waits (read and cleared; caller synchronizes).
cudaError_t read_and_clear_few_error(int *value);

} // namespace fp8bw
