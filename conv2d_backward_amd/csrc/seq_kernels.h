// seq_kernels.h -- launchers of the sequence kernels, called by seq_api.cpp
// after it has checked the arguments.  Each returns hipGetLastError().
#pragma once

#include <hip/hip_runtime_api.h>

#include "sequence_ops.h"

namespace seq {

hipError_t launch_conv_forward(const causal_conv_args &a, hipStream_t s);
hipError_t launch_conv_backward(const causal_conv_backward_args &a, hipStream_t s);
hipError_t launch_conv_step(const causal_conv_step_args &a, hipStream_t s);
int64_t conv_backward_workspace(int B, int D, int L, int K);

hipError_t launch_scan_forward(const state_scan_args &a, hipStream_t s);
int64_t scan_forward_items(const state_scan_args &a);  // of the grid's x
hipError_t launch_scan_step(const state_scan_step_args &a, hipStream_t s);
hipError_t launch_scan_backward(const state_scan_backward_args &a, hipStream_t s);
int64_t scan_backward_workspace(int B, int D, int L, int N, int G);
// How the work is dealt, as text.
void scan_forward_plan(const state_scan_args &a, char *buf, size_t len);
void scan_backward_plan(int B, int D, int L, int N, int G, char *buf, size_t len);

hipError_t launch_norm_forward(const block_norm_args &a, hipStream_t s);
hipError_t launch_norm_backward(const block_norm_backward_args &a, hipStream_t s);
int norm_columns(int64_t B, int64_t D, int64_t L);  // positions of a forward work-group
int64_t norm_workspace(int B, int D, int L, int backward);

hipError_t launch_gated_forward(const gated_scan_args &a, hipStream_t s);
hipError_t launch_gated_backward(const gated_scan_backward_args &a, hipStream_t s);
hipError_t launch_gated_step(const gated_scan_step_args &a, hipStream_t s);
int64_t gated_backward_workspace(int B, int D, int L);  // 0: none needed
void gated_plan(int64_t rows, int64_t L, int backward, char *buf, size_t len);

hipError_t launch_quantize(const quantize_tokens_args &a, hipStream_t s);
hipError_t launch_project(const project_int8_args &a, hipStream_t s);
hipError_t launch_project_step(const project_int8_step_args &a, hipStream_t s);
int64_t project_step_workspace(int32_t dtype, int B, int D, int E);  // 0: none needed

}  // namespace seq
