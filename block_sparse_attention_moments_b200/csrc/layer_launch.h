// layer_launch.h — launches of the layer operators' kernels, one translation
// unit each: the arguments have been checked, dev is the current device.
#pragma once

#include "linear.cuh"
#include "norm.cuh"
#include "rope.cuh"

namespace solattn {

struct LinearOperands {
  const int8_t* a;
  long long a_pitch;
  const int8_t* w;
  long long w_pitch;
};

// vec: rows and vectors can be read 8 channels at a time; wide: rows of a
// 16-bit type 16 at a time.  One for each pair of types (of x and x', and of y
// and h).
using LaunchNorm = int(const NormParams& p, bool vec, bool wide, int dev, int sms, cudaStream_t st);
LaunchNorm launch_norm_bf16, launch_norm_fp16, launch_norm_fp32, launch_norm_fp32_bf16, launch_norm_fp32_fp16;

int launch_rope(const RopeParams& p, int dtype, int dev, int sms, cudaStream_t st);

int launch_linear(const LinearParams& p, const LinearOperands& o, int dtype, int dev, int sms, cudaStream_t st);

// Reads and clears the status word of the products in one step on st, and synchronises it.
int read_linear_status(cudaStream_t st, unsigned* status);

}  // namespace solattn
