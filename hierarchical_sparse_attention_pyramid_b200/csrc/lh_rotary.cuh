// Arguments of the rotary kernel.
#pragma once

#include "lh_common.cuh"

namespace lh {

struct RotaryTensor {
  const void* in;
  void* out;
  int64_t si[3], so[3];  // strides of batch, head, token in elements
};

struct RotaryArgs {
  int64_t B, N;
  int Hq, Hk, d, rot;
  int units, rot_units;  // set by the launch
  RotaryTensor q, k;
  const double* freq;  // [rot/2] radians a position
  const int32_t* pos;  // [B][N] or NULL: 0 .. N-1
  float amp, amp_sin;  // amplitude; with the sign of the direction
};

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool half, cudaStream_t st);

}  // namespace lh
