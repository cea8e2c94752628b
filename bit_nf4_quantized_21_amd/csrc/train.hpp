// Launchers of the operators around a training step beside the linears: the
// cross entropy over a vocabulary (head_loss.hip), the global gradient norm
// and clipping (clip.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlora {

// Operands of so many bytes and more that a call reads once, or whose second
// reading its caches cannot serve, are marked as used once where they are read (three
// quarters of the last cache, 256 MB: about here the mark begins to pay).
constexpr int64_t kStreamBytes = (int64_t)192 << 20;

// Softmax cross entropy of T tokens over the rows of a head W [V,K], and its
// gradient where dX is given.
struct HeadLossArgs {
  const uint16_t* X;       // [T,K] bf16
  const uint16_t* W;       // [V,K] bf16
  const int64_t* targets;  // [T]
  const float* dloss;      // [T] or null (the mean's gradient)
  int64_t T, K, V;
  float* loss;             // [T]
  float* lse;              // [T]
  float* mean;             // [1]
  uint16_t* dX;            // [T,K] bf16 or null
};
size_t head_loss_workspace_bytes(int64_t T, int64_t K, int64_t V, bool grad);
hipError_t launch_head_loss(const HeadLossArgs& a, void* ws, hipStream_t s);

// One gradient of a set: n values of `grad` (fp32 where `wide`, else bf16),
// written clipped to `out` (fp32 where `out_wide`) unless that is null.
struct GradTensor {
  const void* grad;
  void* out;
  int64_t n;
  bool wide, out_wide;
};
size_t clip_grads_workspace_bytes(int count);
hipError_t launch_clip_grads(int count, const GradTensor* g, float max_norm, float* norm_out, void* ws,
                             hipStream_t s);

}  // namespace qlora
