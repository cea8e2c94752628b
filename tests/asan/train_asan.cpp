// Host-side checks of the training step's entry points of libqlora under the
// address and undefined-behaviour sanitizers (host code instrumented, no GPU
// needed): refusals, the workspace queries over many shapes, and what a call that
// is accepted hands to its kernels.  The launchers are replaced at link time
// (-Wl,--wrap) by ones that record their arguments, so nothing here reaches a GPU
// and no address given is ever read.  Exit status 0 means every expectation held.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "kernels.hpp"
#include "qlora.h"
#include "train.hpp"

static int failures = 0, launches = 0;
static qlora::GatedArgs gated;
static int gated_act;
static qlora::HeadLossArgs head;
static std::vector<qlora::GradTensor> grads;

#define EXPECT(cond)                                              \
  do {                                                            \
    if (!(cond)) {                                                \
      fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond);   \
      ++failures;                                                 \
    }                                                             \
  } while (0)
#define REFUSED(call, status)          \
  do {                                 \
    const int before_ = launches;      \
    EXPECT((call) == (status));        \
    EXPECT(launches == before_);       \
  } while (0)
#define LAUNCHED(call)                 \
  do {                                 \
    const int before_ = launches;      \
    EXPECT((call) == QLORA_OK);        \
    EXPECT(launches == before_ + 1);   \
  } while (0)

extern "C" {
hipError_t __wrap__ZN5qlora16launch_gated_fwdERKNS_9GatedArgsEiRKNS_8CodebookEPKtPtS8_PfPvP12ihipStream_t(
    const qlora::GatedArgs& a, int act, const qlora::Codebook&, const uint16_t*, uint16_t*, uint16_t*, float*, void*,
    hipStream_t) {
  gated = a;
  gated_act = act;
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora16launch_gated_bwdERKNS_9GatedArgsERKNS_8CodebookEPKtS7_S7_PKfRKNS_10GatedGradsEPvP12ihipStream_t(
    const qlora::GatedArgs& a, const qlora::Codebook&, const uint16_t*, const uint16_t*, const uint16_t*, const float*,
    const qlora::GatedGrads&, void*, hipStream_t) {
  gated = a;
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora16launch_head_lossERKNS_12HeadLossArgsEPvP12ihipStream_t(const qlora::HeadLossArgs& a, void*,
                                                                                     hipStream_t) {
  head = a;
  ++launches;
  return hipSuccess;
}
hipError_t __wrap__ZN5qlora17launch_clip_gradsEiPKNS_10GradTensorEfPfPvP12ihipStream_t(int n, const qlora::GradTensor* g,
                                                                                       float, float*, void*, hipStream_t) {
  grads.assign(g, g + n);
  ++launches;
  return hipSuccess;
}
}

namespace {
constexpr uintptr_t kBase = 0x100000;
template <class T>
T* at(uintptr_t offset = 0) {
  return reinterpret_cast<T*>(kBase + offset);
}
constexpr size_t kMuch = size_t(1) << 40;

void check_gated() {
  const qlora_adapted_weight w{at<uint8_t>(), at<uint8_t>(16), at<float>(32), at<uint16_t>(48), at<uint16_t>(64)};
  auto fwd = [&](int64_t T, int64_t K, int64_t N, int32_t r, int act, size_t ws) {
    return qlora_gated_fwd(QLORA_QTYPE_FP4, act, at<uint16_t>(), T, K, N, &w, &w, r, 16.0f, at<uint16_t>(), nullptr,
                           at<float>(), at<void>(), ws, nullptr);
  };
  auto bwd = [&](int64_t T, int64_t K, int64_t N, int32_t r, size_t ws) {
    return qlora_gated_bwd(QLORA_QTYPE_NF4, at<uint16_t>(), at<uint16_t>(), at<uint16_t>(), nullptr, T, K, N, &w, &w, r,
                           8.0f, at<uint16_t>(), at<uint16_t>(), at<uint16_t>(), at<uint16_t>(), at<uint16_t>(),
                           at<void>(), ws, nullptr);
  };
  const int64_t Ts[] = {1, 16, 17, 255, 257, 4096, 16384}, Ks[] = {64, 640, 8192, 65536}, Ns[] = {8, 776, 22016};
  for (int64_t T : Ts)
    for (int64_t K : Ks)
      for (int64_t N : Ns)
        for (int32_t r : {8, 72, 128}) {
          const size_t f = qlora_gated_fwd_workspace_bytes(T, K, N, r), b = qlora_gated_bwd_workspace_bytes(T, K, N, r);
          EXPECT((f == 0) == (b == 0));
          if (!f) {
            REFUSED(fwd(T, K, N, r, 0, kMuch), QLORA_ERR_SHAPE);
            continue;
          }
          LAUNCHED(fwd(T, K, N, r, QLORA_ACT_GELU, f));
          EXPECT(gated.T == T && gated.K == K && gated.N == N && gated.r == r && gated_act == QLORA_ACT_GELU);
          EXPECT(gated.s == 16.0f / (float)r && gated.w[1].B == at<uint16_t>(64));
          REFUSED(fwd(T, K, N, r, 0, f - 1), QLORA_ERR_WORKSPACE);
          LAUNCHED(bwd(T, K, N, r, b));
          REFUSED(bwd(T, K, N, r, b - 1), QLORA_ERR_WORKSPACE);
        }
  REFUSED(fwd(8, 64, 64, 8, 3, kMuch), QLORA_ERR_UNSUPPORTED);
  REFUSED(fwd(int64_t(1) << 40, 64, 64, 8, 0, kMuch), QLORA_ERR_SHAPE);
  REFUSED(fwd(8, INT64_MAX - 63, 64, 8, 0, kMuch), QLORA_ERR_SHAPE);
  REFUSED(bwd(INT64_MIN, 64, 64, 8, kMuch), QLORA_ERR_SHAPE);
}

void check_head() {
  auto loss = [&](int64_t T, int64_t K, int64_t V, bool grad, size_t ws) {
    return qlora_head_loss(at<uint16_t>(), T, K, at<uint16_t>(), V, at<int64_t>(), nullptr, at<float>(), at<float>(),
                           at<float>(), grad ? at<uint16_t>() : nullptr, at<void>(), ws, nullptr);
  };
  const int64_t Ts[] = {1, 64, 65, 4096, 4097, 100000, int64_t(1) << 23}, Ks[] = {64, 4096, int64_t(1) << 20},
                Vs[] = {1, 255, 32000, 131072, int64_t(1) << 30};
  for (int64_t T : Ts)
    for (int64_t K : Ks)
      for (int64_t V : Vs)
        for (bool grad : {false, true}) {
          const size_t n = qlora_head_loss_workspace_bytes(T, K, V, grad);
          if (!n) {
            REFUSED(loss(T, K, V, grad, kMuch), QLORA_ERR_SHAPE);
            continue;
          }
          LAUNCHED(loss(T, K, V, grad, n));
          EXPECT(head.T == T && head.K == K && head.V == V && (head.dX != nullptr) == grad);
          REFUSED(loss(T, K, V, grad, n - 1), QLORA_ERR_WORKSPACE);
        }
  const int64_t bad[][3] = {{-1, 64, 8}, {INT64_MAX, 64, 8}, {8, INT64_MAX, 8}, {8, 64, INT64_MAX}, {8, 64, INT64_MIN},
                            {8, 96, 8}, {int64_t(1) << 22, 4096, 8}, {int64_t(1) << 20, 64, int64_t(1) << 20}};
  for (const auto& b : bad) REFUSED(loss(b[0], b[1], b[2], true, kMuch), QLORA_ERR_SHAPE);
}

void check_clip() {
  auto clip = [&](const std::vector<qlora_grad>& g, float max_norm) {
    return qlora_clip_grads((int32_t)g.size(), g.data(), max_norm, at<float>(), at<void>(), kMuch, nullptr);
  };
  auto entry = [](uintptr_t grad, uintptr_t out, int64_t n, int type = 0, int out_type = 0) {
    return qlora_grad{at<void>(grad), at<void>(out), n, type, out_type};
  };
  // Many tensors in any order, in place and beside each other; then one that overlaps.
  std::vector<qlora_grad> many;
  for (int i = 0; i < 3000; ++i) {
    const uintptr_t a = (uintptr_t)((i * 7919) % 3000) * 256;
    many.push_back(entry(a, a, i % 129));
  }
  LAUNCHED(clip(many, 1.0f));
  EXPECT(grads.size() == 3000 - 24);  // those without values are left out
  many[5] = entry((uintptr_t)((5 * 7919) % 3000) * 256, (uintptr_t)((6 * 7919) % 3000) * 256 + 2, 1);
  REFUSED(clip(many, 1.0f), QLORA_ERR_SHAPE);
  LAUNCHED(clip(many, 0.0f));
  for (const auto& g : grads) EXPECT(g.out == nullptr);  // the norm alone writes nothing
  // From fp32 tensors to views of one bf16 buffer.
  std::vector<qlora_grad> flat;
  for (int i = 0; i < 200; ++i) flat.push_back(entry(0x100000 + i * 4096, 0x800000 + i * 200, 100, 1, 0));
  LAUNCHED(clip(flat, 1.0f));
  EXPECT(grads.size() == 200 && grads[7].wide && !grads[7].out_wide && grads[7].n == 100);
  flat.push_back(entry(0x200000, 0x800000 + 199 * 200 + 198, 1, 0, 0));
  REFUSED(clip(flat, 1.0f), QLORA_ERR_SHAPE);
  LAUNCHED(clip({}, 1.0f));
  EXPECT(grads.empty());
  REFUSED(clip({entry(0, 0, INT64_MAX)}, 1.0f), QLORA_ERR_SHAPE);
  std::vector<qlora_grad> huge;
  for (int i = 0; i < 17; ++i) huge.push_back(entry((uintptr_t)i << 42, (uintptr_t)i << 42, int64_t(1) << 40));
  REFUSED(clip(huge, 1.0f), QLORA_ERR_SHAPE);
  REFUSED(clip({entry(0, 0, 4)}, NAN), QLORA_ERR_UNSUPPORTED);
  LAUNCHED(clip({entry(0, 0, 4)}, INFINITY));
}
}  // namespace

int main() {
  check_gated();
  check_head();
  check_clip();
  if (failures) {
    fprintf(stderr, "%d expectation(s) failed\n", failures);
    return 1;
  }
  printf("train_asan: all host checks passed (%d launches recorded)\n", launches);
  return 0;
}
