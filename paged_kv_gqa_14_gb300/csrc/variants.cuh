// What the kernels of the attention variants (decode_variants.cu, prefill_variants.cu) share: the parameters of the
// position bias and of the difference, and the last steps of an output row.
//
//   kBias  out = softmax(scale q.k + bias[bucket(distance)]) V
//   kDiff  out = out_scale [w] x [/ sqrt(mean x^2 + eps)],  x = a_0 V - lambda a_1 V,  a_c the map of q head 2h + c and
//          k head 2g + c, V the two v heads of the pair side by side
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFltMax = 3.4028234663852886e38f;
// A row's reference m, which its weights 2^(s - m) count from, lies this much above the largest score that it was set by (log2
// domain), and is raised only when a score exceeds it.  No weight is above 1, so sums over n keys hold V up to 2^127 / n
// (a row's first weights are near 2^-20, where bf16 and fp32 are as fine as at 1, and V below 2^-106 loses bits).  What a raise
// costs is a rescaling of the row's sums, and in the prefill, where a warp's 32 rows wait for it, a slack of 8 had that happen
// in a third of the tiles of a chunk behind 12,288 keys of random values.
constexpr float kVarSlack = 20.f;

// A bias in the log2 domain.  A finite one stays finite: the lowest values of a type are masks that leave keys alike.
__device__ __forceinline__ float bias_log2(float b) {
  const float x = b * kLog2e;
  const float inf = __int_as_float(0x7f800000);
  return fabsf(x) == inf && fabsf(b) != inf ? copysignf(kFltMax, b) : x;
}
__device__ __forceinline__ float bias_at(const BiasArgs& b, int bucket, int head) {
  const int64_t e = static_cast<int64_t>(bucket) * b.stride + head;
  return bias_log2(b.is_bf16 ? __bfloat162float(__ldg(static_cast<const bf16*>(b.table) + e))
                             : __ldg(static_cast<const float*>(b.table) + e));
}
// The last i < n with starts[i] <= distance (starts[0] = 0).
__device__ __forceinline__ int bucket_of(const int* starts, int n, int distance) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= distance)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// 1 / den, 0 for a row that no key was left for (its sums are 0).
__device__ __forceinline__ float inverse_or_0(float den) { return den == 0.f ? 0.f : 1.f / den; }

}  // namespace pkv
