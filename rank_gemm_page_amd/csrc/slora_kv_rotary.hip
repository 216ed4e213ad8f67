// The table of cosines and sines that an append rotates by (include/slora.h,
// slora_kv_rotary_table).
#include <hip/hip_runtime.h>

#include "slora_device.h"
#include "slora_kv.h"

namespace slora {

// Angles are held in turns: p * (hi + lo) of a position p below 2^31 leaves its
// whole turns exactly (the product's rounding error comes back from the fma, so
// nothing else may be fused with the product), and far positions are as good as
// near ones.
__global__ __launch_bounds__(kThreads) void kv_rotary_kernel(KvRotary R) {
#pragma clang fp contract(off)
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= R.n * R.half) return;
  const int64_t row = i / R.half;
  const int pair = (int)(i - row * R.half);
  const double p = (double)(R.first + row), hi = R.turn_hi[pair], whole = p * hi;
  const double rest = __builtin_fma(p, hi, -whole) + p * R.turn_lo[pair];
  double s, c;
  sincospi(2. * ((whole - rint(whole)) + rest), &s, &c);
  R.out[row * 2 * R.half + pair] = (float)(c * R.amplitude);
  R.out[(row * 2 + 1) * R.half + pair] = (float)(s * R.amplitude);
}

hipError_t launch_kv_rotary(const KvRotary& R, hipStream_t stream) {
  const int64_t blocks = (R.n * R.half + kThreads - 1) / kThreads;
  if (blocks <= 0) return hipSuccess;
  void* args[] = {const_cast<KvRotary*>(&R)};
  return hipLaunchKernel((const void*)kv_rotary_kernel, dim3((unsigned)blocks), dim3(kThreads), args, 0, stream);
}

}  // namespace slora
