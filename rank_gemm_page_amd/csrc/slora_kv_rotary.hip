// The table of cosines and sines that an append rotates by (include/slora.h,
// slora_kv_rotary_table).
//
// What bounds it: a sine and cosine in 64 bits are some sixty instructions for 8
// bytes, at which the table's stores would wait for them (131072 positions of 64
// pairs 29 us with one of each an entry, of which the stores need 13).  So they are
// found for a few positions, and all others by one product of complex numbers,
//     turn(base + j) = turn(base) turn(j),
// four instructions and an error of at most 7 units of 2^-53: 13.4 us, 5.0 TB/s.  4096
// positions, 3.6 us, are too few for that.
#include <hip/hip_runtime.h>

#include "slora_device.h"
#include "slora_kv.h"

namespace slora {

constexpr int kRotSteps = 4;      // positions j of a thread
constexpr int kRotBases = 16;     // bases of a workgroup, at most

// Angles are held in turns: p * (hi + lo) of a position p below 2^31 leaves its
// whole turns exactly (the product's rounding error comes back from the fma, so
// nothing else may be fused with the product).  What far positions lose is the
// frequency's own error times p, 2^-59 p at most: frequencies are found in 64 bits of
// mantissa (about 6 units of 2^-64 of the exponentials, 6 of what follows them).
__device__ __forceinline__ void turn_of(double p, double hi, double lo, double* c, double* s) {
#pragma clang fp contract(off)
  const double whole = p * hi, rest = __builtin_fma(p, hi, -whole) + p * lo;
  sincospi(2. * ((whole - rint(whole)) + rest), s, c);
}

// A workgroup's threads are pairs by positions: `rows` of these side by side, which
// a thread passes in kRotSteps steps for each base, so that bases lie rows *
// kRotSteps apart.
__global__ __launch_bounds__(kThreads) void kv_rotary_kernel(KvRotary R) {
  __shared__ double2 base[kRotBases * 128];
  const int half = R.half, rows = kThreads / half, pair = threadIdx.x % half, j0 = threadIdx.x / half;
  const int step = rows * kRotSteps;
  const int64_t row0 = (int64_t)blockIdx.x * step * R.bases;
  if (R.bases == 1) {                                          // a short table: every position's own angle
    if (j0 < rows)
#pragma unroll
      for (int k = 0; k < kRotSteps; ++k) {
        const int64_t row = row0 + k * rows + j0;
        double c, s;
        turn_of((double)(R.first + row), R.turn_hi[pair], R.turn_lo[pair], &c, &s);
        if (row >= R.n) return;
        R.out[row * 2 * half + pair] = (float)(c * R.amplitude);
        R.out[(row * 2 + 1) * half + pair] = (float)(s * R.amplitude);
      }
    return;
  }
  if (j0 < rows) {
    const double hi = R.turn_hi[pair], lo = R.turn_lo[pair];
    for (int b = j0; b < R.bases; b += rows) {
      double c, s;
      turn_of((double)(R.first + row0 + (int64_t)b * step), hi, lo, &c, &s);
      base[b * half + pair] = make_double2(c * R.amplitude, s * R.amplitude);
    }
  }
  __syncthreads();
  if (j0 >= rows) return;
  double cj[kRotSteps], sj[kRotSteps];
#pragma unroll
  for (int k = 0; k < kRotSteps; ++k)
    turn_of((double)(j0 + k * rows), R.turn_hi[pair], R.turn_lo[pair], &cj[k], &sj[k]);
  for (int b = 0; b < R.bases; ++b) {
    const double2 z = base[b * half + pair];
#pragma unroll
    for (int k = 0; k < kRotSteps; ++k) {
      const int64_t row = row0 + (int64_t)b * step + k * rows + j0;
      if (row >= R.n) return;
      float* out = R.out + row * 2 * half + pair;
      out[0] = (float)(z.x * cj[k] - z.y * sj[k]);
      out[half] = (float)(z.y * cj[k] + z.x * sj[k]);
    }
  }
}

// Bases of a workgroup: what leaves about four workgroups a CU.
hipError_t launch_kv_rotary(const KvRotary& R0, hipStream_t stream) {
  KvRotary R = R0;
  const int64_t step = (int64_t)(kThreads / R.half) * kRotSteps;
  const int64_t want = R.n / (step * 4 * kKvCus);
  R.bases = (int32_t)(want < 1 ? 1 : want > kRotBases ? kRotBases : want);
  const int64_t blocks = (R.n + step * R.bases - 1) / (step * R.bases);
  if (blocks <= 0) return hipSuccess;
  void* args[] = {&R};
  return hipLaunchKernel((const void*)kv_rotary_kernel, dim3((unsigned)blocks), dim3(kThreads), args, 0, stream);
}

}  // namespace slora
