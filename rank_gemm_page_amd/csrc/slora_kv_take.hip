// Sequences made of other sequences' tokens (include/slora.h, slora_kv_take):
// blocks written anew, and rows of the page table.
#include <hip/hip_runtime.h>

#include "slora_kv_device.h"

namespace slora {

constexpr int kTakeChunk = 128;   // tokens whose sources are kept in LDS at a time

// One block of one layer and kv head: its ranges are the largest of its tokens'
// old ones, and codes of smaller ranges are coded again.
template <int CODE>
__device__ __forceinline__ void take_block(const KvTake& A, uint32_t at, int tid) {
  using C = Code<CODE>;
  __shared__ const uint8_t* lds_base[kTakeChunk];
  __shared__ int32_t lds_slot[kTakeChunk];
  __shared__ double lds_ratio[2][kTakeChunk];
  __shared__ uint32_t lds_max[2][kThreads / 64];
  const KvView& kv = A.kv;
  const uint32_t per = (uint32_t)(kv.n_layers * kv.n_kv), c = at / per, x = at - c * per;
  const KvCopy copy = A.copies[c];
  const int32_t* row = kv_row(kv, copy.src, (int)(x / kv.n_kv), (int)(x % kv.n_kv));
  const int32_t* tokens = A.tokens + copy.at;
  const int32_t page = A.pages[at];
  uint8_t* kout = (uint8_t*)kv.base + (int64_t)page * kv.page_bytes;
  uint8_t* vout = kout + (int64_t)kv.block * kv.dim;
  const int dim = kv.dim, ush = 27 - __clz(dim);

  uint32_t mk = 0, mv = 0;
  for (int t = tid; t < copy.count; t += kThreads) {
    const float* r = kv.range + 2 * (int64_t)row[tokens[t] / kv.block];
    mk = max(mk, __float_as_uint(r[0]) & 0x7FFFFFFFu);
    mv = max(mv, __float_as_uint(r[1]) & 0x7FFFFFFFu);
  }
  mk = team_max(mk, lds_max[0]);
  mv = team_max(mv, lds_max[1]);
  const bool bad_k = mk >= 0x7F800000u, bad_v = mv >= 0x7F800000u;
  if (tid == 0) {
    float* r = kv.range + 2 * (int64_t)page;
    r[0] = bad_k ? __uint_as_float(0x7FC00000u) : __uint_as_float(mk);
    r[1] = bad_v ? __uint_as_float(0x7FC00000u) : __uint_as_float(mv);
  }
  for (int t0 = 0; t0 < copy.count; t0 += kTakeChunk) {
    const int n = min(kTakeChunk, copy.count - t0);
    if (tid < n) {
      const int token = tokens[t0 + tid], block = token / kv.block;
      const int32_t from = row[block];
      const float* r = kv.range + 2 * (int64_t)from;
      lds_base[tid] = (const uint8_t*)kv.base + (int64_t)from * kv.page_bytes;
      lds_slot[tid] = token - block * kv.block;
      lds_ratio[0][tid] = mk ? (double)fabsf(r[0]) / (double)__uint_as_float(mk) : 1.;
      lds_ratio[1][tid] = mv ? (double)fabsf(r[1]) / (double)__uint_as_float(mv) : 1.;
    }
    __syncthreads();
    for (int u = tid; u < n << ush; u += kThreads) {
      const int t = u >> ush, d = (u & ((1 << ush) - 1)) * 16;
      uint4 w = ld16(lds_base[t] + kv_k_byte(lds_slot[t], d, dim));
      const double ratio = lds_ratio[0][t];
      if (ratio != 1. && !bad_k) w = again16<CODE>(w, ratio);
      if (bad_k) w = make_uint4(C::kZero * 0x01010101u, C::kZero * 0x01010101u, C::kZero * 0x01010101u,
                                C::kZero * 0x01010101u);
      st16(kout + kv_k_byte(t0 + t, d, dim), w);
    }
    const int groups = (n + 31) >> 5;
    for (int u = tid; u < groups << (ush + 5); u += kThreads) {
      const int group = u >> (ush + 5), e = (u >> 6) & ((1 << (ush - 1)) - 1), g = (u & 63) >> 4, i = u & 15;
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = group * 32 + (j >> 2) * 16 + g * 4 + (j & 3);
        uint32_t c0 = C::kZero, c1 = C::kZero;
        if (t < n && !bad_v) {
          const int slot = lds_slot[t];
          const uint8_t* p = lds_base[t] + (int64_t)kv.block * dim + (int64_t)(slot >> 5) * 32 * dim + e * 1024 +
                             (((slot & 15) >> 2) * 16 + i) * 16 + ((slot >> 4) & 1) * 4 + (slot & 3);
          c0 = p[0];
          c1 = p[8];
          const double ratio = lds_ratio[1][t];
          if (ratio != 1.) {
            c0 = C::nearest((double)C::value(c0) * ratio);
            c1 = C::nearest((double)C::value(c1) * ratio);
          }
        }
        w[j >> 2] |= c0 << (8 * (j & 3));
        w[2 + (j >> 2)] |= c1 << (8 * (j & 3));
      }
      st16(vout + (int64_t)(t0 >> 5) * 32 * dim + (int64_t)u * 16, make_uint4(w[0], w[1], w[2], w[3]));
    }
    __syncthreads();
  }
}

// Page table rows, a wave each.  In place a row's entries only move towards its
// start: the 64 that a wave reads are never before those that it writes.
__device__ __forceinline__ void take_rows(const KvTake& A, int64_t wave, int lane) {
  const KvView& kv = A.kv;
  const int64_t per = (int64_t)kv.n_layers * kv.n_kv;
  if (wave >= A.n_rows * per) return;
  const KvTakeRow r = A.rows[wave / per];
  const int64_t x = wave % per;
  const int32_t* from = kv.table + (r.src * per + x) * kv.max_blocks;
  int32_t* to = const_cast<int32_t*>(kv.table) + (r.dst * per + x) * kv.max_blocks + r.first;
  for (int b0 = 0; b0 < r.n; b0 += 64) {
    const int b = b0 + lane;
    int32_t page = 0;
    if (b < r.n) {
      const int32_t e = A.entries[r.at + b];
      page = e >= 0 ? from[e] : A.pages[~e * per + x];
    }
    if (b < r.n) to[b] = page;
  }
}

template <int CODE>
__global__ __launch_bounds__(kThreads) void kv_take_kernel(KvTake A) {
  const int64_t copies = (int64_t)A.n_copies * A.kv.n_layers * A.kv.n_kv, at = A.first + blockIdx.x;
  if (at < copies) take_block<CODE>(A, (uint32_t)at, threadIdx.x);
  else take_rows(A, (at - copies) * (kThreads / 64) + (threadIdx.x >> 6), threadIdx.x & 63);
}

hipError_t launch_kv_take(const KvTake& A0, bool in_place, hipStream_t stream) {
  KvTake A = A0;
  const int64_t per = (int64_t)A.kv.n_layers * A.kv.n_kv, copies = A.n_copies * per;
  const int64_t all = copies + (A.n_rows * per + kThreads / 64 - 1) / (kThreads / 64);
  const void* kernel = A.kv.code == SLORA_KV_INT8 ? (const void*)kv_take_kernel<SLORA_KV_INT8>
                                                  : (const void*)kv_take_kernel<SLORA_KV_FP8>;
  // copies find their sources through rows that in place are written: these go second
  const int64_t ends[] = {in_place ? copies : all, all};
  for (int64_t end : ends) {
    if (end <= A.first) continue;
    void* args[] = {&A};
    const hipError_t e =
        hipLaunchKernel(kernel, dim3((unsigned)(end - A.first)), dim3(kThreads), args, 0, stream);
    if (e != hipSuccess) return e;
    A.first = end;
  }
  return hipSuccess;
}

}  // namespace slora
