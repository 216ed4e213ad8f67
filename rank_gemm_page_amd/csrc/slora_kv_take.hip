// Sequences made of other sequences' tokens (include/slora.h, slora_kv_take):
// blocks written anew, and rows of the page table.
#include <hip/hip_runtime.h>

#include "slora_kv_device.h"

namespace slora {

constexpr int kTakeChunk = kThreads;   // tokens whose sources are in LDS at a time

// Where a quad of tokens' values come from: the words that hold its bytes (one
// where the quad is one of the source, two where it lies across two, up to four
// where tokens were left out), and which byte of words 0 and 1 and of words 2 and 3
// each token takes (0x0c: none).
struct Quad { const uint8_t* word[4]; uint32_t take01, take23, rest, words; };

// One block of one layer and kv head: its ranges are the largest of its tokens'
// old ones, and codes of smaller ranges are coded again.  Keys go in their 16-byte
// units, of one token each; a unit of values holds two elements of 8 tokens, in two
// quads, and is put together from the words that hold them: bytes one by one took
// 98 us instead of XX for 16007 tokens of 8 heads in 4 layers.
template <int CODE>
__device__ __forceinline__ void take_block(const KvTake& A, uint32_t at, int tid) {
  using C = Code<CODE>;
  __shared__ const uint8_t* lds_base[kTakeChunk];
  __shared__ int32_t lds_slot[kTakeChunk];
  __shared__ double lds_ratio[2][kTakeChunk];
  __shared__ Quad lds_quad[kTakeChunk / 4];
  __shared__ uint32_t lds_max[2][kThreads / 64];
  const KvView& kv = A.kv;
  const uint32_t per = (uint32_t)(kv.n_layers * kv.n_kv), c = at / per, x = at - c * per;
  const KvCopy copy = A.copies[c];
  const int32_t* row = kv_row(kv, copy.src, (int)(x / kv.n_kv), (int)(x % kv.n_kv));
  const int32_t* tokens = A.tokens + copy.at;
  const int32_t page = A.pages[at];
  const int dim = kv.dim, ush = 27 - __clz(dim);
  const int64_t vbase = (int64_t)kv.block * dim;
  uint8_t* out = (uint8_t*)kv.base + (int64_t)page * kv.page_bytes;

  // this thread's token of the first chunk, and the largest ranges of all
  int32_t from = 0;
  int slot = 0;
  uint32_t rk = 0, rv = 0, mk = 0, mv = 0;
  auto find = [&](int t) {
    const int token = tokens[t], block = (int)((uint32_t)token / (uint32_t)kv.block);
    from = row[block];
    slot = token - block * kv.block;
    const float2 r = *reinterpret_cast<const float2*>(kv.range + 2 * (int64_t)from);
    rk = __float_as_uint(r.x) & 0x7FFFFFFFu;
    rv = __float_as_uint(r.y) & 0x7FFFFFFFu;
  };
  for (int t = copy.count - 1 - (copy.count - 1 - tid) % kThreads; t >= tid && t < copy.count; t -= kThreads) {
    find(t);                                                   // the last one found is the first chunk's
    mk = max(mk, rk);
    mv = max(mv, rv);
  }
  mk = team_max(mk, lds_max[0]);
  mv = team_max(mv, lds_max[1]);
  const bool bad_k = mk >= 0x7F800000u, bad_v = mv >= 0x7F800000u;
  if (tid == 0) {
    float* r = kv.range + 2 * (int64_t)page;
    r[0] = bad_k ? __uint_as_float(0x7FC00000u) : __uint_as_float(mk);
    r[1] = bad_v ? __uint_as_float(0x7FC00000u) : __uint_as_float(mv);
  }
  const uint32_t none = C::kZero * 0x01010101u;
  for (int t0 = 0; t0 < copy.count; t0 += kTakeChunk) {
    const int n = min(kTakeChunk, copy.count - t0);
    if (t0 && tid < n) find(t0 + tid);
    if (tid < n) {
      lds_base[tid] = (const uint8_t*)kv.base + (int64_t)from * kv.page_bytes;
      lds_slot[tid] = slot;
    }
    lds_ratio[0][tid] = tid < n ? (double)__uint_as_float(rk) / (double)__uint_as_float(mk) : 1.;
    lds_ratio[1][tid] = tid < n ? (double)__uint_as_float(rv) / (double)__uint_as_float(mv) : 1.;
    const bool again_k = __syncthreads_or(tid < n && rk != mk && !bad_k);
    const bool again_v = __syncthreads_or(tid < n && rv != mv && !bad_v);
    if (tid * 4 < ((n + 31) & ~31)) {
      const uint8_t* last = nullptr;
      uint32_t words = 0, take01 = 0x0c0c0c0cu, take23 = 0x0c0c0c0cu, rest = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = tid * 4 + j;
        if (t >= n) {
          rest |= C::kZero << (8 * j);
          continue;
        }
        const int s = lds_slot[t];
        const uint8_t* p = lds_base[t] + vbase + (int64_t)(s >> 5) * 32 * dim + ((s & 15) >> 2) * 256 + ((s >> 4) & 1) * 4;
        if (p != last) lds_quad[tid].word[words++] = last = p; // (tokens ascend: a word is never met again)
        const uint32_t w = words - 1, byte = (s & 3) + 4 * (w & 1);
        const uint32_t one = (0x0cu ^ byte) << (8 * j);        // in the place of "none"
        take01 ^= w < 2 ? one : 0;
        take23 ^= w < 2 ? 0 : one;
      }
      lds_quad[tid].take01 = take01;
      lds_quad[tid].take23 = take23;
      lds_quad[tid].rest = rest;
      lds_quad[tid].words = words;
    }
    __syncthreads();
    const int units_k = n << ush, units_v = ((n + 31) >> 5) << (ush + 5);
    for (int u = tid; u < units_v; u += kThreads) {
      const int t = u >> ush, d = (u & ((1 << ush) - 1)) * 16;
      uint4 k = make_uint4(none, none, none, none);
      if (u < units_k && !bad_k) k = ld16(lds_base[t] + kv_k_byte(lds_slot[t], d, dim));

      const int group = u >> (ush + 5), e = (u >> 6) & ((1 << (ush - 1)) - 1), g = (u & 63) >> 4, i = u & 15;
      const int off = e * 1024 + i * 16;
      uint32_t v[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Quad& q = lds_quad[group * 8 + h * 4 + g];
        uint32_t w[2][4] = {};
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (m < (int)q.words && !bad_v) {
            w[0][m] = *reinterpret_cast<const uint32_t*>(q.word[m] + off);
            w[1][m] = *reinterpret_cast<const uint32_t*>(q.word[m] + off + 8);
          }
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          v[2 * o + h] = __builtin_amdgcn_perm(w[o][1], w[o][0], q.take01) |
                         __builtin_amdgcn_perm(w[o][3], w[o][2], q.take23) | q.rest;
          if (bad_v) v[2 * o + h] = none;
        }
      }
      if (again_k && u < units_k) k = again16<CODE>(k, lds_ratio[0][t]);
      if (again_v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const double* ratio = &lds_ratio[1][group * 32 + h * 16 + g * 4];
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            uint32_t y = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y |= C::nearest((double)C::value((v[2 * o + h] >> (8 * j)) & 0xFF) * ratio[j]) << (8 * j);
            v[2 * o + h] = y;
          }
        }
      }
      if (u < units_k) st16(out + kv_k_byte(t0 + t, d, dim), k);
      st16(out + vbase + (int64_t)(t0 >> 5) * 32 * dim + (int64_t)u * 16, make_uint4(v[0], v[1], v[2], v[3]));
    }
    if (t0 + kTakeChunk < copy.count) __syncthreads();
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
