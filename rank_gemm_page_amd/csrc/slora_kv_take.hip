// Sequences made of other sequences' tokens (include/slora.h, slora_kv_take):
// blocks written anew, and rows of the page table.
#include <hip/hip_runtime.h>

#include "slora_kv_device.h"

namespace slora {

constexpr int kTakeChunk = kThreads;   // tokens whose sources are in LDS at a time

// Where a quad of tokens' values come from: the words that hold its bytes (one
// where the quad is one of the source, two where it lies across two, up to four
// where tokens were left out; of one, the second is the first again), and which
// byte of words 0 and 1 and of words 2 and 3 each token takes (0x0c: none).
struct Quad { const uint8_t* word[4]; uint32_t take01, take23, rest, words; };

template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
  v = max(v, dpp<0xB1>(v));                                    // lane ^ 1, lane ^ 2, 7 - lane, 15 - lane
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  v = max(v, dpp<0x140>(v));
  const int x = (int)v;
  return max(max((uint32_t)__builtin_amdgcn_readlane(x, 0), (uint32_t)__builtin_amdgcn_readlane(x, 16)),
             max((uint32_t)__builtin_amdgcn_readlane(x, 32), (uint32_t)__builtin_amdgcn_readlane(x, 48)));
}

// One block of one layer and kv head: its ranges are the largest of its tokens'
// old ones, and codes of smaller ranges are coded again.  Keys go in their 16-byte
// units, of one token each; a unit of values holds two elements of 8 tokens, in two
// quads, and is put together from the words that hold them (byte by byte 16007
// tokens of 8 heads in 4 layers took 98 us).  A page is little work for a workgroup,
// so what comes before the copy counts: every wave finds the ranges of all tokens by
// itself, and there is one barrier (with reductions over the workgroup and ten
// barriers 69 us).
//
// What bounds it: the copy itself.  Those tokens take 65 us, 4.0 TB/s of the bytes
// that the counters see (a large copy reaches 5.2); half the tokens of 16
// conversations in runs of three, 8 heads in 2 layers, 65 us at 3.5 TB/s, where most
// of the lines that are read hold tokens that are left out.  Two units a thread at a
// time (94 registers) took 82 us instead of 74, the units loaded before the ranges
// are found 73 instead of 65.
template <int CODE, int DIM>
__device__ __forceinline__ void take_block(const KvTake& A, uint32_t at, int tid) {
  using C = Code<CODE>;
  constexpr int KU = DIM / 16, VU = 2 * DIM;                   // units of a key, and of 32 tokens' values
  __shared__ const uint8_t* lds_base[kTakeChunk];
  __shared__ int32_t lds_slot[kTakeChunk];
  __shared__ double lds_ratio[2][kTakeChunk];
  __shared__ Quad lds_quad[kTakeChunk / 4];
  const KvView& kv = A.kv;
  const uint32_t per = (uint32_t)(kv.n_layers * kv.n_kv), c = at / per, x = at - c * per;
  const KvCopy copy = A.copies[c];
  const int32_t* row = kv_row(kv, copy.src, (int)(x / kv.n_kv), (int)(x % kv.n_kv));
  const int32_t* tokens = A.tokens + copy.at;
  const int32_t page = A.pages[at];
  const int lane = tid & 63, wave = tid >> 6;
  const int64_t vbase = (int64_t)kv.block * DIM;
  uint8_t* out = (uint8_t*)kv.base + (int64_t)page * kv.page_bytes;

  struct Source { int32_t page, slot; uint32_t rk, rv; };
  auto find = [&](int t) {
    const int token = tokens[t], block = (int)((uint32_t)token / (uint32_t)kv.block);
    const int32_t from = row[block];
    const float2 r = *reinterpret_cast<const float2*>(kv.range + 2 * (int64_t)from);
    return Source{from, token - block * kv.block, __float_as_uint(r.x) & 0x7FFFFFFFu,
                  __float_as_uint(r.y) & 0x7FFFFFFFu};
  };
  Source mine = {0, 0, 0, 0};                                  // of token tid
  uint32_t mk = 0, mv = 0, nk = 0, nv = 0;                     // largest, and largest of what the smallest leaves
  for (int t0 = 0; t0 < copy.count; t0 += 64)
    if (t0 + lane < copy.count) {
      const Source s = find(t0 + lane);
      mk = max(mk, s.rk);
      mv = max(mv, s.rv);
      nk = max(nk, ~s.rk);
      nv = max(nv, ~s.rv);
      if (t0 == wave * 64) mine = s;
    }
  mk = wave_most(mk);
  mv = wave_most(mv);
  nk = wave_most(nk);
  nv = wave_most(nv);
  const bool bad_k = mk >= 0x7F800000u, bad_v = mv >= 0x7F800000u;
  const bool again_k = !bad_k && mk != ~nk, again_v = !bad_v && mv != ~nv;
  if (tid == 0)
    *reinterpret_cast<float2*>(kv.range + 2 * (int64_t)page) =
        make_float2(__uint_as_float(bad_k ? 0x7FC00000u : mk), __uint_as_float(bad_v ? 0x7FC00000u : mv));
  constexpr uint32_t kNone = C::kZero * 0x01010101u;

  for (int t0 = 0; t0 < copy.count; t0 += kTakeChunk) {
    const int n = min(kTakeChunk, copy.count - t0);
    if (t0) {
      __syncthreads();                                         // the last chunk's are no longer read
      if (tid < n) mine = find(t0 + tid);
    }
    if (wave * 64 < ((n + 31) & ~31)) {
      const uint8_t* base = (const uint8_t*)kv.base + (int64_t)mine.page * kv.page_bytes;
      lds_base[tid] = base;
      lds_slot[tid] = mine.slot;
      if (again_k) lds_ratio[0][tid] = tid < n ? (double)__uint_as_float(mine.rk) / (double)__uint_as_float(mk) : 1.;
      if (again_v) lds_ratio[1][tid] = tid < n ? (double)__uint_as_float(mine.rv) / (double)__uint_as_float(mv) : 1.;
      // the quad's four tokens are in neighbouring lanes
      const int s = mine.slot;
      const uint64_t p = reinterpret_cast<uint64_t>(base) + vbase + (s >> 5) * 32 * DIM + ((s & 15) >> 2) * 256 +
                         ((s >> 4) & 1) * 4;
      const uint32_t lo = (uint32_t)p, hi = (uint32_t)(p >> 32);
      const uint32_t ps[4][3] = {{dpp<0x00>(lo), dpp<0x00>(hi), dpp<0x00>(s)},
                                 {dpp<0x55>(lo), dpp<0x55>(hi), dpp<0x55>(s)},
                                 {dpp<0xAA>(lo), dpp<0xAA>(hi), dpp<0xAA>(s)},
                                 {dpp<0xFF>(lo), dpp<0xFF>(hi), dpp<0xFF>(s)}};
      if ((tid & 3) == 0) {
        Quad& q = lds_quad[tid >> 2];
        uint64_t last = 0;
        uint32_t words = 0, take01 = 0x0c0c0c0cu, take23 = 0x0c0c0c0cu, rest = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t pj = (uint64_t)ps[j][1] << 32 | ps[j][0];
          if (tid + j >= n) {
            rest |= C::kZero << (8 * j);
          } else {
            // (tokens ascend: no word comes again)
            if (pj != last) q.word[words++] = reinterpret_cast<const uint8_t*>(pj);
            last = pj;
            const uint32_t w = words - 1, byte = (ps[j][2] & 3) + 4 * (w & 1);
            const uint32_t one = (0x0cu ^ byte) << (8 * j);    // in the place of "none"
            take01 ^= w < 2 ? one : 0;
            take23 ^= w < 2 ? 0 : one;
          }
        }
        if (words < 2) q.word[1] = words ? reinterpret_cast<const uint8_t*>(last) : base;
        if (words == 0) q.word[0] = base;                      // (a quad behind the last token: any page's)
        q.take01 = take01;
        q.take23 = take23;
        q.rest = rest;
        q.words = words;
      }
    }
    __syncthreads();
    const int units_k = n * KU, units_v = ((n + 31) >> 5) * VU;
    for (int u = tid; u < units_v; u += kThreads) {
      const int t = u / KU, d = u % KU * 16, group = u / VU, e = u % VU / 64, g = (u & 63) >> 4, i = u & 15;
      uint4 k = make_uint4(kNone, kNone, kNone, kNone);
      if (u < units_k) k = ld16(lds_base[t] + kv_k_byte(lds_slot[t], d, DIM));
      const int off = e * 1024 + i * 16;
      uint32_t v[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Quad& q = lds_quad[group * 8 + h * 4 + g];
        const uint8_t *p0 = q.word[0] + off, *p1 = q.word[1] + off;
        const uint32_t a0 = *reinterpret_cast<const uint32_t*>(p0), b0 = *reinterpret_cast<const uint32_t*>(p0 + 8);
        const uint32_t a1 = *reinterpret_cast<const uint32_t*>(p1), b1 = *reinterpret_cast<const uint32_t*>(p1 + 8);
        v[h] = __builtin_amdgcn_perm(a1, a0, q.take01) | q.rest;
        v[2 + h] = __builtin_amdgcn_perm(b1, b0, q.take01) | q.rest;
        if (q.words > 2) {
          const uint8_t *p2 = q.word[2] + off, *p3 = q.words > 3 ? q.word[3] + off : p2;
          const uint32_t a2 = *reinterpret_cast<const uint32_t*>(p2), b2 = *reinterpret_cast<const uint32_t*>(p2 + 8);
          const uint32_t a3 = *reinterpret_cast<const uint32_t*>(p3), b3 = *reinterpret_cast<const uint32_t*>(p3 + 8);
          v[h] |= __builtin_amdgcn_perm(a3, a2, q.take23);
          v[2 + h] |= __builtin_amdgcn_perm(b3, b2, q.take23);
        }
      }
      if (again_k && u < units_k) {
        const double ratio = lds_ratio[0][t];
        if (ratio != 1.) k = again16<CODE>(k, ratio);
      }
      if (again_v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const double* r = &lds_ratio[1][group * 32 + h * 16 + g * 4];
          const double r0 = r[0], r1 = r[1], r2 = r[2], r3 = r[3];
          if (r0 != 1. || r1 != 1. || r2 != 1. || r3 != 1.) {
            v[h] = Again<CODE>::four(v[h], r0, r1, r2, r3);
            v[2 + h] = Again<CODE>::four(v[2 + h], r0, r1, r2, r3);
          }
        }
      }
      if (bad_k) k = make_uint4(kNone, kNone, kNone, kNone);
      if (bad_v) v[0] = v[1] = v[2] = v[3] = kNone;
      if (u < units_k) st16(out + kv_k_byte(t0 + t, d, DIM), k);
      st16(out + vbase + (int64_t)(t0 >> 5) * 32 * DIM + (int64_t)u * 16, make_uint4(v[0], v[1], v[2], v[3]));
    }
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

template <int CODE, int DIM>
__global__ __launch_bounds__(kThreads) void kv_take_kernel(KvTake A) {
  const int64_t copies = (int64_t)A.n_copies * A.kv.n_layers * A.kv.n_kv, at = A.first + blockIdx.x;
  if (at < copies) take_block<CODE, DIM>(A, (uint32_t)at, threadIdx.x);
  else take_rows(A, (at - copies) * (kThreads / 64) + (threadIdx.x >> 6), threadIdx.x & 63);
}

template <int CODE>
static const void* take_of(int dim) {
  return dim == 64 ? (const void*)kv_take_kernel<CODE, 64>
         : dim == 128 ? (const void*)kv_take_kernel<CODE, 128> : (const void*)kv_take_kernel<CODE, 256>;
}

hipError_t launch_kv_take(const KvTake& A0, bool in_place, hipStream_t stream) {
  KvTake A = A0;
  const int64_t per = (int64_t)A.kv.n_layers * A.kv.n_kv, copies = A.n_copies * per;
  const int64_t all = copies + (A.n_rows * per + kThreads / 64 - 1) / (kThreads / 64);
  const void* kernel = A.kv.code == SLORA_KV_INT8 ? take_of<SLORA_KV_INT8>(A.kv.dim) : take_of<SLORA_KV_FP8>(A.kv.dim);
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
