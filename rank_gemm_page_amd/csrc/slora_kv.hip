// Kernels of the 8-bit paged KV cache (include/slora.h, "KV cache in the
// pool"): append with the rotation by positions, attention over the cached
// blocks, and reading blocks back.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "slora_device.h"
#include "slora_kv.h"

namespace slora {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float8v __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Codes.  An int8 code c is kept as the byte c + 128: the byte with 0x64 above
// it is the fp16 number 1024 + c + 128, so two codes become fp16 with one byte
// permute and one packed subtraction.  An e4m3 code is its byte.

template <int CODE> struct Code;

template <> struct Code<SLORA_KV_INT8> {
  static constexpr float kTop = 127.f;
  static constexpr uint32_t kZero = 0x80;
  static __device__ __forceinline__ half8 halves(uint32_t a, uint32_t b) {
    const half2v bias = {(_Float16)1152.f, (_Float16)1152.f};
    union { uint32_t u; half2v h; } p[4];
    p[0].u = __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u);
    p[1].u = __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u);
    p[2].u = __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u);
    p[3].u = __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u);
    half8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2v h = p[i].h - bias;
      r[2 * i] = h[0];
      r[2 * i + 1] = h[1];
    }
    return r;
  }
  static __device__ __forceinline__ float value(uint32_t byte) { return (float)(int)byte - 128.f; }
  static __device__ __forceinline__ uint32_t nearest(double x) { return (uint32_t)((int)__builtin_rint(x) + 128) & 0xFF; }
};

template <> struct Code<SLORA_KV_FP8> {
  static constexpr float kTop = 448.f;
  static constexpr uint32_t kZero = 0;
  static __device__ __forceinline__ half8 halves(uint32_t a, uint32_t b) {
    const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
    const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
    const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
    const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
    return half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  static __device__ __forceinline__ float value(uint32_t byte) {
    return __builtin_amdgcn_cvt_pk_f32_fp8((int)byte, false)[0];
  }
  // The definition rounds the 64-bit product to fp32 and then to e4m3.
  static __device__ __forceinline__ uint32_t nearest(double x) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32((float)x, 0.f, 0, false) & 0xFF;
  }
};

template <int CODE>
__device__ __forceinline__ float8v floats8(uint32_t a, uint32_t b) {
  float8v r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = Code<CODE>::value((a >> (8 * i)) & 0xFF);
    r[4 + i] = Code<CODE>::value((b >> (8 * i)) & 0xFF);
  }
  return r;
}

// Row stride of the page table per (sequence, layer, head), 64-bit.
__device__ __forceinline__ const int32_t* kv_row(const KvView& kv, int seq, int layer, int head) {
  return kv.table + (((int64_t)seq * kv.n_layers + layer) * kv.n_kv + head) * kv.max_blocks;
}

// ---------------------------------------------------------------------------
// Page table entries of a step's new blocks.

__global__ __launch_bounds__(kThreads) void kv_patch_kernel(int32_t* table, const KvPatch* patches, int32_t n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < n) table[((int64_t)patches[i].hi << 32) | patches[i].lo] = patches[i].page;
}

// ---------------------------------------------------------------------------
// Append.

// Element d of a row rotated by the angles cs (cosines, then sines): products
// of an fp16 or fp32 element and an fp32 cosine are exact in 64 bits, so the
// result is rounded once whether or not the compiler fuses them.
template <typename T>
__device__ __forceinline__ double rotated(const T* row, const float* cs, int d, int rot, int pairs) {
  const double x = (double)(float)row[d];
  if (d >= rot) return x;
  const int half = rot >> 1;
  int i, o;
  bool second;
  if (pairs == SLORA_KV_HALVES) {
    second = d >= half;
    i = second ? d - half : d;
    o = second ? i : d + half;
  } else {
    second = d & 1;
    i = d >> 1;
    o = d ^ 1;
  }
  const double c = cs[i], s = cs[half + i], y = (double)(float)row[o];
  return second ? x * c + y * s : x * c - y * s;
}

// Largest of the workgroup's values (bit patterns of non-negative floats order
// as integers, with infinities and NaN above every finite one).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = max(v, lds[w]);
  __syncthreads();
  return v;
}

__device__ __forceinline__ uint32_t magnitude(double x) { return __float_as_uint(fabsf((float)x)); }

// One workgroup per touched block and kv head: the largest magnitudes of the
// block's new keys and values, then the codes, 16 bytes of the page layout a
// thread.  Workgroups behind those rotate q, 16 elements a thread.
template <typename T, int CODE>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppend A) {
  using C = Code<CODE>;
  const KvView& kv = A.kv;
  const int dim = kv.dim, tid = threadIdx.x;
  __shared__ uint32_t lds[kThreads / 64];
  const int64_t stores = (int64_t)A.n_blocks * kv.n_kv;
  if (blockIdx.x >= stores) {
    // units of 16 elements: 8 pairs of the rotated part, or 16 elements behind it
    const int per = dim / 16;
    const int64_t u = (blockIdx.x - stores) * kThreads + tid;
    const int64_t head = u / per;
    const int unit = (int)(u % per), row = (int)(head / kv.n_heads), h = (int)(head % kv.n_heads);
    if (row >= A.n_rows) return;
    const T* x = (const T*)A.q + row * A.q_stride + h * dim;
    T* y = (T*)A.q_out + row * A.q_out_stride + h * dim;
    const float* cs = A.cos_sin + (int64_t)A.row_pos[row] * kv.rot;
    const int half = kv.rot >> 1;
    double r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int d = unit * 16 >= kv.rot ? unit * 16 + j
                    : kv.pairs == SLORA_KV_HALVES ? (j < 8 ? unit * 8 + j : half + unit * 8 + j - 8) : unit * 16 + j;
      r[j] = rotated(x, cs, d, kv.rot, kv.pairs);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int d = unit * 16 >= kv.rot ? unit * 16 + j
                    : kv.pairs == SLORA_KV_HALVES ? (j < 8 ? unit * 8 + j : half + unit * 8 + j - 8) : unit * 16 + j;
      y[d] = (T)r[j];
    }
    return;
  }
  const KvBlock blk = A.blocks[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const KvSeq sq = A.seqs[blk.s];
  const int32_t page = kv_row(kv, sq.seq, A.layer, head)[blk.block];
  char* kbase = kv.base + (int64_t)page * kv.page_bytes;
  char* vbase = kbase + (int64_t)kv.block * dim;
  float* range = kv.range + 2 * (int64_t)page;
  const int pos0 = blk.block * kv.block;                       // position of slot 0
  const int64_t row0 = (int64_t)sq.row0 + pos0 - sq.start;     // batch row of slot 0 (negative before the first new slot)
  const int count = blk.slot1 - blk.slot0;
  const T* kin = (const T*)A.k + (int64_t)head * dim;
  const T* vin = (const T*)A.v + (int64_t)head * dim;

  uint32_t mk = 0, mv = 0;
  for (int i = tid; i < count * dim; i += kThreads) {
    const int slot = blk.slot0 + i / dim, d = i % dim;
    const T* krow = kin + (row0 + slot) * A.k_stride;
    mk = max(mk, magnitude(rotated(krow, A.cos_sin + (int64_t)(pos0 + slot) * kv.rot, d, kv.rot, kv.pairs)));
    mv = max(mv, magnitude((double)(float)vin[(row0 + slot) * A.v_stride + d]));
  }
  mk = block_max(mk, lds);
  mv = block_max(mv, lds);
  const uint32_t held_k = blk.slot0 ? __float_as_uint(range[0]) & 0x7FFFFFFFu : 0;
  const uint32_t held_v = blk.slot0 ? __float_as_uint(range[1]) & 0x7FFFFFFFu : 0;
  __syncthreads();
  mk = max(mk, held_k);
  mv = max(mv, held_v);
  const bool bad_k = mk >= 0x7F800000u, bad_v = mv >= 0x7F800000u;
  if (tid == 0) {
    range[0] = bad_k ? __uint_as_float(0x7FC00000u) : __uint_as_float(mk);
    range[1] = bad_v ? __uint_as_float(0x7FC00000u) : __uint_as_float(mv);
  }
  const double new_k = __uint_as_float(mk), new_v = __uint_as_float(mv);
  const double inv_k = mk ? (double)C::kTop / new_k : 0., inv_v = mv ? (double)C::kTop / new_v : 0.;
  const double again_k = mk ? (double)__uint_as_float(held_k) / new_k : 0.;
  const double again_v = mv ? (double)__uint_as_float(held_v) / new_v : 0.;

  // keys: a 16-byte unit is 16 elements of one slot
  const int first_k = mk != held_k ? 0 : blk.slot0;
  for (int u = tid; u < (blk.slot1 - first_k) * (dim / 16); u += kThreads) {
    const int slot = first_k + u / (dim / 16), d0 = u % (dim / 16) * 16;
    uint8_t* at = (uint8_t*)kbase + kv_k_byte(slot, d0, dim);
    uint32_t w[4] = {0, 0, 0, 0};
    if (slot >= blk.slot0) {
      const T* krow = kin + (row0 + slot) * A.k_stride;
      const float* cs = A.cos_sin + (int64_t)(pos0 + slot) * kv.rot;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j >> 2] |= (bad_k ? C::kZero : C::nearest(rotated(krow, cs, d0 + j, kv.rot, kv.pairs) * inv_k)) << (8 * (j & 3));
    } else {
      const uint4 old = ld16(at);
      const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j >> 2] |= (bad_k ? C::kZero : C::nearest((double)C::value((o[j >> 2] >> (8 * (j & 3))) & 0xFF) * again_k))
                     << (8 * (j & 3));
    }
    st16(at, make_uint4(w[0], w[1], w[2], w[3]));
  }
  // values: a 16-byte unit is 2 elements of 8 slots
  const int first_v = (mv != held_v ? 0 : blk.slot0) / 32;
  const int groups = (blk.slot1 + 31) / 32 - first_v;
  for (int u = tid; u < groups * dim * 2; u += kThreads) {
    const int group = first_v + u / (dim * 2), lane = u % 64, e = u % (dim * 2) / 64;
    const int g = lane >> 4, i = lane & 15;
    uint8_t* at = (uint8_t*)vbase + (int64_t)group * 32 * dim + e * 1024 + lane * 16;
    const uint4 old = ld16(at);
    const uint32_t o[4] = {old.x, old.y, old.z, old.w};
    uint32_t w[4];
    bool any = false;
#pragma unroll
    for (int b = 0; b < 16; ++b) {
      const int j = b & 7, d = e * 32 + (b >> 3) * 16 + i;
      const int slot = group * 32 + (j >> 2) * 16 + g * 4 + (j & 3);
      uint32_t byte = (o[b >> 2] >> (8 * (b & 3))) & 0xFF;
      if (slot >= blk.slot0 && slot < blk.slot1) {
        any = true;
        byte = bad_v ? C::kZero : C::nearest((double)(float)vin[(row0 + slot) * A.v_stride + d] * inv_v);
      } else if (slot < blk.slot0 && mv != held_v) {
        any = true;
        byte = bad_v ? C::kZero : C::nearest((double)C::value(byte) * again_v);
      }
      w[b >> 2] = (b & 3 ? w[b >> 2] : 0) | byte << (8 * (b & 3));
    }
    if (any) st16(at, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// ---------------------------------------------------------------------------
// Attention of 16 query rows (row r of a sequence and kv head is query head
// r % G of token r / G, G = query heads per kv head) over a range of keys.
//
// Per 32 keys: S^T = K Q^T, two 16x16 tiles whose rows are keys and columns
// query rows, then the softmax weights, which lane (g, i) holds for query row
// i and the 8 keys that the page layout puts in its 16 bytes of V, so they are
// the second operand of O^T += V^T P^T without leaving their registers.  The
// four waves of a workgroup take consecutive quarters of the keys and join
// through LDS at the end.

template <typename T> struct Frag;
template <> struct Frag<_Float16> { typedef half8 type; };
template <> struct Frag<float> { typedef float8v type; };

template <int CODE>
__device__ __forceinline__ void codes8(uint32_t a, uint32_t b, half8* r) { *r = Code<CODE>::halves(a, b); }
template <int CODE>
__device__ __forceinline__ void codes8(uint32_t a, uint32_t b, float8v* r) { *r = floats8<CODE>(a, b); }

__device__ __forceinline__ float4v mma(half8 a, half8 b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// fp32: the same 8 products a lane as eight 16x16x4 instructions.
__device__ __forceinline__ float4v mma(float8v a, float8v b, float4v c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ half8 frag8(const float* p, half8*) {
  half8 r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = (_Float16)p[j];
  return r;
}
__device__ __forceinline__ float8v frag8(const float* p, float8v*) {
  float8v r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = p[j];
  return r;
}

// The softmax's reference is raised only when some score passes it by more
// than this (weights stay below 2^8, far inside fp16): most steps then need no
// reduction across lanes and no rescaling of the sums.
constexpr float kLazy = 8.f;

template <typename T, int CODE, int D>
__global__ __launch_bounds__(kThreads) void kv_attend_rows_kernel(KvAttend A) {
  using F = typename Frag<T>::type;
  constexpr int NC = D / 64, NE = D / 32, NT = D / 16;
  constexpr int DC = D < 128 ? D : 128;          // columns joined at a time
  __shared__ float lds_o[4][kKvRows][DC + 4];
  __shared__ float lds_ml[4][kKvRows][2];
  __shared__ float lds_ref[4];
  const KvView& kv = A.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), i = lane & 15, g = lane >> 4;
  const KvTile tile = A.tiles[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const KvSeq sq = A.seqs[tile.s];
  const int G = kv.n_heads / kv.n_kv, packed = sq.rows * G;

  // this lane's query row (rows past the last one repeat it and are not stored)
  const int r = min(tile.tile * kKvRows + i, packed - 1);
  const int t = r / G, pos = sq.start + t;
  const int lo = A.window ? max(0, pos - A.window + 1) : 0;
  const int t_first = tile.tile * kKvRows / G, t_last = (min(tile.tile * kKvRows + kKvRows, packed) - 1) / G;
  const int pos_first = sq.start + t_first, pos_last = sq.start + t_last, len = sq.start + sq.rows;
  const int tile_lo = A.window ? max(0, pos_first - A.window + 1) : 0;
  const int all_lo = A.window ? max(0, pos_last - A.window + 1) : 0;

  F qf[2 * NC];
  {
    const T* q = (const T*)A.q + (int64_t)(sq.row0 + t) * A.q_stride + (head * G + r % G) * D;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 2; ++s) qf[2 * c + s] = *(const F*)(q + c * 64 + g * 16 + s * 8);
  }

  // groups of 32 keys of this tile, of this split, of this wave
  const int first = tile_lo / kKvGroup, last = pos_last / kKvGroup + 1;
  const int per = (last - first + tile.splits - 1) / tile.splits;
  const int s_lo = first + tile.split * per, s_hi = min(last, s_lo + per);
  const int per_wave = (max(0, s_hi - s_lo) + 3) / 4;
  int gi = uni(s_lo + wave * per_wave);
  const int ge = uni(min(s_hi, gi + per_wave));

  const int32_t* row = kv_row(kv, sq.seq, A.layer, head);
  const int nb = kv.block / kKvGroup;
  float4v acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = float4v{0.f, 0.f, 0.f, 0.f};
  float m = -FLT_MAX, l = 0.f, ref = 0.f;

  int b = gi / nb, sub = gi - b * nb;
  uint4 kf[2 * NC], vf[NE];
  float rk = 0.f, rv = 0.f;
  auto load = [&](uint4* kx, uint4* vx, float& xk, float& xv) {
    const int32_t page = uni(row[b]);
    const char* kb = kv.base + (int64_t)page * kv.page_bytes + (int64_t)sub * kKvGroup * D;
    const char* vb = kb + (int64_t)kv.block * D;
#pragma unroll
    for (int n = 0; n < 2 * NC; ++n) kx[n] = ld16(kb + n * 1024 + i * 64 + g * 16);
#pragma unroll
    for (int e = 0; e < NE; ++e) vx[e] = ld16(vb + e * 1024 + lane * 16);
    xk = kv.range[2 * (int64_t)page];
    xv = kv.range[2 * (int64_t)page + 1];
    if (++sub == nb) { sub = 0; ++b; }
  };
  if (gi < ge) load(kf, vf, rk, rv);
  for (; gi < ge; ++gi) {
    uint4 kn[2 * NC], vn[NE];
    float rkn = 0.f, rvn = 0.f;
    if (gi + 1 < ge) load(kn, vn, rkn, rvn);
    const int key0 = gi * kKvGroup;

    float4v s0 = {0.f, 0.f, 0.f, 0.f}, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F a;
      codes8<CODE>(kf[c].x, kf[c].y, &a);
      s0 = mma(a, qf[2 * c], s0);
      codes8<CODE>(kf[c].z, kf[c].w, &a);
      s0 = mma(a, qf[2 * c + 1], s0);
      codes8<CODE>(kf[NC + c].x, kf[NC + c].y, &a);
      s1 = mma(a, qf[2 * c], s1);
      codes8<CODE>(kf[NC + c].z, kf[NC + c].w, &a);
      s1 = mma(a, qf[2 * c + 1], s1);
    }
    const float ck = rk / Code<CODE>::kTop * A.scale_log2;
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) { x[j] = s0[j] * ck; x[4 + j] = s1[j] * ck; }
    // keys behind the sequence hold anything: their scores are replaced, and
    // their e4m3 bytes, which may be NaN, are cleared
    bool seen = true;
    if (key0 + kKvGroup - 1 > pos_first || key0 < all_lo) {
      seen = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + (j >> 2) * 16 + g * 4 + (j & 3);
        const bool in = key <= pos && key >= lo;
        x[j] = in ? x[j] : -INFINITY;
        seen |= in;
      }
      if (CODE == SLORA_KV_FP8 && key0 + kKvGroup > len) {
        uint32_t keep[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (key0 + (j >> 2) * 16 + g * 4 + (j & 3) < len) keep[j >> 2] |= 0xFFu << (8 * (j & 3));
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          vf[e].x &= keep[0];
          vf[e].y &= keep[1];
          vf[e].z &= keep[0];
          vf[e].w &= keep[1];
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
    if (__any(top > m + kLazy)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n] *= f;
    }
    // values of a block count in units of its range: the sums are kept in
    // units of a reference range, replaced when a block's is far from it
    float unit = 1.f;
    if (rv > 0.f) {
      unit = rv / ref;
      if (!(unit > 0x1p-10f && unit < 0x1p6f)) {
        const float f = ref / rv;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] *= f;
        ref = rv;
        unit = 1.f;
      }
    }
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = __builtin_amdgcn_exp2f(x[j] - m);
      l += p[j];
      p[j] *= unit;
    }
    // a block whose range is NaN holds zero codes; the rows that see it are NaN
    if (rv != rv && seen) l = __uint_as_float(0x7FC00000u);
    const F pf = frag8(p, (F*)nullptr);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      F a;
      codes8<CODE>(vf[e].x, vf[e].y, &a);
      acc[2 * e] = mma(a, pf, acc[2 * e]);
      codes8<CODE>(vf[e].z, vf[e].w, &a);
      acc[2 * e + 1] = mma(a, pf, acc[2 * e + 1]);
    }
#pragma unroll
    for (int n = 0; n < 2 * NC; ++n) kf[n] = kn[n];
#pragma unroll
    for (int e = 0; e < NE; ++e) vf[e] = vn[e];
    rk = rkn;
    rv = rvn;
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) { lds_ml[wave][i][0] = m; lds_ml[wave][i][1] = l; }
  if (lane == 0) lds_ref[wave] = ref / Code<CODE>::kTop;
  float* part = tile.splits > 1 ? A.part + ((int64_t)(tile.part + tile.split) * kv.n_kv + head) * kv_part_floats(D) : nullptr;
  constexpr int PER = DC / 16;                   // columns of a thread
  const int orow = tid >> 4, od = (tid & 15) * PER, gr = tile.tile * kKvRows + orow;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += DC) {
    if (c0) __syncthreads();
#pragma unroll
    for (int n = 0; n < DC / 16; ++n) *(float4v*)&lds_o[wave][i][n * 16 + g * 4] = acc[c0 / 16 + n];
    __syncthreads();
    float mm = lds_ml[0][orow][0];
#pragma unroll
    for (int w = 1; w < 4; ++w) mm = fmaxf(mm, lds_ml[w][orow][0]);
    float ll = 0.f, o[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) o[j] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(lds_ml[w][orow][0] - mm), fo = f * lds_ref[w];
      ll += f * lds_ml[w][orow][1];
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] += fo * lds_o[w][orow][od + j];
    }
    if (part) {
#pragma unroll
      for (int j = 0; j < PER; j += 4) *(float4v*)(part + orow * D + c0 + od + j) = float4v{o[j], o[j + 1], o[j + 2], o[j + 3]};
      if (c0 == 0 && (tid & 15) == 0) {
        part[kKvRows * D + 2 * orow] = mm;
        part[kKvRows * D + 2 * orow + 1] = ll;
      }
    } else if (gr < packed) {
      T* out = (T*)A.out + (int64_t)(sq.row0 + gr / G) * A.out_stride + (head * G + gr % G) * D + c0 + od;
      const float inv = 1.f / ll;
#pragma unroll
      for (int j = 0; j < PER; ++j) out[j] = (T)(o[j] * inv);
    }
  }
}

// Joins the splits of a row tile: one workgroup per tile and kv head.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_combine_kernel(KvAttend A) {
  constexpr int PER = D / 16;
  const KvView& kv = A.kv;
  const KvTile tile = A.tiles[A.n_tiles + blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const KvSeq sq = A.seqs[tile.s];
  const int G = kv.n_heads / kv.n_kv, tid = threadIdx.x, orow = tid >> 4, od = (tid & 15) * PER;
  const int gr = tile.tile * kKvRows + orow;
  if (gr >= sq.rows * G) return;
  const int64_t step = kv.n_kv * kv_part_floats(D);
  const float* part = A.part + ((int64_t)tile.part * kv.n_kv + head) * kv_part_floats(D);
  float mm = -FLT_MAX;
  for (int s = 0; s < tile.splits; ++s) mm = fmaxf(mm, part[s * step + kKvRows * D + 2 * orow]);
  float ll = 0.f, o[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) o[j] = 0.f;
  for (int s = 0; s < tile.splits; ++s) {
    const float* ps = part + s * step;
    const float f = __builtin_amdgcn_exp2f(ps[kKvRows * D + 2 * orow] - mm);
    ll += f * ps[kKvRows * D + 2 * orow + 1];
#pragma unroll
    for (int j = 0; j < PER; j += 4) {
      const float4v x = *(const float4v*)(ps + orow * D + od + j);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[j + c] += f * x[c];
    }
  }
  T* out = (T*)A.out + (int64_t)(sq.row0 + gr / G) * A.out_stride + (head * G + gr % G) * D + od;
  const float inv = 1.f / ll;
#pragma unroll
  for (int j = 0; j < PER; ++j) out[j] = (T)(o[j] * inv);
}

// ---------------------------------------------------------------------------
// Reading back: one workgroup per touched block and kv head, an element a thread.

template <typename T, int CODE>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvRead R) {
  using C = Code<CODE>;
  const KvView& kv = R.kv;
  const int dim = kv.dim;
  const KvBlock blk = R.blocks[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const KvSeq sq = R.seqs[blk.s];
  const int32_t page = kv_row(kv, sq.seq, R.layer, head)[blk.block];
  const uint8_t* kbase = (const uint8_t*)kv.base + (int64_t)page * kv.page_bytes;
  const uint8_t* vbase = kbase + (int64_t)kv.block * dim;
  const float uk = kv.range[2 * (int64_t)page] / C::kTop, uv = kv.range[2 * (int64_t)page + 1] / C::kTop;
  const int64_t row0 = (int64_t)sq.row0 + blk.block * kv.block - sq.start;
  for (int u = threadIdx.x; u < (blk.slot1 - blk.slot0) * dim; u += kThreads) {
    const int slot = blk.slot0 + u / dim, d = u % dim;
    if (R.k) ((T*)R.k)[(row0 + slot) * R.k_stride + (int64_t)head * dim + d] = (T)(C::value(kbase[kv_k_byte(slot, d, dim)]) * uk);
    if (R.v) ((T*)R.v)[(row0 + slot) * R.v_stride + (int64_t)head * dim + d] = (T)(C::value(vbase[kv_v_byte(slot, d, dim)]) * uv);
  }
}

// ---------------------------------------------------------------------------
// Launches.

template <typename Arg>
static hipError_t run(const void* kernel, int64_t blocks, const Arg& arg, hipStream_t stream) {
  if (blocks <= 0) return hipSuccess;
  void* args[] = {const_cast<Arg*>(&arg)};
  return hipLaunchKernel(kernel, dim3((unsigned)blocks), dim3(kThreads), args, 0, stream);
}

hipError_t launch_kv_patch(int32_t* table, const KvPatch* patches, int32_t n, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  void* args[] = {&table, &patches, &n};
  return hipLaunchKernel((const void*)kv_patch_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads),
                         args, 0, stream);
}

template <typename T>
static const void* append_of(int code) {
  return code == SLORA_KV_INT8 ? (const void*)kv_append_kernel<T, SLORA_KV_INT8>
                               : (const void*)kv_append_kernel<T, SLORA_KV_FP8>;
}
template <typename T>
static const void* read_of(int code) {
  return code == SLORA_KV_INT8 ? (const void*)kv_read_kernel<T, SLORA_KV_INT8>
                               : (const void*)kv_read_kernel<T, SLORA_KV_FP8>;
}
template <typename T, int CODE>
static const void* rows_of(int dim) {
  return dim == 64 ? (const void*)kv_attend_rows_kernel<T, CODE, 64>
         : dim == 128 ? (const void*)kv_attend_rows_kernel<T, CODE, 128> : (const void*)kv_attend_rows_kernel<T, CODE, 256>;
}
template <typename T>
static const void* rows_of(int code, int dim) {
  return code == SLORA_KV_INT8 ? rows_of<T, SLORA_KV_INT8>(dim) : rows_of<T, SLORA_KV_FP8>(dim);
}
template <typename T>
static const void* combine_of(int dim) {
  return dim == 64 ? (const void*)kv_combine_kernel<T, 64>
         : dim == 128 ? (const void*)kv_combine_kernel<T, 128> : (const void*)kv_combine_kernel<T, 256>;
}

hipError_t launch_kv_append(const KvAppend& A, hipStream_t stream) {
  int64_t blocks = (int64_t)A.n_blocks * A.kv.n_kv;
  if (A.q) blocks += ((int64_t)A.n_rows * A.kv.n_heads * (A.kv.dim / 16) + kThreads - 1) / kThreads;
  return run(A.kv.dtype == SLORA_F16 ? append_of<_Float16>(A.kv.code) : append_of<float>(A.kv.code), blocks, A, stream);
}

hipError_t launch_kv_attend(const KvAttend& A, hipStream_t stream) {
  const bool half = A.kv.dtype == SLORA_F16;
  hipError_t e = run(half ? rows_of<_Float16>(A.kv.code, A.kv.dim) : rows_of<float>(A.kv.code, A.kv.dim),
                     (int64_t)A.n_tiles * A.kv.n_kv, A, stream);
  if (e != hipSuccess) return e;
  return run(half ? combine_of<_Float16>(A.kv.dim) : combine_of<float>(A.kv.dim), (int64_t)A.n_combine * A.kv.n_kv, A,
             stream);
}

hipError_t launch_kv_read(const KvRead& R, hipStream_t stream) {
  return run(R.kv.dtype == SLORA_F16 ? read_of<_Float16>(R.kv.code) : read_of<float>(R.kv.code),
             (int64_t)R.n_blocks * R.kv.n_kv, R, stream);
}

}  // namespace slora
