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

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
// 16 bytes that nobody else reads: they do not displace what is in the caches.
__device__ __forceinline__ uint4 ld16_once(const void* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const uint4v*>(p)));
}

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
  // Added to 1.5 * 2^52, a number this small is rounded to an integer (ties to
  // even) that stands in the low bits.  A subnormal range may lie below its
  // largest value by half a unit, which takes codes up to half as much again:
  // they are held at the largest one.
  static __device__ __forceinline__ uint32_t nearest(double x) {
#pragma clang fp contract(off)
    return (uint32_t)min(max(__double2loint(x + (0x1.8p52 + 128.)), 1), 255);
  }
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
  // The definition rounds the 64-bit product to fp32 and then to e4m3.  A
  // subnormal range's values are held at the last code as above.
  static __device__ __forceinline__ uint32_t nearest(double x) {
    const float y = __builtin_amdgcn_fmed3f((float)x, -kTop, kTop);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, 0.f, 0, false) & 0xFF;
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
// Elements in memory, 8 at a time.

template <typename T> struct Vec;
template <> struct Vec<_Float16> { typedef half8 v8; };
template <> struct Vec<float> { typedef float8v v8; };

// Unit u of a row is eight of its pairs (a, b): of the rotated part, and behind
// it, turned by no angle, elements 16u .. 16u + 15 as pairs of neighbours
// (halves: of 8 and 8).  Their elements lie in two runs of 8.
template <typename T> struct Pairs { typename Vec<T>::v8 a, b; };
struct Turn { float8v c, s; };

__device__ __forceinline__ void unit_runs(const KvView& kv, int u, int* a, int* b) {
  const bool split = kv.pairs == SLORA_KV_HALVES && u * 16 < kv.rot;
  *a = split ? u * 8 : u * 16;
  *b = split ? (kv.rot >> 1) + u * 8 : u * 16 + 8;
}
template <typename T>
__device__ __forceinline__ Pairs<T> load_pairs(const KvView& kv, const T* head, int a, int b) {
  typedef typename Vec<T>::v8 V;
  const V x = *reinterpret_cast<const V*>(head + a), y = *reinterpret_cast<const V*>(head + b);
  if (kv.pairs == SLORA_KV_HALVES) return {x, y};
  return {__builtin_shufflevector(x, y, 0, 2, 4, 6, 8, 10, 12, 14),
          __builtin_shufflevector(x, y, 1, 3, 5, 7, 9, 11, 13, 15)};
}
__device__ __forceinline__ Turn load_turn(const KvView& kv, const float* cos_sin, int64_t pos, int u) {
  if (u * 16 >= kv.rot) return {float8v{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, float8v{}};
  const float* row = cos_sin + pos * kv.rot + u * 8;
  return {*reinterpret_cast<const float8v*>(row), *reinterpret_cast<const float8v*>(row + (kv.rot >> 1))};
}
// Products of an fp16 or fp32 element and an fp32 cosine are exact in 64 bits,
// so the result is rounded once whether or not the compiler fuses them.
__device__ __forceinline__ void turned(float a, float b, float c, float s, double* ra, double* rb) {
  *ra = (double)a * c - (double)b * s;
  *rb = (double)b * c + (double)a * s;
}

// The same in fp32: one rounding of a product, one of the sum.
__device__ __forceinline__ void turned(float a, float b, float c, float s, float* ra, float* rb) {
  *ra = __builtin_fmaf(a, c, -(b * s));
  *rb = __builtin_fmaf(b, c, a * s);
}

// 4 x 4 bytes across four lanes: lane k of a quad gets byte k of lanes 0 .. 3.
__device__ __forceinline__ uint32_t quad_transpose(uint32_t x, int lane) {
  uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true);       // lane ^ 1
  x = __builtin_amdgcn_perm(y, x, lane & 1 ? 0x03070105u : 0x06020400u);
  y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true);                // lane ^ 2
  return __builtin_amdgcn_perm(y, x, lane & 2 ? 0x03020706u : 0x05040100u);
}

// ---------------------------------------------------------------------------
// Append.  Blocks that gain one token (decode) are a wave's work, keys and
// values together, a pair of elements of each a lane (store_one).  Otherwise an
// item is the keys or the values of one touched block of one kv head, and a
// workgroup's work: keys go in units of 8 pairs of a token; values in the page's 16-byte units (2
// elements of 8 tokens), read token by token, 8 elements a lane, and turned by
// byte transposes across four lanes.  The first pass finds the largest
// magnitude and keeps one unit a thread in registers (all there is where a page
// holds 8 KiB); what is beyond it is read again by the second pass, which
// writes the codes.

// Bit patterns of non-negative floats order as integers, with infinities and
// NaN above every finite one.
__device__ __forceinline__ uint32_t magnitude(double x) { return __float_as_uint(fabsf((float)x)); }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(fabsf(x)); }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* lds) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v = max(v, lds[w]);
  return v;
}

template <int CODE>
__device__ __forceinline__ uint32_t again4(uint32_t old, double ratio) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w |= Code<CODE>::nearest((double)Code<CODE>::value((old >> (8 * j)) & 0xFF) * ratio) << (8 * j);
  return w;
}
template <int CODE>
__device__ __forceinline__ uint4 again16(uint4 o, double ratio) {
  return make_uint4(again4<CODE>(o.x, ratio), again4<CODE>(o.y, ratio), again4<CODE>(o.z, ratio),
                    again4<CODE>(o.w, ratio));
}

// Elements of a value unit as they are read: 8 of each of two tokens.  old: the
// unit as the page holds it, where the append leaves some of its tokens as they
// are.
template <typename T> struct Values { typename Vec<T>::v8 x[2]; uint4 old; };

// What both kinds of item need.
struct Item {
  KvBlock blk;
  int head, dim, ush, pos0;     // ush: log2 of the units of a token (dim / 16); pos0: position of slot 0
  int64_t row0;                 // batch row of slot 0 (negative before the first new slot)
  uint8_t* page;
  float* range;
};
__device__ __forceinline__ Item item_of(const KvAppend& A, uint32_t at) {
  const KvView& kv = A.kv;
  Item it;
  const uint32_t b = at / (uint32_t)kv.n_kv;
  it.blk = A.blocks[b];
  it.head = (int)(at - b * kv.n_kv);
  it.dim = kv.dim;
  it.ush = 27 - __clz(kv.dim);
  it.pos0 = it.blk.block * kv.block;
  it.row0 = (int64_t)it.blk.row - it.blk.slot0;
  const int32_t page = kv_row(kv, it.blk.seq, A.layer, it.head)[it.blk.block];
  it.page = (uint8_t*)kv.base + (int64_t)page * kv.page_bytes;
  it.range = kv.range + 2 * (int64_t)page;
  return it;
}

// One token of one head by a wave: lane v takes pair v of the keys and, of the
// values, elements 2v and 2v + 1, which are two bytes of one 16-byte unit.
template <typename T, int CODE>
__device__ __forceinline__ void store_one(const KvAppend& A, uint32_t at, int lane) {
  using C = Code<CODE>;
  constexpr int N = 2;                                         // pairs a lane: 1 up to 128 elements, 2 for 256
  const KvView& kv = A.kv;
  const Item it = item_of(A, at);
  const int dim = it.dim, slot = it.blk.slot0, t = slot & 31, g = (t & 15) >> 2;
  const int half = kv.rot >> 1, shift = 8 * (t & 3), high = t >> 4;
  uint8_t* vbase = it.page + (int64_t)kv.block * dim;
  const T* kin = (const T*)A.k + it.blk.row * A.k_stride + (int64_t)it.head * dim;
  const T* vin = (const T*)A.v + it.blk.row * A.v_stride + (int64_t)it.head * dim;
  const float* cs = A.cos_sin + (int64_t)(it.pos0 + slot) * kv.rot;
  const uint32_t held_k = slot ? __float_as_uint(it.range[0]) & 0x7FFFFFFFu : 0;
  const uint32_t held_v = slot ? __float_as_uint(it.range[1]) & 0x7FFFFFFFu : 0;
  double ka[N], kb[N];
  float v0[N], v1[N];
  uint4 old[N];
  int da[N], db[N];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = lane + 64 * n;
    if (2 * p >= dim) continue;
    const bool turns = p < half, split = turns && kv.pairs == SLORA_KV_HALVES;
    da[n] = split ? p : 2 * p;
    db[n] = split ? half + p : 2 * p + 1;
    turned((float)kin[da[n]], (float)kin[db[n]], turns ? cs[p] : 1.f, turns ? cs[half + p] : 0.f, &ka[n], &kb[n]);
    v0[n] = (float)vin[2 * p];
    v1[n] = (float)vin[2 * p + 1];
    // the unit's other tokens, of which none is there yet in the first one's case
    old[n] = ld16(vbase + (int64_t)(slot >> 5) * 32 * dim + (p >> 4) * 1024 + g * 256 + (p & 15) * 16);
    mk = max(mk, max(magnitude(ka[n]), magnitude(kb[n])));
    mv = max(mv, max(magnitude(v0[n]), magnitude(v1[n])));
  }
  mk = max(wave_max(mk), held_k);
  mv = max(wave_max(mv), held_v);
  const bool bad_k = mk >= 0x7F800000u, bad_v = mv >= 0x7F800000u;
  if (lane == 0) {
    it.range[0] = bad_k ? __uint_as_float(0x7FC00000u) : __uint_as_float(mk);
    it.range[1] = bad_v ? __uint_as_float(0x7FC00000u) : __uint_as_float(mv);
  }
  const double new_k = __uint_as_float(mk), new_v = __uint_as_float(mv);
  const double inv_k = mk ? (double)C::kTop / new_k : 0., inv_v = mv ? (double)C::kTop / new_v : 0.;
  const bool grew_k = slot && mk != held_k, grew_v = slot && mv != held_v;
  const double ratio_v = grew_v && !bad_v ? (double)__uint_as_float(held_v) / new_v : 0.;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = lane + 64 * n;
    if (2 * p >= dim) continue;
    it.page[kv_k_byte(slot, da[n], dim)] = (uint8_t)(bad_k ? C::kZero : C::nearest(ka[n] * inv_k));
    it.page[kv_k_byte(slot, db[n], dim)] = (uint8_t)(bad_k ? C::kZero : C::nearest(kb[n] * inv_k));
    const uint32_t c0 = bad_v ? C::kZero : C::nearest((double)v0[n] * inv_v);
    const uint32_t c1 = bad_v ? C::kZero : C::nearest((double)v1[n] * inv_v);
    uint4 w = grew_v ? again16<CODE>(old[n], ratio_v) : old[n];
    uint32_t& w0 = high ? w.y : w.x;
    uint32_t& w1 = high ? w.w : w.z;
    w0 = (w0 & ~(0xFFu << shift)) | c0 << shift;
    w1 = (w1 & ~(0xFFu << shift)) | c1 << shift;
    st16(vbase + (int64_t)(slot >> 5) * 32 * dim + (p >> 4) * 1024 + g * 256 + (p & 15) * 16, w);
  }
  if (grew_k) {
    const double ratio = bad_k ? 0. : (double)__uint_as_float(held_k) / new_k;
    for (int u = lane; u < slot << it.ush; u += 64) {
      uint8_t* p = it.page + kv_k_byte(u >> it.ush, (u & ((1 << it.ush) - 1)) * 16, dim);
      st16(p, again16<CODE>(ld16(p), ratio));
    }
  }
  if (grew_v)                                                  // every unit but those the token is in
    for (int u = lane; u < ((slot >> 5) + 1) << (it.ush + 5); u += 64) {
      if (u >> (it.ush + 5) == slot >> 5 && ((u >> 4) & 3) == g) continue;
      st16(vbase + (int64_t)u * 16, again16<CODE>(ld16(vbase + (int64_t)u * 16), ratio_v));
    }
}

template <typename T, int CODE>
__device__ __forceinline__ void store_keys(const KvAppend& A, uint32_t at, int tid, uint32_t* lds) {
  using C = Code<CODE>;
  const KvView& kv = A.kv;
  const Item it = item_of(A, at);
  const KvBlock& blk = it.blk;
  const int ush = it.ush, units = (blk.slot1 - blk.slot0) << ush;
  const T* in = (const T*)A.k + (int64_t)it.head * it.dim;
  const uint32_t held = blk.slot0 ? __float_as_uint(it.range[0]) & 0x7FFFFFFFu : 0;

  auto load = [&](int u, Pairs<T>* x, Turn* t) {
    const int slot = blk.slot0 + (u >> ush), c = u & ((1 << ush) - 1);
    int a, b;
    unit_runs(kv, c, &a, &b);
    *x = load_pairs(kv, in + (it.row0 + slot) * A.k_stride, a, b);
    *t = load_turn(kv, A.cos_sin, it.pos0 + slot, c);
  };
  auto largest = [&](const Pairs<T>& x, const Turn& t) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double ra, rb;
      turned((float)x.a[j], (float)x.b[j], t.c[j], t.s[j], &ra, &rb);
      m = max(m, max(magnitude(ra), magnitude(rb)));
    }
    return m;
  };
  Pairs<T> kept{};
  Turn kept_turn{};
  if (tid < units) load(tid, &kept, &kept_turn);
  uint32_t m = largest(kept, kept_turn);
  for (int u = tid + kThreads; u < units; u += kThreads) {
    Pairs<T> x;
    Turn t;
    load(u, &x, &t);
    m = max(m, largest(x, t));
  }
  m = max(team_max(m, lds), held);
  const bool bad = m >= 0x7F800000u;
  if (tid == 0) it.range[0] = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(m);
  const double grown = __uint_as_float(m), inv = m ? (double)C::kTop / grown : 0.;

  auto put = [&](int u, const Pairs<T>& x, const Turn& t) {
    const int slot = blk.slot0 + (u >> ush), c = u & ((1 << ush) - 1);
    int a, b;
    unit_runs(kv, c, &a, &b);
    uint32_t wa[2] = {0, 0}, wb[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double ra, rb;
      turned((float)x.a[j], (float)x.b[j], t.c[j], t.s[j], &ra, &rb);
      wa[j >> 2] |= C::nearest(ra * inv) << (8 * (j & 3));
      wb[j >> 2] |= C::nearest(rb * inv) << (8 * (j & 3));
    }
    uint2 first = make_uint2(wa[0], wa[1]), second = make_uint2(wb[0], wb[1]);
    if (kv.pairs == SLORA_KV_NEIGHBOURS) {
      first = make_uint2(__builtin_amdgcn_perm(wb[0], wa[0], 0x05010400u),
                         __builtin_amdgcn_perm(wb[0], wa[0], 0x07030602u));
      second = make_uint2(__builtin_amdgcn_perm(wb[1], wa[1], 0x05010400u),
                          __builtin_amdgcn_perm(wb[1], wa[1], 0x07030602u));
    }
    if (bad) first = second = make_uint2(C::kZero * 0x01010101u, C::kZero * 0x01010101u);
    *reinterpret_cast<uint2*>(it.page + kv_k_byte(slot, a, it.dim)) = first;
    *reinterpret_cast<uint2*>(it.page + kv_k_byte(slot, b, it.dim)) = second;
  };
  if (tid < units) put(tid, kept, kept_turn);
  for (int u = tid + kThreads; u < units; u += kThreads) {
    Pairs<T> x;
    Turn t;
    load(u, &x, &t);
    put(u, x, t);
  }
  if (blk.slot0 && m != held) {                                // the range grew: older keys are coded again
    const double ratio = bad ? 0. : (double)__uint_as_float(held) / grown;
    for (int u = tid; u < blk.slot0 << ush; u += kThreads) {
      uint8_t* p = it.page + kv_k_byte(u >> ush, (u & ((1 << ush) - 1)) * 16, it.dim);
      st16(p, again16<CODE>(ld16(p), ratio));
    }
  }
}

template <typename T, int CODE>
__device__ __forceinline__ void store_values(const KvAppend& A, uint32_t at, int tid, uint32_t* lds) {
  using C = Code<CODE>;
  typedef typename Vec<T>::v8 V8;
  const KvView& kv = A.kv;
  const Item it = item_of(A, at);
  const KvBlock& blk = it.blk;
  const int ush = it.ush, lane = tid & 63;
  const int group0 = blk.slot0 >> 5, group1 = (blk.slot1 + 31) >> 5;
  const int units = (group1 - group0) << (ush + 5);            // a multiple of 64: a wave's lanes act alike
  const int g = lane >> 4, quad = (lane >> 2) & 3, k4 = lane & 3;
  uint8_t* base = it.page + (int64_t)kv.block * it.dim;
  const T* in = (const T*)A.v + (int64_t)it.head * it.dim + quad * 8;
  const uint32_t held = blk.slot0 ? __float_as_uint(it.range[1]) & 0x7FFFFFFFu : 0;

  auto load = [&](int u, Values<T>* x) {
    const int group = group0 + (u >> (ush + 5)), e = (u >> 6) & ((1 << (ush - 1)) - 1);
    x->old = make_uint4(0, 0, 0, 0);
    if (group * 32 < blk.slot0 || group * 32 + 32 > blk.slot1)
      x->old = ld16(base + (int64_t)(group0 * it.dim * 2 + u) * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = group * 32 + h * 16 + g * 4 + k4;
      x->x[h] = V8{};
      if (slot >= blk.slot0 && slot < blk.slot1)
        x->x[h] = *reinterpret_cast<const V8*>(in + (it.row0 + slot) * A.v_stride + e * 32);
    }
  };
  auto largest = [&](const Values<T>& x) {
    uint32_t m = 0;
#pragma unroll
    for (int n = 0; n < 16; ++n) m = max(m, magnitude((float)x.x[n >> 3][n & 7]));
    return m;
  };
  Values<T> kept{};
  if (tid < units) load(tid, &kept);
  uint32_t m = largest(kept);
  for (int u = tid + kThreads; u < units; u += kThreads) {
    Values<T> x;
    load(u, &x);
    m = max(m, largest(x));
  }
  m = max(team_max(m, lds), held);
  const bool bad = m >= 0x7F800000u, grew = blk.slot0 && m != held;
  if (tid == 0) it.range[1] = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(m);
  const double grown = __uint_as_float(m), inv = m ? (double)C::kTop / grown : 0.;
  const double ratio = grew && !bad ? (double)__uint_as_float(held) / grown : 0.;

  auto put = [&](int u, const Values<T>& x) {
    const int group = group0 + (u >> (ush + 5));
    uint32_t w[4], mask[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int slot = group * 32 + h * 16 + g * 4 + b;
        if (slot >= blk.slot0 && slot < blk.slot1) mask[h] |= 0xFFu << (8 * b);
      }
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) c |= C::nearest((double)(float)x.x[h][2 * j + d] * inv) << (8 * j);
        w[2 * d + h] = quad_transpose(bad ? C::kZero * 0x01010101u : c, lane);
      }
    }
    if ((mask[0] & mask[1]) != 0xFFFFFFFFu) {
      if (!(mask[0] | mask[1]) && !grew) return;
      const uint4 old = grew ? again16<CODE>(x.old, ratio) : x.old;
      w[0] = (w[0] & mask[0]) | (old.x & ~mask[0]);
      w[1] = (w[1] & mask[1]) | (old.y & ~mask[1]);
      w[2] = (w[2] & mask[0]) | (old.z & ~mask[0]);
      w[3] = (w[3] & mask[1]) | (old.w & ~mask[1]);
    }
    st16(base + (int64_t)(group0 * it.dim * 2 + u) * 16, make_uint4(w[0], w[1], w[2], w[3]));
  };
  if (tid < units) put(tid, kept);
  for (int u = tid + kThreads; u < units; u += kThreads) {
    Values<T> x;
    load(u, &x);
    put(u, x);
  }
  if (grew)                                                    // groups of older values only
    for (int u = tid; u < group0 << (ush + 5); u += kThreads)
      st16(base + (int64_t)u * 16, again16<CODE>(ld16(base + (int64_t)u * 16), ratio));
}

// Workgroups: single tokens, four (block, head) pairs each; items of the other
// blocks; and q, whose workgroups stream and are spread evenly among those,
// which wait: a thread rotates one unit of A.q_heads heads of a row, so that a
// row's angles are read once for them.
template <typename T, int CODE>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppend A) {
  typedef typename Vec<T>::v8 V8;
  const KvView& kv = A.kv;
  __shared__ uint32_t lds[kThreads / 64];
  const int tid = threadIdx.x;
  // q workgroups up to here, and whether this is one
  const uint32_t q_wg = __umulhi(blockIdx.x, A.q_share);
  const bool is_q = __umulhi(blockIdx.x + 1, A.q_share) != q_wg;
  if (!is_q) {
    const uint32_t wg = blockIdx.x - q_wg, small = (uint32_t)A.n_small * kv.n_kv, small_wgs = (small + 3) / 4;
    if (wg < small_wgs) {
      const uint32_t item = uni(wg * 4 + (tid >> 6));
      if (item < small) store_one<T, CODE>(A, item, tid & 63);
    } else {
      const uint32_t item = wg - small_wgs;
      if (item & 1) store_values<T, CODE>(A, small + (item >> 1), tid, lds);
      else store_keys<T, CODE>(A, small + (item >> 1), tid, lds);
    }
    return;
  }
  const uint32_t chunks = (kv.n_heads + A.q_heads - 1) / A.q_heads;
  const int ush = 27 - __clz(kv.dim);
  const uint64_t i = (uint64_t)q_wg * kThreads + tid;
  const uint32_t rc = (uint32_t)(i >> ush);
  const int u = (int)(i & ((1u << ush) - 1)), row = (int)(rc / chunks), h0 = (int)(rc - row * chunks) * A.q_heads;
  if (row >= A.n_rows) return;
  int a, b;
  unit_runs(kv, u, &a, &b);
  const bool turns = u * 16 < kv.rot;
  const Turn t = load_turn(kv, A.cos_sin, A.row_pos[row], u);
  const T* in = (const T*)A.q + row * A.q_stride;
  T* out = (T*)A.q_out + row * A.q_out_stride;
  const int h1 = min(kv.n_heads, h0 + A.q_heads);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    Pairs<T> x = load_pairs(kv, in + h * kv.dim, a, b);
    if (turns) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float ra, rb;
        turned((float)x.a[j], (float)x.b[j], t.c[j], t.s[j], &ra, &rb);
        x.a[j] = (T)ra;
        x.b[j] = (T)rb;
      }
    }
    V8 first = x.a, second = x.b;
    if (kv.pairs == SLORA_KV_NEIGHBOURS) {
      first = __builtin_shufflevector(x.a, x.b, 0, 8, 1, 9, 2, 10, 3, 11);
      second = __builtin_shufflevector(x.a, x.b, 4, 12, 5, 13, 6, 14, 7, 15);
    }
    *reinterpret_cast<V8*>(out + h * kv.dim + a) = first;
    *reinterpret_cast<V8*>(out + h * kv.dim + b) = second;
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
//
// Of 16 rows a single token fills only G; the matrix cores have ten times what
// HBM can feed that way, and a vector dot product would spend its instructions
// on the conversions alone.  256 requests of 300 to 2000 tokens, 32 heads: 350 us,
// 6.5 TB/s of codes (the largest copy runs at 5.2, reads alone at up to 6.6); 32
// heads of 64 187 us (6.1), 16 of 256 346 us (6.6).

template <typename T> struct Frag;
template <> struct Frag<_Float16> { typedef half8 type; };
template <> struct Frag<float> { typedef float8v type; };

// Operands of the products: fp16 takes the codes, which it holds exactly, fp32
// the cached values, code * unit.
template <int CODE>
__device__ __forceinline__ void codes8(uint32_t a, uint32_t b, float, half8* r) { *r = Code<CODE>::halves(a, b); }
template <int CODE>
__device__ __forceinline__ void codes8(uint32_t a, uint32_t b, float unit, float8v* r) {
  *r = floats8<CODE>(a, b) * unit;
}

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

// Joining the key splits of a row tile in the same launch: every split's
// workgroup writes its sums where all of them can see them (agent-scope atomic
// stores, which are done at the level that the XCDs share), waits until they are
// there, and counts itself; the one that finds the others counted joins all
// sums, read at that level too, in the order of the splits, and sets the counter
// back for the next launch.  No cache has to be written back or dropped for
// this: with an acquire-release counter, which does both, 12 long conversations
// took 196 us instead of 120.  One launch instead of two: 7.5 us instead of 8.4
// for a single token.
typedef unsigned long long u64;
__device__ __forceinline__ void put_shared(float* p, float a, float b) {
  const u64 w = (u64)__float_as_uint(b) << 32 | __float_as_uint(a);
  __hip_atomic_store(reinterpret_cast<u64*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2v get_shared(const float* p) {
  const u64 w = __hip_atomic_load(reinterpret_cast<const u64*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return float2v{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ __forceinline__ bool last_of(uint32_t* counter, int splits, uint32_t* lds) {
  __builtin_amdgcn_s_waitcnt(0);                 // this wave's sums are where the others see them
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == (uint32_t)splits - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds = before;
  }
  __syncthreads();
  return *lds == (uint32_t)splits - 1;
}

// The bound of two waves a SIMD makes the compiler spare registers: three run at
// heads of 128 (147 registers instead of 184, decode batch 374 to 350 us) and five
// at 64.  Heads of 256 reach two by loading the next keys only when these are
// multiplied (f16 324 to 194 registers, 16 requests of 4500 to 9000 tokens, 16
// heads on 4, 88 to 59 us).
template <typename T, int CODE, int D>
__global__ __launch_bounds__(kThreads, 2) void kv_attend_rows_kernel(KvAttend A) {
  using F = typename Frag<T>::type;
  constexpr int NC = D / 64, NE = D / 32, NT = D / 16;
  constexpr int DC = D < 128 ? D : 128;          // columns joined at a time
  // fp32 multiplies cached values and weights of at most 1, so that ranges may lie
  // as far apart as fp32 numbers: sums in units of one block's range, which fp16
  // codes need, would overflow or vanish beside another's.
  constexpr bool values = sizeof(T) == 4;
  __shared__ float lds_o[4][kKvRows][DC + 4];
  __shared__ float lds_ml[4][kKvRows][2];
  __shared__ float lds_ref[4];
  __shared__ uint32_t lds_last;
  const KvView& kv = A.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), i = lane & 15, g = lane >> 4;
  const KvTile tile = A.tiles[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const int G = kv.n_heads / kv.n_kv, packed = tile.rows * G;

  // this lane's query row (rows past the last one repeat it and are not stored)
  const int r = min(tile.tile * kKvRows + i, packed - 1);
  const int t = r / G, pos = tile.start + t;
  const int lo = A.window ? max(0, pos - A.window + 1) : 0;
  const int t_first = tile.tile * kKvRows / G, t_last = (min(tile.tile * kKvRows + kKvRows, packed) - 1) / G;
  const int pos_first = tile.start + t_first, pos_last = tile.start + t_last, len = tile.start + tile.rows;
  const int tile_lo = A.window ? max(0, pos_first - A.window + 1) : 0;
  const int all_lo = A.window ? max(0, pos_last - A.window + 1) : 0;

  F qf[2 * NC];
  {
    const T* q = (const T*)A.q + (int64_t)(tile.row0 + t) * A.q_stride + (head * G + r % G) * D;
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

  const int32_t* row = kv_row(kv, tile.seq, A.layer, head);
  const int nb = kv.block / kKvGroup;
  float4v acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = float4v{0.f, 0.f, 0.f, 0.f};
  float m = -FLT_MAX, l = 0.f, ref = 0.f;

  const bool once = packed <= kKvRows;
  int b = gi / nb, sub = gi - b * nb;
  uint4 kf[2 * NC], vf[NE];
  float rk = 0.f, rv = 0.f;
  auto load = [&](uint4* kx, uint4* vx, float& xk, float& xv) {
    const int32_t page = uni(row[b]);
    const char* kb = kv.base + (int64_t)page * kv.page_bytes + (int64_t)sub * kKvGroup * D;
    const char* vb = kb + (int64_t)kv.block * D;
    // With one tile a sequence its keys are read once: loads that leave the
    // caches alone took the 256-request decode batch from 394 to 355 us.  Further tiles find them in the caches.
    if (once) {
#pragma unroll
      for (int n = 0; n < 2 * NC; ++n) kx[n] = ld16_once(kb + n * 1024 + i * 64 + g * 16);
#pragma unroll
      for (int e = 0; e < NE; ++e) vx[e] = ld16_once(vb + e * 1024 + lane * 16);
    } else {
#pragma unroll
      for (int n = 0; n < 2 * NC; ++n) kx[n] = ld16(kb + n * 1024 + i * 64 + g * 16);
#pragma unroll
      for (int e = 0; e < NE; ++e) vx[e] = ld16(vb + e * 1024 + lane * 16);
    }
    xk = kv.range[2 * (int64_t)page];
    xv = kv.range[2 * (int64_t)page + 1];
    if (++sub == nb) { sub = 0; ++b; }
  };
  if (gi < ge) load(kf, vf, rk, rv);
  for (; gi < ge; ++gi) {
    uint4 kn[2 * NC], vn[NE];
    float rkn = 0.f, rvn = 0.f;
    if (D < 256 && gi + 1 < ge) load(kn, vn, rkn, rvn);
    const int key0 = gi * kKvGroup;

    // (a NaN range holds zero codes: its keys must be NaN, its values stay 0 for the rows that do not see them)
    const float uk = values ? rk / Code<CODE>::kTop : 1.f, uv = values && rv > 0.f ? rv / Code<CODE>::kTop : 0.f;
    float4v s0 = {0.f, 0.f, 0.f, 0.f}, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F a;
      codes8<CODE>(kf[c].x, kf[c].y, uk, &a);
      s0 = mma(a, qf[2 * c], s0);
      codes8<CODE>(kf[c].z, kf[c].w, uk, &a);
      s0 = mma(a, qf[2 * c + 1], s0);
      codes8<CODE>(kf[NC + c].x, kf[NC + c].y, uk, &a);
      s1 = mma(a, qf[2 * c], s1);
      codes8<CODE>(kf[NC + c].z, kf[NC + c].w, uk, &a);
      s1 = mma(a, qf[2 * c + 1], s1);
    }
    const float ck = values ? A.scale_log2 : rk / Code<CODE>::kTop * A.scale_log2;
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
    // fp16: values of a block count in units of its range: the sums are kept in
    // units of a reference range, replaced when a block's is far from it
    float unit = 1.f;
    if (!values && rv > 0.f) {
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
      p[j] = __builtin_amdgcn_exp2f(x[j] - (values ? m + kLazy : m));
      l += p[j];
      p[j] *= unit;
    }
    // a block whose range is NaN holds zero codes; the rows that see it are NaN
    if (rv != rv && seen) l = __uint_as_float(0x7FC00000u);
    // fp16: each weight as the sum of two, so that the output's rounding is all
    // that shows (with one, the error against 64 bits was up to 1.4 times that);
    // the second product cost 3 % of a decode batch
    const F pf = frag8(p, (F*)nullptr);
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rest[j] = p[j] - (float)pf[j];
    const F pr = frag8(rest, (F*)nullptr);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      F a;
      codes8<CODE>(vf[e].x, vf[e].y, uv, &a);
      acc[2 * e] = mma(a, pf, acc[2 * e]);
      if (sizeof(T) == 2) acc[2 * e] = mma(a, pr, acc[2 * e]);
      codes8<CODE>(vf[e].z, vf[e].w, uv, &a);
      acc[2 * e + 1] = mma(a, pf, acc[2 * e + 1]);
      if (sizeof(T) == 2) acc[2 * e + 1] = mma(a, pr, acc[2 * e + 1]);
    }
    if (D == 256) {
      if (gi + 1 < ge) load(kf, vf, rk, rv);
      continue;
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
  if (lane == 0) lds_ref[wave] = values ? 1.f : ref / Code<CODE>::kTop;
  float* part = tile.splits > 1
                    ? A.part + ((int64_t)(tile.part + tile.split) * kv.n_kv + head) * kv_part_floats(D) : nullptr;
  constexpr int PER = DC / 16;                   // columns of a thread
  const int orow = tid >> 4, od = (tid & 15) * PER, gr = tile.tile * kKvRows + orow;
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += DC) {
    if (c0) __syncthreads();
#pragma unroll
    for (int e = 0; e < DC / 32; ++e) {
      const float4v a = acc[c0 / 16 + 2 * e], b = acc[c0 / 16 + 2 * e + 1];
      *(float4v*)&lds_o[wave][i][e * 32 + g * 8] = float4v{a[0], b[0], a[1], b[1]};
      *(float4v*)&lds_o[wave][i][e * 32 + g * 8 + 4] = float4v{a[2], b[2], a[3], b[3]};
    }
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
      if (gr < packed) {
#pragma unroll
        for (int j = 0; j < PER; j += 2) put_shared(part + orow * D + c0 + od + j, o[j], o[j + 1]);
        if (c0 == 0 && (tid & 15) == 0) put_shared(part + kKvRows * D + 2 * orow, mm, ll);
      }
    } else if (gr < packed) {
      T* out = (T*)A.out + (int64_t)(tile.row0 + gr / G) * A.out_stride + (head * G + gr % G) * D + c0 + od;
      const float inv = 1.f / ll;
#pragma unroll
      for (int j = 0; j < PER; ++j) out[j] = (T)(o[j] * inv);
    }
  }
  if (!part || !last_of(A.counters + (int64_t)tile.part * kv.n_kv + head, tile.splits, &lds_last)) return;
  if (gr >= packed) return;
  const int64_t step = kv.n_kv * kv_part_floats(D);
  part = A.part + ((int64_t)tile.part * kv.n_kv + head) * kv_part_floats(D);
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += DC) {
    float mm = -FLT_MAX, ll = 0.f, o[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) o[j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < tile.splits; ++k) {
      const float* ps = part + k * step;
      const float2v ml = get_shared(ps + kKvRows * D + 2 * orow);
      float2v x[PER / 2];
#pragma unroll
      for (int j = 0; j < PER / 2; ++j) x[j] = get_shared(ps + orow * D + c0 + od + 2 * j);
      const float mn = fmaxf(mm, ml[0]), f = __builtin_amdgcn_exp2f(mm - mn), fs = __builtin_amdgcn_exp2f(ml[0] - mn);
      mm = mn;
      ll = ll * f + ml[1] * fs;
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] = o[j] * f + x[j / 2][j & 1] * fs;
    }
    T* out = (T*)A.out + (int64_t)(tile.row0 + gr / G) * A.out_stride + (head * G + gr % G) * D + c0 + od;
    const float inv = 1.f / ll;
#pragma unroll
    for (int j = 0; j < PER; ++j) out[j] = (T)(o[j] * inv);
  }
}

// ---------------------------------------------------------------------------
// Attention of a long run of rows (prompts), fp16: 128 packed rows of one kv
// head a workgroup, 32 a wave, over keys staged 32 or 64 at a time.  The codes
// of the next keys are loaded while these are multiplied, then converted once
// for all four waves into fp16 in LDS, two buffers in turn.
//
// The 32x32x16 instruction as in the row tiles: S^T = K Q^T leaves lane (h, n) =
// 32 h + n with query row n and keys 8a + 4h + b (a, b = 0 .. 3), registers 4a +
// b.  Eight registers are the second operand of O^T += V^T P^T for 16 keys.  V^T
// lies in LDS with a row's keys in that order, and its row m = 8a + 4h + b is
// element 16h + 4a + b, so that a lane ends with 16 consecutive elements.

typedef float float16v __attribute__((ext_vector_type(16)));

// 16-byte slot of 8 elements of a staged key, and of the keys (t, h) of element
// d of staged values; the low bits are exchanged so that the 16 lanes that read
// or write together meet all 64 banks.
template <int D>
__device__ __forceinline__ int k_slot(int key, int s) {
  return key * (D / 8) + (s ^ (D == 64 ? key >> 1 & 7 : key & 15));
}
__device__ __forceinline__ int v_slot(int d, int t, int h) {
  const int p = d >> 1;
  return p * 8 + (((d & 1) * 4 + 2 * t + h) ^ ((p >> 1 & 1) | (p >> 2 & 2) | (p & 4)));
}

template <int CODE, int D, bool TRIPLE>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : TRIPLE ? 3 : 2) void kv_attend_prompt_kernel(KvAttend A) {
  constexpr int NG = D == 256 || TRIPLE ? 1 : 2; // groups of 32 keys staged at a time
  constexpr int KS = D / 16, NB = D / 32;        // steps of the K product, blocks of 32 elements
  constexpr int UG = 2 * D, NU = NG * UG / kThreads;   // 16-byte units of a group (of K, of V) and of a thread
  __shared__ uint4 lds_k[2][NG][32 * D / 8];
  __shared__ uint4 lds_v[2][NG][D * 4];
  const KvView& kv = A.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), n = lane & 31, h = lane >> 5;
  const KvTile tile = A.prompts[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const int G = kv.n_heads / kv.n_kv, packed = tile.rows * G, r0 = tile.tile * kKvPromptRows;

  // this lane's query row; rows past the last one repeat it and are not stored
  const int r = r0 + wave * 32 + n, rr = min(r, packed - 1);
  int pos = tile.start + rr / G;
  asm("" : "+v"(pos));                           // all that is kept of its row: the rest would be spilled
  const uint32_t window = A.window ? (uint32_t)A.window : 1u << 31;
  const int len = tile.start + tile.rows;
  const int wg_first = tile.start + r0 / G, wg_last = tile.start + (min(r0 + kKvPromptRows, packed) - 1) / G;
  const int w_first = uni(tile.start + min(r0 + wave * 32, packed - 1) / G);
  const int w_last = uni(tile.start + min(r0 + wave * 32 + 31, packed - 1) / G);
  // a wave without rows only stages (asked for in the two-workgroup form, the
  // loop came out 12 % slower, where such waves are rare)
  const bool idle = r0 + wave * 32 >= packed;
  const int w_lo = A.window ? max(0, w_first - A.window + 1) : 0, w_all = A.window ? max(0, w_last - A.window + 1) : 0;
  half8 qf[KS];
  {
    const _Float16* q =
        (const _Float16*)A.q + (int64_t)(tile.row0 + pos - tile.start) * A.q_stride + (head * G + rr % G) * D;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qf[k] = *(const half8*)(q + k * 16 + h * 8);
      if (A.scale_log2 < 0.f) qf[k] = -qf[k];
    }
  }
  const float scale = fabsf(A.scale_log2) / Code<CODE>::kTop;
  const int g_lo = (A.window ? max(0, wg_first - A.window + 1) : 0) / kKvGroup, g_hi = wg_last / kKvGroup + 1;
  const int per = (g_hi - g_lo + tile.splits - 1) / tile.splits;
  const int g_begin = uni(g_lo + tile.split * per), g_end = uni(min(g_hi, g_begin + per));
  const int32_t* row = kv_row(kv, tile.seq, A.layer, head);
  const int nb = kv.block / kKvGroup;

  uint4 kc[NU], vc[NU];
  float rk[NG], rv[NG], rk_next[NG], rv_next[NG];
  // codes of groups g .. g + NG - 1 (those before g_end) and their ranges
  auto load = [&](int g) {
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      const int gg = min(g + x, g_end - 1), b = gg / nb, sub = gg - b * nb;
      const int32_t page = uni(row[b]);
      const char* kb = kv.base + (int64_t)page * kv.page_bytes + (int64_t)sub * kKvGroup * D;
      const char* vb = kb + (int64_t)kv.block * D;
      rk_next[x] = kv.range[2 * (int64_t)page];
      rv_next[x] = kv.range[2 * (int64_t)page + 1];
      // unit u of the thread's NU belongs to group u * kThreads / UG
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int at = u * kThreads + tid;
        if (NG == 1 || (UG >= kThreads ? u * kThreads / UG == x : at / UG == x)) {
          kc[u] = ld16(kb + (at % UG) * 16);
          vc[u] = ld16(vb + (at % UG) * 16);
        }
      }
    }
  };
  auto stage = [&](int buf, int g) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int at = u * kThreads + tid, x = at / UG, uu = at % UG;
      const int key = uu / D * 16 + uu % 64 / 4, slot = uu % D / 64 * 8 + uu % 4 * 2;
      lds_k[buf][x][k_slot<D>(key, slot)] = __builtin_bit_cast(uint4, Code<CODE>::halves(kc[u].x, kc[u].y));
      lds_k[buf][x][k_slot<D>(key, slot + 1)] = __builtin_bit_cast(uint4, Code<CODE>::halves(kc[u].z, kc[u].w));
      const int vg = uu % 64 / 16, d = uu / 64 * 32 + uu % 16 * 2;
      uint4 c = vc[u];
      // e4m3 bytes behind the sequence may be NaN, which a weight of zero keeps
      if (CODE == SLORA_KV_FP8 && (g + x) * kKvGroup + kKvGroup > len) {
        uint32_t keep[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((g + x) * kKvGroup + (j >> 2) * 16 + vg * 4 + (j & 3) < len) keep[j >> 2] |= 0xFFu << (8 * (j & 3));
        c = make_uint4(c.x & keep[0], c.y & keep[1], c.z & keep[0], c.w & keep[1]);
      }
      // lanes vg and vg + 2 (32 apart) hold the two quads of tokens of a slot: the
      // lower lane takes those of the group's first half, the upper the second's
      const auto even = __builtin_amdgcn_permlane32_swap(c.x, c.y, false, false);
      const auto odd = __builtin_amdgcn_permlane32_swap(c.z, c.w, false, false);
      lds_v[buf][x][v_slot(d, vg >> 1, vg & 1)] = __builtin_bit_cast(uint4, Code<CODE>::halves(even[0], even[1]));
      lds_v[buf][x][v_slot(d + 1, vg >> 1, vg & 1)] = __builtin_bit_cast(uint4, Code<CODE>::halves(odd[0], odd[1]));
    }
#pragma unroll
    for (int x = 0; x < NG; ++x) { rk[x] = rk_next[x]; rv[x] = rv_next[x]; }
  };

  float16v acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = float16v{};
  float m = -FLT_MAX, l = 0.f, ref = 0.f, minus = -1.f;
  asm("" : "+s"(minus));
  const int vd = (n >> 2 & 1) * 16 + (n >> 3) * 4 + (n & 3);     // element of this lane's row of a block of V^T

  if (g_begin < g_end) {
    load(g_begin);
    stage(0, g_begin);
  }
  lds_barrier();
  int buf = 0;
  for (int gb = g_begin; gb < g_end; gb += NG) {
    const bool more = gb + NG < g_end;
    if (more) load(gb + NG);
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      const int key0 = (gb + x) * kKvGroup;
      if (gb + x >= g_end || key0 > w_last || key0 + kKvGroup <= w_lo || (TRIPLE && idle)) continue;
      float16v s = {};
#pragma unroll
      for (int k = 0; k < KS; ++k)
        s = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(half8, lds_k[buf][x][k_slot<D>(n, 2 * k + h)]), qf[k], s, 0, 0, 0);
      // scores are s * ck with ck > 0: q carries the scale's sign, and a factor
      // of 0 or NaN would give hidden keys a weight
      float ck = rk[x] * scale;
      ck = ck > 0.f ? ck : FLT_MIN;
      bool seen = true;
      if (key0 + kKvGroup - 1 > w_first || key0 < w_all) {
        seen = false;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int key = key0 + (j >> 2) * 8 + h * 4 + (j & 3);
          const bool in = (uint32_t)(pos - key) < window;      // key <= pos and key > pos - window
          s[j] = in ? s[j] : -INFINITY;
          seen |= in;
        }
      }
      float top = s[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
      top *= ck;
      if (__any(top > m + kLazy)) {
        // both halves of the wave, without an address register as a shuffle takes
        const auto two = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        const float mn = fmaxf(m, fmaxf(__uint_as_float(two[0]), __uint_as_float(two[1])));
        const float f = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] *= f;
      }
      // values of a block count in units of its range: sums are kept in units of
      // a reference range, replaced when a block's is far from it.  The weights
      // carry the factor in their exponent, and their sum is freed of it; the
      // approximate reciprocal and logarithm weigh the block wrongly by 2^-20, where
      // the output has 11 bits.
      float unit = 1.f;
      if (rv[x] > 0.f) {
        unit = rv[x] * __builtin_amdgcn_rcpf(ref);
        if (!(unit > 0x1p-10f && unit < 0x1p6f)) {
          const float f = ref / rv[x];
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[b] *= f;
          ref = rv[x];
          unit = 1.f;
        }
      }
      const float shift = __builtin_amdgcn_logf(unit) - m;
      // each weight as the sum of two fp16 numbers, as in the row tiles: with one,
      // the error against 64 bits was 1.1 to 1.35 times that of the output's own
      // rounding.  The second product costs 547 to 700 us for 2048 tokens after
      // 6001 and 78 to 88 us for 32 prompts, wherever it is placed among the other
      // instructions.  The rest of a weight is one mixed-precision fma, for which
      // the factor -1 must not look like a constant.
      float sum = 0.f;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        half8 p, rest;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * tt + j], ck, shift));
          const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * tt + j + 1], ck, shift));
          sum += e0;
          sum += e1;
          const half2v two = __builtin_convertvector(float2v{e0, e1}, half2v);
          p[j] = two[0];
          p[j + 1] = two[1];
          rest[j] = (_Float16)__builtin_fmaf((float)two[0], minus, e0);
          rest[j + 1] = (_Float16)__builtin_fmaf((float)two[1], minus, e1);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const half8 a = __builtin_bit_cast(half8, lds_v[buf][x][v_slot(b * 32 + vd, tt, h)]);
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, p, acc[b], 0, 0, 0);
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, rest, acc[b], 0, 0, 0);
        }
      }
      l = __builtin_fmaf(sum, __builtin_amdgcn_rcpf(unit), l);
      // a block whose range is NaN holds zero codes; the rows that see it are NaN
      if ((rk[x] != rk[x] || rv[x] != rv[x]) && seen) l = __uint_as_float(0x7FC00000u);
    }
    if (more) {
      stage(buf ^ 1, gb + NG);
      lds_barrier();
    }
    buf ^= 1;
  }
  l += __shfl_xor(l, 32);
  if (tile.splits > 1) {
    // one slot for each 16 rows, as the row tiles'
    const int64_t at = tile.part + (wave * 2 + (n >> 4)) * tile.splits + tile.split;
    float* part = A.part + (at * kv.n_kv + head) * kv_part_floats(D);
    const float f = ref / Code<CODE>::kTop;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *(float4v*)(part + (n & 15) * D + b * 32 + h * 16 + c * 4) =
            float4v{acc[b][4 * c] * f, acc[b][4 * c + 1] * f, acc[b][4 * c + 2] * f, acc[b][4 * c + 3] * f};
    if (h == 0) {
      part[kKvRows * D + 2 * (n & 15)] = m;
      part[kKvRows * D + 2 * (n & 15) + 1] = l;
    }
  } else if (r < packed) {
    int again = r;                               // r < packed here: its head is found again instead of kept
    asm("" : "+v"(again));
    _Float16* out =
        (_Float16*)A.out + (int64_t)(tile.row0 + pos - tile.start) * A.out_stride + (head * G + again % G) * D;
    const float f = ref / Code<CODE>::kTop / l;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        half8 y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (_Float16)(acc[b][8 * c + j] * f);
        *(half8*)(out + b * 32 + h * 16 + c * 8) = y;
      }
  }
}

// Joins the splits of a prompt tile, 16 rows of it at a time: one workgroup per row.  D / 4 threads read a
// split's row, so 1024 / D splits are read side by side and then joined in LDS.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_combine_kernel(KvAttend A) {
  constexpr int TR = D / 4, NS = kThreads / TR;
  __shared__ float lds_o[NS][D];
  __shared__ float lds_m[NS], lds_l[NS];
  const KvView& kv = A.kv;
  const int tid = threadIdx.x, orow = blockIdx.x % kKvRows, at = blockIdx.x / kKvRows;
  const KvTile tile = A.combine[at / kv.n_kv];
  const int head = at % kv.n_kv;
  const int G = kv.n_heads / kv.n_kv, gr = tile.tile * kKvRows + orow, side = tid / TR, d = tid % TR * 4;
  if (gr >= tile.rows * G) return;
  const int64_t step = kv.n_kv * kv_part_floats(D);
  const float* part = A.part + ((int64_t)tile.part * kv.n_kv + head) * kv_part_floats(D);
  float m = -FLT_MAX, l = 0.f;
  float4v o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = side; s < tile.splits; s += NS) {
    const float* ps = part + s * step;
    const float ms = ps[kKvRows * D + 2 * orow], ls = ps[kKvRows * D + 2 * orow + 1];
    const float4v x = *(const float4v*)(ps + orow * D + d);
    const float mn = fmaxf(m, ms), f = __builtin_amdgcn_exp2f(m - mn), fs = __builtin_amdgcn_exp2f(ms - mn);
    m = mn;
    l = l * f + ls * fs;
    o = o * f + x * fs;
  }
  *(float4v*)&lds_o[side][d] = o;
  if (d == 0) { lds_m[side] = m; lds_l[side] = l; }
  __syncthreads();
  if (side) return;
  float mm = lds_m[0];
#pragma unroll
  for (int s = 1; s < NS; ++s) mm = fmaxf(mm, lds_m[s]);
  float ll = 0.f;
  o = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const float f = __builtin_amdgcn_exp2f(lds_m[s] - mm);
    ll += f * lds_l[s];
    o += f * *(const float4v*)&lds_o[s][d];
  }
  _Float16* out = (_Float16*)A.out + (int64_t)(tile.row0 + gr / G) * A.out_stride + (head * G + gr % G) * D + d;
  const float inv = 1.f / ll;
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = (_Float16)(o[j] * inv);
}

// ---------------------------------------------------------------------------
// Reading back: one workgroup per touched block and kv head.  A thread takes 8
// elements of a token from K, and a 16-byte unit of V, turned across four lanes
// into 8 elements of each of two tokens, so that stores are 16 bytes a lane and
// 64 bytes or more a run.  Nothing here reads them again: non-temporal stores
// took 8 sequences of up to 4000 tokens from 22.0 to 18.2 us (now 17.8, 5.2 TB/s).
// fp32 rows are stored in two halves of every 32 bytes, which such stores do not
// merge (3.2 TB/s against 4.6 when both were tried); the same sequences in fp32 take
// 37 us (4.2 TB/s).

// Fp32 values are multiplied in 64 bits, where the unit of a small range is as
// exact as any: in fp32, ranges below 127 times the smallest number read as 0.
template <typename T> struct Unit { typedef float type; };
template <> struct Unit<float> { typedef double type; };

template <typename T, int CODE>
__device__ __forceinline__ void put8(T* p, uint32_t a, uint32_t b, typename Unit<T>::type unit) {
  typename Vec<T>::v8 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = (T)(Code<CODE>::value((a >> (8 * j)) & 0xFF) * unit);
    y[4 + j] = (T)(Code<CODE>::value((b >> (8 * j)) & 0xFF) * unit);
  }
  if (sizeof(T) == 2) __builtin_nontemporal_store(y, reinterpret_cast<typename Vec<T>::v8*>(p));
  else *reinterpret_cast<typename Vec<T>::v8*>(p) = y;
}

template <typename T, int CODE>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvRead R) {
  using C = Code<CODE>;
  const KvView& kv = R.kv;
  const int dim = kv.dim, tid = threadIdx.x, lane = tid & 63;
  const KvBlock blk = R.blocks[blockIdx.x / kv.n_kv];
  const int head = blockIdx.x % kv.n_kv;
  const int32_t page = kv_row(kv, blk.seq, R.layer, head)[blk.block];
  const uint8_t* kbase = (const uint8_t*)kv.base + (int64_t)page * kv.page_bytes;
  const uint8_t* vbase = kbase + (int64_t)kv.block * dim;
  const float* range = kv.range + 2 * (int64_t)page;
  const int64_t row0 = (int64_t)blk.row - blk.slot0;
  const int ush = 27 - __clz(dim), g = lane >> 4, quad = (lane >> 2) & 3, k4 = lane & 3;
  const int group0 = blk.slot0 >> 5, group1 = (blk.slot1 + 31) >> 5;
  const int units_k = R.k ? (blk.slot1 - blk.slot0) << (ush + 1) : 0;
  const int units_v = R.v ? (group1 - group0) << (ush + 5) : 0;             // a multiple of 64: whole waves
  T* kout = (T*)R.k + (int64_t)head * dim;
  T* vout = (T*)R.v + (int64_t)head * dim;
  // four units of K and two of V a thread at a time, all loaded before the first is used
  for (int u0 = 0; u0 < max(units_k, 2 * units_v); u0 += 4 * kThreads) {
    uint2 kw[4];
    uint4 vw[2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int u = u0 + tid + n * kThreads;
      if (u < units_k)
        kw[n] = *reinterpret_cast<const uint2*>(
            kbase + kv_k_byte(blk.slot0 + (u >> (ush + 1)), (u & ((2 << ush) - 1)) * 8, dim));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int u = u0 / 2 + tid + n * kThreads;
      if (u < units_v)
        vw[n] = ld16(vbase + ((int64_t)(group0 + (u >> (ush + 5))) << (ush + 9)) +
                     ((u >> 6) & ((1 << (ush - 1)) - 1)) * 1024 + lane * 16);
    }
    typedef typename Unit<T>::type U;
    const U uk = (U)range[0] / C::kTop, uv = (U)range[1] / C::kTop;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int u = u0 + tid + n * kThreads;
      if (u < units_k)
        put8<T, CODE>(kout + (row0 + blk.slot0 + (u >> (ush + 1))) * R.k_stride + (u & ((2 << ush) - 1)) * 8, kw[n].x,
                      kw[n].y, uk);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int u = u0 / 2 + tid + n * kThreads;
      if (u < units_v) {
        const int group = group0 + (u >> (ush + 5)), e = (u >> 6) & ((1 << (ush - 1)) - 1);
        const uint32_t even[2] = {quad_transpose(vw[n].x, lane), quad_transpose(vw[n].y, lane)};
        const uint32_t odd[2] = {quad_transpose(vw[n].z, lane), quad_transpose(vw[n].w, lane)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int slot = group * 32 + h * 16 + g * 4 + k4;
          if (slot >= blk.slot0 && slot < blk.slot1)
            put8<T, CODE>(vout + (row0 + slot) * R.v_stride + e * 32 + quad * 8,
                          __builtin_amdgcn_perm(odd[h], even[h], 0x05010400u),
                          __builtin_amdgcn_perm(odd[h], even[h], 0x07030602u), uv);
        }
      }
    }
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
         : dim == 128 ? (const void*)kv_attend_rows_kernel<T, CODE, 128>
                      : (const void*)kv_attend_rows_kernel<T, CODE, 256>;
}
template <typename T>
static const void* rows_of(int code, int dim) {
  return code == SLORA_KV_INT8 ? rows_of<T, SLORA_KV_INT8>(dim) : rows_of<T, SLORA_KV_FP8>(dim);
}
template <int CODE>
static const void* prompt_of(int dim, bool triple) {
  return dim == 64 ? (const void*)kv_attend_prompt_kernel<CODE, 64, false>
         : dim == 256 ? (const void*)kv_attend_prompt_kernel<CODE, 256, false>
         : triple ? (const void*)kv_attend_prompt_kernel<CODE, 128, true>
                  : (const void*)kv_attend_prompt_kernel<CODE, 128, false>;
}
static const void* combine_of(int dim) {
  return dim == 64 ? (const void*)kv_combine_kernel<64>
         : dim == 128 ? (const void*)kv_combine_kernel<128> : (const void*)kv_combine_kernel<256>;
}

hipError_t launch_kv_append(const KvAppend& A0, hipStream_t stream) {
  KvAppend A = A0;
  const int64_t items = ((int64_t)A.n_small * A.kv.n_kv + 3) / 4 + 2 * (int64_t)(A.n_blocks - A.n_small) * A.kv.n_kv;
  int64_t q = 0;
  if (A.q) {
    const int64_t chunks = (A.kv.n_heads + A.q_heads - 1) / A.q_heads;
    q = ((int64_t)A.n_rows * chunks * (A.kv.dim / 16) + kThreads - 1) / kThreads;
  }
  // workgroup b has q workgroups floor(b * share / 2^32) before it: with the
  // share rounded up, exactly q of all (there is always an item: q < all)
  A.q_share = (uint32_t)((((uint64_t)q << 32) + (uint64_t)(q + items) - 1) / (uint64_t)(q + items));
  return run(A.kv.dtype == SLORA_F16 ? append_of<_Float16>(A.kv.code) : append_of<float>(A.kv.code), q + items, A,
             stream);
}

hipError_t launch_kv_attend(const KvAttend& A, hipStream_t stream) {
  const bool half = A.kv.dtype == SLORA_F16;
  // Heads of 128 run two workgroups a CU that stage 64 keys at a time, or three
  // that stage 32.  What counts is how often the places of the chip fill: three
  // where that saves a round, two, which are faster each, where it does not.
  // us with two | three, 32 query and kv heads, prompts of 512 tokens, n of them
  // (n / 2 workgroups a CU): 4: 27.7 | 30.9, 6: 39.5 | 33.9, 8: 46.0 | 45.2, 10:
  // 55 | 53, 14: 74 | 67, 16: 79 | 74, 32: 163 | 157; 32 prompts of 64 to 512
  // (11.1 a CU): 86 | 77; with 64 query and 8 kv heads 2048 tokens after 6001 (4 a
  // CU): 684 | 719, 512 after 16000 (4 a CU): 433 | 451; against the rule, with 32
  // and 8 heads one prompt of 4096 (5 a CU): 239 | 247.
  const int64_t prompts = (int64_t)A.n_prompts * A.kv.n_kv;
  const bool triple = (prompts - 1) / (3 * kKvCus) < (prompts - 1) / (2 * kKvCus);
  hipError_t e = run(A.kv.code == SLORA_KV_INT8 ? prompt_of<SLORA_KV_INT8>(A.kv.dim, triple)
                                                : prompt_of<SLORA_KV_FP8>(A.kv.dim, triple),
                     prompts, A, stream);
  if (e != hipSuccess) return e;
  e = run(half ? rows_of<_Float16>(A.kv.code, A.kv.dim) : rows_of<float>(A.kv.code, A.kv.dim),
                     (int64_t)A.n_tiles * A.kv.n_kv, A, stream);
  if (e != hipSuccess) return e;
  return run(combine_of(A.kv.dim), (int64_t)A.n_combine * A.kv.n_kv * kKvRows, A, stream);
}

hipError_t launch_kv_read(const KvRead& R, hipStream_t stream) {
  return run(R.kv.dtype == SLORA_F16 ? read_of<_Float16>(R.kv.code) : read_of<float>(R.kv.code),
             (int64_t)R.n_blocks * R.kv.n_kv, R, stream);
}

}  // namespace slora
