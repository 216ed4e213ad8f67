// Internal interface between the KV cache's host side (slora_kv_host.cpp) and
// its kernels (slora_kv.hip): the records of a step and the launches.
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "slora_internal.h"

namespace slora {

constexpr int kKvGroup = 32;      // tokens of one attention step: block_tokens is a multiple
constexpr int kKvRows = 16;       // query rows of one row tile
constexpr int kKvCus = 256;       // compute units of an MI355X
constexpr int kKvPromptRows = 128;   // query rows of one prompt tile

// Page layout (one block of one kv head): the K codes, then the V codes, both
// in the order in which the 16x16x32 matrix instruction takes them, so that
// every lane reads 16 contiguous bytes and a wave 1 KiB.
//  K: per 16 tokens and 64 elements of the head, 16 rows (tokens) of 64 bytes.
//  V: per 32 tokens and 32 elements, 64 lanes of 16 bytes; lane (g, i) = 16 g + i
//     holds, for elements 2i and 2i + 1, the 8 tokens 4g .. 4g+3 and
//     16 + 4g .. 16 + 4g+3: the tokens whose softmax weights lane (g, *) holds
//     after the K product, which therefore feed the V product from registers.
inline constexpr int64_t kv_k_byte(int slot, int d, int dim) {
  return (int64_t)(slot >> 4) * 16 * dim + (d >> 6) * 1024 + (slot & 15) * 64 + (d & 63);
}

struct KvView {
  char* base;              // pages of the class
  int64_t page_bytes;
  const int32_t* table;    // [max_seqs][n_layers][n_kv][max_blocks] page ids
  float* range;            // [n_pages][2]: of the keys, of the values
  int32_t dtype, code, n_layers, n_heads, n_kv, dim, block, max_blocks, rot, pairs;
};

// Records of a step (device metadata, int32 words).
// A touched block: sequence id, block, its slots [slot0, slot1) among the rows, batch row of slot0.
struct KvBlock { int32_t seq, block, slot0, slot1, row, pad[3]; };
// A tile of a sequence's packed rows: number, key split of how many, slots (see below); and the sequence: its first
// row's position, its rows, the batch row of the first.
struct KvTile { int32_t seq, tile, split, splits, part, start, rows, row0; };
struct KvPatch { uint32_t lo, hi; int32_t page, pad; };      // page table entry (hi:lo) = page

// A tile whose keys are split writes, per kv head, kKvRows x dim fp32 sums and
// kKvRows (maximum, sum) pairs to slot (part + split) * n_kv + head.  The last
// workgroup of a row tile joins its slots, by the counter at part * n_kv + head;
// a prompt tile has the slots of its eight runs of 16 rows one after another,
// and a combine entry (split 0) for each.
constexpr int64_t kv_part_floats(int dim) { return (int64_t)kKvRows * (dim + 2); }

struct KvAppend {
  KvView kv;
  const KvBlock* blocks;      // n_small blocks that gain one token, then the others
  int32_t n_blocks, n_small, n_rows, layer;
  int32_t q_heads;            // heads a thread rotates
  uint32_t q_share;           // workgroups of q among all, of 2^32 (set by the launch)
  const void* q; void* q_out; const void* k; const void* v;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  const float* cos_sin;
  const int32_t* row_pos;     // [n_rows] position of every row
};

struct KvAttend {
  KvView kv;
  const KvTile* prompts;      // tiles of a long run of rows (fp16)
  const KvTile* tiles;        // row tiles
  const KvTile* combine;      // of split prompt tiles
  uint32_t* counters;         // of split row tiles: zero before and after every launch
  int32_t n_prompts, n_tiles, n_combine, layer, window;
  const void* q; void* out;
  int64_t q_stride, out_stride;
  float scale_log2;           // scale * log2(e)
  float* part;
};

struct KvRead {
  KvView kv;
  const KvBlock* blocks;
  int32_t n_blocks, layer;
  void* k; void* v;
  int64_t k_stride, v_stride;
};

hipError_t launch_kv_patch(int32_t* table, const KvPatch* patches, int32_t n, hipStream_t stream);
hipError_t launch_kv_append(const KvAppend& A, hipStream_t stream);
hipError_t launch_kv_attend(const KvAttend& A, hipStream_t stream);
hipError_t launch_kv_read(const KvRead& R, hipStream_t stream);

}  // namespace slora
