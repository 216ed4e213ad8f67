// Host side of the 8-bit paged KV cache (include/slora.h, "KV cache in the
// pool"): sequences and their pages, the steps of a batch with their work
// lists, and the C ABI.  Pages come from the pool's own allocator, so adapters
// and KV blocks compete for the same memory (summary page "S-LoRA: Serving
// Thousands of Concurrent LoRA Adapters", "Unified Paging").
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <numeric>
#include <string>
#include <vector>

#include "slora.h"
#include "slora_kv.h"

using namespace slora;

namespace {

slora_status fail(slora_status st, const std::string& msg) {
  set_last_error(msg.c_str());
  return st;
}

struct Seq {
  int64_t len = 0;
  int32_t blocks = 0;      // blocks of one layer and head
  int32_t entered = 0;     // of these, in the device's page table
  uint64_t gen = 0;        // counts drops
  std::vector<int32_t> held;    // [block] record of its pages
  std::vector<int32_t> stored;  // [block][layer] tokens that appends have been launched for
  // from token first on, the rotation's position is the token's number + shift (no runs: 0)
  struct Run { int32_t first, shift; };
  std::vector<Run> runs;
  int32_t shift() const { return runs.empty() ? 0 : runs.back().shift; }
};

// The pages of blocks, [layer][head] of each, and how many sequences hold it.  A
// block that more than one holds is full, and nothing writes to it.
struct Blocks {
  std::vector<int32_t> pages, refs, spare;
  size_t room = 0;
  // Room for n more, after which add and release cannot fail.
  void reserve(int64_t n, int64_t per) {
    const size_t want = refs.size() + (size_t)std::max<int64_t>(0, n - (int64_t)spare.size());
    if (want <= room) return;
    const size_t grown = std::max(want, 2 * room);
    pages.reserve(grown * (size_t)per);
    spare.reserve(grown);
    refs.reserve(grown);
    room = grown;
  }
  int32_t add(const int32_t* ids, int64_t per) {
    int32_t at = (int32_t)refs.size();
    if (spare.empty()) {
      refs.push_back(1);
      pages.insert(pages.end(), ids, ids + per);
    } else {
      at = spare.back();
      spare.pop_back();
      refs[at] = 1;
      std::copy(ids, ids + per, pages.begin() + at * per);
    }
    return at;
  }
  // Whether the last holder let go of it.
  bool release(int32_t at) {
    if (--refs[at]) return false;
    spare.push_back(at);
    return true;
  }
};

constexpr int64_t kMostPositions = (int64_t)1 << 30;
// a launch holds fewer than 2^32 threads, and counts in the kernels are 31 bits
constexpr int64_t kMostGroups = ((int64_t)1 << 32) / kThreads - 1;

// Checks a description against a pool; the block size and blocks of the
// longest sequence on success, a message otherwise.
const char* check_desc(const slora_pool* pool, const slora_kv_desc* d, PoolInfo* info, int32_t* block,
                       int32_t* max_blocks) {
  if (!pool || !d) return "NULL argument";
  pool_info(pool, info);
  if (d->cls < 0 || d->cls >= info->n_classes) return "bad page class";
  if (d->code != SLORA_KV_INT8 && d->code != SLORA_KV_FP8) return "code must be SLORA_KV_INT8 or SLORA_KV_FP8";
  if (d->n_layers < 1 || d->n_layers > 1024) return "n_layers must be 1..1024";
  if (d->n_heads < 1 || d->n_heads > 1024) return "n_heads must be 1..1024";
  if (d->n_kv_heads < 1 || d->n_heads % d->n_kv_heads) return "n_heads must be a multiple of n_kv_heads";
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return "head_dim must be 64, 128 or 256";
  if (d->max_seqs < 1 || d->max_tokens < 1) return "max_seqs and max_tokens must be positive";
  if (d->max_tokens > (1 << 30)) return "max_tokens must be at most 2^30";
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16)
    return "rot_dim must be a multiple of 16 up to head_dim";
  if (d->rot_pairs != SLORA_KV_HALVES && d->rot_pairs != SLORA_KV_NEIGHBOURS)
    return "rot_pairs must be SLORA_KV_HALVES or SLORA_KV_NEIGHBOURS";
  if (d->reserved0 != 0) return "reserved0 must be 0";
  const int64_t most = info->page_bytes[d->cls] / (2 * d->head_dim) / kKvGroup * kKvGroup;
  if (most < kKvGroup) return "a page of this class holds fewer than 32 tokens of a head";
  if (d->block_tokens < 0 || d->block_tokens % kKvGroup || d->block_tokens > most)
    return "block_tokens must be a multiple of 32 that a page of this class holds (0: the most)";
  *block = d->block_tokens ? d->block_tokens : (int32_t)most;
  *max_blocks = (d->max_tokens + *block - 1) / *block;
  const double entries = (double)d->max_seqs * d->n_layers * d->n_kv_heads * *max_blocks;
  if (entries > 1e15) return "the page table would not fit";
  return nullptr;
}

size_t table_bytes(const slora_kv_desc& d, int32_t max_blocks) {
  const size_t n = (size_t)d.max_seqs * d.n_layers * d.n_kv_heads * max_blocks * sizeof(int32_t);
  return (n + 15) / 16 * 16;
}

}  // namespace

struct slora_kv {
  slora_pool* pool = nullptr;
  slora_kv_desc d{};
  PoolInfo info{};
  int32_t block = 0, max_blocks = 0;
  char* dev = nullptr;
  std::vector<Seq> seqs;
  Blocks blocks;

  const int32_t* pages_of(int32_t record) const { return blocks.pages.data() + record * per_block(); }
  int32_t elem() const { return info.dtype == SLORA_F16 ? 2 : 4; }
  int64_t per_block() const { return (int64_t)d.n_layers * d.n_kv_heads; }
  int32_t* table() const { return reinterpret_cast<int32_t*>(dev); }
  KvView view() const {
    KvView v{};
    v.base = info.base[d.cls];
    v.page_bytes = info.page_bytes[d.cls];
    v.table = table();
    v.range = reinterpret_cast<float*>(dev + table_bytes(d, max_blocks));
    v.dtype = info.dtype;
    v.code = d.code;
    v.n_layers = d.n_layers;
    v.n_heads = d.n_heads;
    v.n_kv = d.n_kv_heads;
    v.dim = d.head_dim;
    v.block = block;
    v.max_blocks = max_blocks;
    v.rot = d.rot_dim;
    v.pairs = d.rot_pairs;
    return v;
  }
};

// A sequence's part in a step: its id, the position of its first row, its rows
// and the batch row of the first.
struct StepSeq { int32_t seq, start, rows, row0; };

struct slora_kv_step {
  slora_kv* kv = nullptr;
  bool reread = false;
  std::vector<StepSeq> seqs;
  std::vector<uint64_t> gens;
  std::vector<int32_t> ends;       // blocks of each sequence at the end of the step
  std::vector<KvBlock> blocks;
  std::vector<int32_t> row_pos;
  std::vector<KvTile> prompts, tiles, combine;
  std::vector<KvPatch> patches;
  int32_t n_rows = 0, max_len = 0, n_small = 0;
  int32_t n_positions = 0;         // one more than the rows' largest position
  int64_t n_new_pages = 0;
  int64_t n_parts = 0, n_row_parts = 0;   // slots of split tiles, those of row tiles first
  const char* dev = nullptr;

  // byte offsets in the device metadata (every record is 16 bytes or more)
  size_t prompts_off() const { return blocks.size() * sizeof(KvBlock); }
  size_t tiles_off() const { return prompts_off() + prompts.size() * sizeof(KvTile); }
  size_t patches_off() const { return tiles_off() + (tiles.size() + combine.size()) * sizeof(KvTile); }
  size_t row_pos_off() const { return patches_off() + patches.size() * sizeof(KvPatch); }
  size_t counters_off() const { return row_pos_off() + row_pos.size() * sizeof(int32_t); }
  size_t bytes() const { return counters_off() + (size_t)n_row_parts * kv->d.n_kv_heads * sizeof(uint32_t); }
  size_t workspace() const {
    return (size_t)n_parts * kv->d.n_kv_heads * kv_part_floats(kv->d.head_dim) * sizeof(float);
  }
};

namespace {

// Row tiles: key groups of 32 a workgroup takes at least, and the workgroups a
// launch is split into at most.  us with at least 4 | 8 | 16 groups: one token
// after 777, 64 heads of 128 on 8, 8.1 | 7.9 | 9.7, 16 fp32 heads of 128 10.4 |
// 12.6 | 20.4; one after 32000 51 | 42 | 29, where the join of the splits counts.
// us with at most 1024 | 1536 | 2560 | 3840 workgroups, which is 1.3 to 5 times
// the places of the chip for heads of 128: 12 conversations of 12000 to 33000
// tokens, heads of 64 55 | 60 | 62 | 65, of 128 108 | 109 | 112 | 120, of 256 199 |
// 205 | 214 | 227; 32 requests of 1000 to 3000, 32 heads on 8, of 64 18 | 20 | 21 |
// 21, of 128 32 | 33 | 35 | 35, of 256 56 | 60 | 64 | 64.
constexpr int64_t kMinGroups = 8, kWantGroups = 1536;
// Steps cut for a window: three workgroups a CU (heads of 256: two), a round of the
// chip's places for heads of 128.  (Heads of 64 have four places a CU, fp32 e4m3 ones of
// 128 with first tokens two; the rule leaves that out.)  us with at most 1536 | 768 | 512 workgroups, window
// 4096, 8 requests, 32 heads on 8, of 64 14.7 | 12.9 | 13.2, of 128 22.3 | 18.9 | 18.9,
// of 256 39.3 | 36.6 | 30.2, fp32 of 128 39.7 | 35.9 | 39.2; window 1024, 64 requests,
// of 128 34.2 | 27.8 | 27.8, of 256 62.7 | 48.7 | 48.7; one request alike.
constexpr int64_t window_groups(int32_t dim) { return dim == 256 ? 512 : 768; }

// Sequences with at least kPromptMin packed rows (query heads of a kv head times
// rows), or kFreshMin where nothing was cached before them, take the prompt tiles
// (fp16), which do the work of 128 rows however few there are.  Row | prompt
// tiles, us, heads of 128: 16 sequences of 1000 tokens, 32 heads, 48 more rows 53
// | 102, 64: 69 | 99, 96: 93 | 104, 128: 119 | 115, 160: 146 | 123; of 2000 tokens
// 64: 125 | 146, 96: 173 | 162; with 32 heads on 8 16 rows 40 | 46, 28: 53 | 51;
// 32 fresh prompts of 48 rows 18 | 16, 64: 23 | 17, 96: 33 | 24.  The rule leaves
// out how many sequences there are: one with 24 rows after 1000 tokens takes 9 |
// 25, after 20000 tokens 59 | 42; a single token of 96 query heads a kv head 9 | 22
// after 800 tokens, 74 | 32 after 20000, for 32 such requests of 2000 54 | 56.
// Their keys are split only where a launch has fewer tiles than kWantPrompts, two
// rounds of two workgroups a CU: a workgroup takes at least kPromptGroups groups.
constexpr int64_t kPromptMin = 96, kFreshMin = 48, kPromptGroups = 16, kWantPrompts = 1024;

// Tiles of 128 packed rows for long runs of rows (fp16), and row tiles of 16 for
// the others, with their key splits, longest first.  Splits are cut for a window
// (0: none) and the first `sinks` tokens.
void build_tiles(slora_kv_step* st, int32_t window, int32_t sinks) {
  const slora_kv_desc& d = st->kv->d;
  const int32_t G = d.n_heads / d.n_kv_heads;
  const bool half = st->kv->info.dtype == SLORA_F16;
  auto prompt = [&](const StepSeq& s) { return half && (int64_t)s.rows * G >= (s.start ? kPromptMin : kFreshMin); };
  // key groups that the tile of packed rows [r0, r0 + n) sees
  auto groups_of = [&](const StepSeq& s, int64_t r0, int64_t n) {
    const int64_t last = (s.start + (std::min<int64_t>(r0 + n, (int64_t)s.rows * G) - 1) / G) / kKvGroup + 1;
    if (!window) return last;
    const int64_t first = std::max<int64_t>(0, s.start + r0 / G - window + 1) / kKvGroup;
    return last - first + std::min<int64_t>(((int64_t)sinks + kKvGroup - 1) / kKvGroup, first);
  };
  // groups of a workgroup: the fewest for which all row tiles' workgroups are at most `want`
  const int64_t want = window ? window_groups(d.head_dim) : kWantGroups;
  std::vector<int64_t> lens;
  for (const StepSeq& s : st->seqs)
    for (int64_t r0 = 0; !prompt(s) && r0 < (int64_t)s.rows * G; r0 += kKvRows)
      lens.push_back(groups_of(s, r0, kKvRows));
  int64_t chunk = kMinGroups;
  if (!lens.empty()) {
    int64_t high = std::max(chunk, *std::max_element(lens.begin(), lens.end()));
    while (chunk < high) {
      const int64_t mid = (chunk + high) / 2;
      int64_t wgs = 0;
      for (int64_t n : lens) wgs += (n + mid - 1) / mid;
      if (wgs * d.n_kv_heads <= want) high = mid;
      else chunk = mid + 1;
    }
  }
  // longest first
  std::vector<std::pair<int64_t, KvTile>> found;
  auto take = [&](std::vector<KvTile>* to) {
    std::stable_sort(found.begin(), found.end(), [](const auto& a, const auto& b) { return a.first > b.first; });
    for (const auto& t : found) to->push_back(t.second);
    found.clear();
  };
  for (const StepSeq& s : st->seqs) {
    if (prompt(s)) continue;
    for (int64_t t = 0; t * kKvRows < (int64_t)s.rows * G; ++t) {
      const int64_t groups = groups_of(s, t * kKvRows, kKvRows);
      const int32_t splits = (int32_t)((groups + chunk - 1) / chunk);
      for (int32_t k = 0; k < splits; ++k)
        found.push_back({(groups + splits - 1) / splits,
                         {s.seq, (int32_t)t, k, splits, (int32_t)st->n_parts, s.start, s.rows, s.row0}});
      if (splits > 1) st->n_parts += splits;
    }
  }
  take(&st->tiles);
  st->n_row_parts = st->n_parts;

  int64_t total = 0;
  for (const StepSeq& s : st->seqs)
    for (int64_t r0 = 0; prompt(s) && r0 < (int64_t)s.rows * G; r0 += kKvPromptRows)
      total += groups_of(s, r0, kKvPromptRows);
  const int64_t most = std::max<int64_t>(kPromptGroups, (total * d.n_kv_heads + kWantPrompts - 1) / kWantPrompts);
  constexpr int32_t kRuns = kKvPromptRows / kKvRows;
  for (const StepSeq& s : st->seqs) {
    const int64_t packed = (int64_t)s.rows * G;
    if (!prompt(s)) continue;
    for (int64_t t = 0; t * kKvPromptRows < packed; ++t) {
      const int64_t groups = groups_of(s, t * kKvPromptRows, kKvPromptRows);
      const int32_t splits = (int32_t)std::max<int64_t>(1, (groups + most / 2) / most);
      for (int32_t k = 0; k < splits; ++k)
        found.push_back({(groups + splits - 1) / splits,
                         {s.seq, (int32_t)t, k, splits, (int32_t)st->n_parts, s.start, s.rows, s.row0}});
      if (splits == 1) continue;
      for (int32_t run = 0; run < kRuns && t * kKvPromptRows + run * kKvRows < packed; ++run)
        st->combine.push_back({s.seq, (int32_t)t * kRuns + run, 0, splits, (int32_t)st->n_parts + run * splits, s.start,
                               s.rows, s.row0});
      st->n_parts += (int64_t)splits * kRuns;
    }
  }
  take(&st->prompts);
}

slora_status check_launch(const std::string& f, const slora_kv* kv, const slora_kv_step* st, int32_t layer) {
  if (!kv || !st) return fail(SLORA_E_INVAL, f + ": NULL cache or step");
  if (st->kv != kv) return fail(SLORA_E_INVAL, f + ": the step belongs to another cache");
  if (layer < 0 || layer >= kv->d.n_layers) return fail(SLORA_E_INVAL, f + ": layer out of range");
  for (size_t i = 0; i < st->seqs.size(); ++i)
    if (kv->seqs[st->seqs[i].seq].gen != st->gens[i])
      return fail(SLORA_E_STALE,
                  f + ": sequence " + std::to_string(st->seqs[i].seq) + " was dropped since the step was built");
  return SLORA_OK;
}

// Pointer and stride of a [n_rows][heads][head_dim] operand.
slora_status check_rows(const std::string& f, const char* name, const slora_kv* kv, const void* p, int64_t stride,
                        int32_t heads) {
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(SLORA_E_INVAL, f + ": " + name + " must be 16-byte aligned");
  if (stride < (int64_t)heads * kv->d.head_dim || stride * kv->elem() % 16 || stride > ((int64_t)1 << 40))
    return fail(SLORA_E_INVAL,
                f + ": the stride of " + name + " must be at least heads * head_dim and a multiple of 16 bytes");
  return SLORA_OK;
}

// A range stands for its whole block, so tokens enter a block in their order: an
// append takes up where the last one of the layer ended, or repeats it.
slora_status check_order(const std::string& f, const slora_kv* kv, const slora_kv_step* st, int32_t layer) {
  for (const KvBlock& b : st->blocks) {
    const int32_t have = kv->seqs[b.seq].stored[(size_t)b.block * kv->d.n_layers + layer];
    if (have < b.slot0)
      return fail(SLORA_E_INVAL, f + ": earlier tokens of a block have not been appended in this layer");
    if (have > b.slot1)
      return fail(SLORA_E_INVAL, f + ": later tokens of a block have been appended in this layer");
    if (kv->blocks.refs[kv->seqs[b.seq].held[b.block]] > 1)
      return fail(SLORA_E_INVAL, f + ": another sequence shares a block of the step");
  }
  return SLORA_OK;
}

slora_status launched(const std::string& f, hipError_t e) {
  if (e == hipSuccess) return SLORA_OK;
  return fail(SLORA_E_HIP, f + " launch: " + hipGetErrorString(e));
}

// An append, with the norms of q and k where norm is given.
slora_status append(const std::string& f, slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q,
                    int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, const slora_kv_norm* norm, const float* cos_sin, int64_t n_positions,
                    void* stream) {
  slora_status ok = check_launch(f, kv, st, layer);
  if (ok != SLORA_OK) return ok;
  if (st->reread) return fail(SLORA_E_INVAL, f + ": a reread step has no new tokens");
  if (st->n_rows == 0) return SLORA_OK;
  if (!k || !v) return fail(SLORA_E_INVAL, f + ": NULL k or v");
  if (!q != !q_out) return fail(SLORA_E_INVAL, f + ": q and q_out must be given together");
  if ((ok = check_rows(f, "k", kv, k, k_stride, kv->d.n_kv_heads)) != SLORA_OK) return ok;
  if ((ok = check_rows(f, "v", kv, v, v_stride, kv->d.n_kv_heads)) != SLORA_OK) return ok;
  if (q) {
    if ((ok = check_rows(f, "q", kv, q, q_stride, kv->d.n_heads)) != SLORA_OK) return ok;
    if ((ok = check_rows(f, "q_out", kv, q_out, q_out_stride, kv->d.n_heads)) != SLORA_OK) return ok;
    if (q == q_out && q_stride != q_out_stride) return fail(SLORA_E_INVAL, f + ": q_out is q with another stride");
  }
  if (kv->d.rot_dim) {
    if (!cos_sin || reinterpret_cast<uintptr_t>(cos_sin) & 15)
      return fail(SLORA_E_INVAL, f + ": cos_sin must be non-NULL and 16-byte aligned");
    if (n_positions < st->n_positions)
      return fail(SLORA_E_INVAL, f + ": cos_sin does not hold every position of the step");
  }
  if ((ok = check_order(f, kv, st, layer)) != SLORA_OK) return ok;
  if (!st->dev) return fail(SLORA_E_INVAL, f + ": step not uploaded (call slora_kv_step_upload)");
  if ((ok = pool_device_current(kv->pool)) != SLORA_OK) return ok;
  KvAppend A{};
  A.kv = kv->view();
  A.blocks = reinterpret_cast<const KvBlock*>(st->dev);
  A.n_blocks = (int32_t)st->blocks.size();
  A.n_small = st->n_small;
  A.n_rows = st->n_rows;
  // enough threads for about eight waves a SIMD; beyond that, more heads a thread
  const int64_t units = (int64_t)st->n_rows * kv->d.n_heads * kv->d.head_dim / 16;
  A.q_heads = (int32_t)std::min<int64_t>(8, std::max<int64_t>(1, units / (1 << 19)));
  A.layer = layer;
  A.q = q;
  A.q_out = q_out;
  A.k = k;
  A.v = v;
  A.q_stride = q_stride;
  A.q_out_stride = q_out_stride;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  A.cos_sin = cos_sin;
  A.row_pos = reinterpret_cast<const int32_t*>(st->dev + st->row_pos_off());
  if (norm) {
    A.q_weight = norm->q_weight;
    A.k_weight = norm->k_weight;
    A.eps = norm->eps;
    A.w_mean = 1.f / (float)kv->d.head_dim;
    A.w_stride = norm->per_head ? kv->d.head_dim : 0;
  }
  ok = launched(f, launch_kv_append(A, norm != nullptr, static_cast<hipStream_t>(stream)));
  if (ok == SLORA_OK)
    for (const KvBlock& b : st->blocks) kv->seqs[b.seq].stored[(size_t)b.block * kv->d.n_layers + layer] = b.slot1;
  return ok;
}

slora_status attend(const std::string& f, slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q,
                    int64_t q_stride, void* out, int64_t out_stride, float scale, int32_t window, int32_t sinks,
                    void* workspace, size_t workspace_bytes, void* stream) {
  slora_status ok = check_launch(f, kv, st, layer);
  if (ok != SLORA_OK) return ok;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(SLORA_E_INVAL, f + ": scale times log2(e) must be finite in fp32");
  if (window < 0) return fail(SLORA_E_INVAL, f + ": window must be 0 (none) or positive");
  if (sinks < 0) return fail(SLORA_E_INVAL, f + ": sinks must be 0 or positive");
  if (st->n_rows == 0) return SLORA_OK;
  if (!q || !out) return fail(SLORA_E_INVAL, f + ": NULL q or out");
  if ((ok = check_rows(f, "q", kv, q, q_stride, kv->d.n_heads)) != SLORA_OK) return ok;
  if ((ok = check_rows(f, "out", kv, out, out_stride, kv->d.n_heads)) != SLORA_OK) return ok;
  if (st->workspace() > 0) {
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) & 15)
      return fail(SLORA_E_INVAL, f + ": workspace must be non-NULL and 16-byte aligned");
    if (workspace_bytes < st->workspace()) return fail(SLORA_E_NOMEM, f + ": workspace smaller than workspace_bytes");
  }
  if (!st->dev) return fail(SLORA_E_INVAL, f + ": step not uploaded (call slora_kv_step_upload)");
  if ((ok = pool_device_current(kv->pool)) != SLORA_OK) return ok;
  KvAttend A{};
  A.kv = kv->view();
  A.tiles = reinterpret_cast<const KvTile*>(st->dev + st->tiles_off());
  A.prompts = reinterpret_cast<const KvTile*>(st->dev + st->prompts_off());
  A.n_prompts = (int32_t)st->prompts.size();
  A.n_tiles = (int32_t)st->tiles.size();
  A.combine = A.tiles + A.n_tiles;
  A.counters = reinterpret_cast<uint32_t*>(const_cast<char*>(st->dev + st->counters_off()));
  A.n_combine = (int32_t)st->combine.size();
  A.layer = layer;
  A.window = window;
  A.sinks = window ? std::min(sinks, kv->d.max_tokens) : 0;    // without a window all are visible
  A.q = q;
  A.out = out;
  A.q_stride = q_stride;
  A.out_stride = out_stride;
  A.scale_log2 = scale_log2;
  A.part = static_cast<float*>(workspace);
  return launched(f, launch_kv_attend(A, static_cast<hipStream_t>(stream)));
}

// What a call of slora_kv_take does: the device's records, and what its sequences
// are afterwards.
struct TakePlan {
  struct Part {
    int32_t dst, src;
    int64_t len = 0;
    std::vector<int32_t> from;     // [block] the block of src whose pages it shares, or ~copy
    std::vector<Seq::Run> runs;
  };
  std::vector<Part> parts;
  std::vector<KvTakeRow> rows;
  std::vector<KvCopy> copies;
  std::vector<int32_t> entries, tokens;
  bool in_place = false;           // a launch of copies reads rows that the call changes
  int64_t per = 0;

  size_t copies_off() const { return rows.size() * sizeof(KvTakeRow); }
  size_t entries_off() const { return copies_off() + copies.size() * sizeof(KvCopy); }
  size_t tokens_off() const { return entries_off() + entries.size() * sizeof(int32_t); }
  size_t pages_off() const { return tokens_off() + tokens.size() * sizeof(int32_t); }
  size_t bytes() const { return pages_off() + copies.size() * (size_t)per * sizeof(int32_t); }
};

// The plan of a call; a message if it is refused.  (Throws std::bad_alloc.)
const char* plan_take(const slora_kv* kv, int32_t n, const int32_t* dst, const int32_t* src, const int32_t* n_ranges,
                      const int64_t* ranges, TakePlan* plan) {
  if (!kv || n < 0 || (n > 0 && (!dst || !src || !n_ranges))) return "NULL argument";
  plan->per = kv->per_block();
  std::vector<uint8_t> changed((size_t)kv->d.max_seqs, 0);
  for (int32_t i = 0; i < n; ++i) {
    if (dst[i] < 0 || dst[i] >= kv->d.max_seqs || src[i] < 0 || src[i] >= kv->d.max_seqs)
      return "sequence id out of range";
    if (changed[dst[i]]++) return "a sequence is made twice";
    if (n_ranges[i] < 0 || (n_ranges[i] > 0 && !ranges)) return "NULL or negative ranges";
  }
  const int32_t bt = kv->block, layers = kv->d.n_layers;
  int64_t at = 0;
  std::vector<std::pair<int64_t, int64_t>> kept;               // ranges, those that touch joined
  std::vector<int32_t> ready;                                  // [block] tokens of the source in every layer
  for (int32_t i = 0; i < n; ++i) {
    const bool same = dst[i] == src[i];
    if (!same && changed[src[i]]) return "the source of a sequence is changed by the same call";
    const Seq& s = kv->seqs[src[i]];
    if (!same && kv->seqs[dst[i]].blocks) return "a sequence that is made from another one must be empty";
    if (i == 0 || src[i] != src[i - 1]) {
      ready.resize((size_t)s.entered);
      for (int32_t b = 0; b < s.entered; ++b)
        ready[b] =
            *std::min_element(s.stored.begin() + (size_t)b * layers, s.stored.begin() + (size_t)(b + 1) * layers);
    }
    kept.clear();
    int64_t end = 0, b = 0;                                    // b: block of the range's first token
    TakePlan::Part part;
    part.runs.reserve((size_t)n_ranges[i]);
    kept.reserve((size_t)n_ranges[i]);
    part.dst = dst[i];
    part.src = src[i];
    for (int32_t r = 0; r < n_ranges[i]; ++r, ++at) {
      const int64_t lo = ranges[2 * at], hi = ranges[2 * at + 1];
      if (lo < end || hi < lo || hi > s.len) return "ranges must ascend within the sequence's tokens";
      end = hi;
      if (lo == hi) continue;
      while ((b + 1) * bt <= lo) ++b;
      for (;; ++b) {
        if (b >= s.entered) return "the step of a token has not been uploaded";
        if (ready[b] < std::min<int64_t>(bt, hi - b * bt)) return "a token has not been appended in every layer";
        if ((b + 1) * bt >= hi) break;
      }
      if (!kept.empty() && kept.back().second == lo) kept.back().second = hi;
      else kept.push_back({lo, hi});
    }
    // positions: the source's runs, cut by the ranges
    size_t run = 0;
    for (const auto& k : kept) {
      for (int64_t p = k.first; p < k.second;) {
        while (run + 1 < s.runs.size() && s.runs[run + 1].first <= p) ++run;
        const bool last = run + 1 >= s.runs.size();
        const int64_t stop = last ? k.second : std::min<int64_t>(k.second, s.runs[run + 1].first);
        // a run holds from its first token on, the first from token 0
        const int32_t shift = s.runs.empty() ? 0 : s.runs[run].shift;
        const Seq::Run made = {(int32_t)part.len, (int32_t)(p + shift - part.len)};
        if (part.runs.empty() || part.runs.back().shift != made.shift) part.runs.push_back(made);
        part.len += stop - p;
        p = stop;
      }
    }
    // blocks
    size_t k = 0;
    int64_t p = kept.empty() ? 0 : kept[0].first;
    part.from.reserve((size_t)((part.len + bt - 1) / bt));
    for (int64_t left = part.len; left > 0;) {
      const int64_t count = std::min<int64_t>(bt, left), block = p / bt;
      left -= count;
      const bool alike = p % bt == 0 && kept[k].second - p >= count;
      if (alike && (count == bt || (same && kv->blocks.refs[s.held[block]] == 1))) {
        part.from.push_back((int32_t)block);
        p += count;
      } else {
        part.from.push_back(~(int32_t)plan->copies.size());
        plan->copies.push_back({src[i], (int32_t)count, (int32_t)plan->tokens.size(), 0});
        if (same) plan->in_place = true;
        for (int64_t want = count; want > 0;) {
          const int64_t take = std::min(want, kept[k].second - p);
          plan->tokens.resize(plan->tokens.size() + (size_t)take);
          std::iota(plan->tokens.end() - take, plan->tokens.end(), (int32_t)p);
          want -= take;
          p += take;
          if (p == kept[k].second && want > 0) p = kept[++k].first;
        }
        if (plan->tokens.size() > (size_t)INT32_MAX / 2) return "the call is too large for one launch";
      }
      if (left > 0 && p == kept[k].second) p = kept[++k].first;
    }
    int32_t first = 0;                                         // what stays where it is
    const int32_t blocks = (int32_t)part.from.size();
    while (same && first < blocks && part.from[first] == first) ++first;
    if (first < blocks) {
      plan->rows.push_back({dst[i], src[i], first, blocks - first, (int32_t)plan->entries.size(), {0, 0, 0}});
      plan->entries.insert(plan->entries.end(), part.from.begin() + first, part.from.end());
    }
    plan->parts.push_back(std::move(part));
    if (plan->entries.size() > (size_t)INT32_MAX / 2) return "the call is too large for one launch";
  }
  if ((double)(plan->copies.size() + plan->rows.size()) * plan->per > kMostGroups ||
      (double)plan->copies.size() * plan->per > INT32_MAX / 2)
    return "the call is too large for one launch";
  return nullptr;
}

}  // namespace

extern "C" {

size_t slora_kv_device_bytes(const slora_pool* pool, const slora_kv_desc* desc) {
  PoolInfo info;
  int32_t block, max_blocks;
  if (const char* why = check_desc(pool, desc, &info, &block, &max_blocks)) {
    fail(SLORA_E_INVAL, std::string("slora_kv_device_bytes: ") + why);
    return 0;
  }
  return table_bytes(*desc, max_blocks) + (size_t)info.n_pages[desc->cls] * 2 * sizeof(float);
}

slora_status slora_kv_create(slora_pool* pool, const slora_kv_desc* desc, void* dev, size_t dev_bytes, slora_kv** out) {
  if (!out || !dev) return fail(SLORA_E_INVAL, "slora_kv_create: NULL argument");
  PoolInfo info;
  int32_t block, max_blocks;
  if (const char* why = check_desc(pool, desc, &info, &block, &max_blocks))
    return fail(SLORA_E_INVAL, std::string("slora_kv_create: ") + why);
  if (reinterpret_cast<uintptr_t>(dev) & 15) return fail(SLORA_E_INVAL, "slora_kv_create: dev must be 16-byte aligned");
  if (dev_bytes < slora_kv_device_bytes(pool, desc))
    return fail(SLORA_E_NOMEM, "slora_kv_create: dev smaller than slora_kv_device_bytes");
  slora_kv* kv = new (std::nothrow) slora_kv();
  if (!kv) return fail(SLORA_E_NOMEM, "slora_kv_create: out of host memory");
  try {
    kv->seqs.resize((size_t)desc->max_seqs);
  } catch (const std::bad_alloc&) {
    delete kv;
    return fail(SLORA_E_NOMEM, "slora_kv_create: out of host memory");
  }
  kv->pool = pool;
  kv->d = *desc;
  kv->info = info;
  kv->block = block;
  kv->max_blocks = max_blocks;
  kv->dev = static_cast<char*>(dev);
  *out = kv;
  return SLORA_OK;
}

slora_status slora_kv_drop(slora_kv* kv, int32_t seq) {
  if (!kv) return fail(SLORA_E_INVAL, "slora_kv_drop: NULL cache");
  if (seq < 0 || seq >= kv->d.max_seqs) return fail(SLORA_E_INVAL, "slora_kv_drop: sequence id out of range");
  Seq& s = kv->seqs[seq];
  try {
    std::vector<int32_t> alone;                                // pages that no other sequence holds
    for (int32_t record : s.held)
      if (kv->blocks.refs[record] == 1)
        alone.insert(alone.end(), kv->pages_of(record), kv->pages_of(record) + kv->per_block());
    slora_status st = slora_free_pages(kv->pool, kv->d.cls, (int64_t)alone.size(), alone.data());
    if (st != SLORA_OK) return st;
  } catch (const std::bad_alloc&) {
    return fail(SLORA_E_NOMEM, "slora_kv_drop: out of host memory");
  }
  for (int32_t record : s.held) (void)kv->blocks.release(record);
  s.held.clear();
  s.held.shrink_to_fit();
  s.stored.clear();
  s.runs.clear();
  s.len = 0;
  s.blocks = s.entered = 0;
  ++s.gen;
  return SLORA_OK;
}

void slora_kv_destroy(slora_kv* kv) {
  if (!kv) return;
  for (int32_t i = 0; i < kv->d.max_seqs; ++i)
    if (kv->seqs[i].blocks) (void)slora_kv_drop(kv, i);
  delete kv;
}

int64_t slora_kv_position(const slora_kv* kv, int32_t seq) {
  if (!kv || seq < 0 || seq >= kv->d.max_seqs) return -1;
  return kv->seqs[seq].len + kv->seqs[seq].shift();
}

int64_t slora_kv_length(const slora_kv* kv, int32_t seq) {
  if (!kv || seq < 0 || seq >= kv->d.max_seqs) return -1;
  return kv->seqs[seq].len;
}

slora_status slora_kv_pages(const slora_kv* kv, int32_t seq, int32_t layer, int32_t head, int32_t* ids, int32_t cap,
                            int32_t* n) {
  if (!kv || !n || cap < 0 || (cap > 0 && !ids)) return fail(SLORA_E_INVAL, "slora_kv_pages: NULL argument");
  if (seq < 0 || seq >= kv->d.max_seqs || layer < 0 || layer >= kv->d.n_layers || head < 0 || head >= kv->d.n_kv_heads)
    return fail(SLORA_E_INVAL, "slora_kv_pages: sequence, layer or head out of range");
  const Seq& s = kv->seqs[seq];
  for (int32_t b = 0; b < std::min(cap, s.blocks); ++b)
    ids[b] = kv->pages_of(s.held[b])[(int64_t)layer * kv->d.n_kv_heads + head];
  *n = s.blocks;
  return SLORA_OK;
}

slora_status slora_kv_build_step(slora_kv* kv, int32_t n, const int32_t* seqs, const int32_t* counts, int32_t reread,
                                 slora_kv_step** out) {
  return slora_kv_build_step_window(kv, n, seqs, counts, reread, 0, 0, out);
}

slora_status slora_kv_build_step_window(slora_kv* kv, int32_t n, const int32_t* seqs, const int32_t* counts,
                                        int32_t reread, int32_t window, int32_t sinks, slora_kv_step** out) {
  if (!kv || !out || n < 0 || (n > 0 && (!seqs || !counts)))
    return fail(SLORA_E_INVAL, "slora_kv_build_step: NULL argument");
  if (reread != 0 && reread != 1) return fail(SLORA_E_INVAL, "slora_kv_build_step: reread must be 0 or 1");
  if (window < 0 || sinks < 0) return fail(SLORA_E_INVAL, "slora_kv_build_step: window and sinks must not be negative");
  slora_kv_step* st = nullptr;
  try {
    std::vector<uint8_t> named((size_t)kv->d.max_seqs, 0);
    int64_t rows = 0;
    for (int32_t i = 0; i < n; ++i) {
      if (seqs[i] < 0 || seqs[i] >= kv->d.max_seqs)
        return fail(SLORA_E_INVAL, "slora_kv_build_step: sequence id out of range");
      if (named[seqs[i]]++) return fail(SLORA_E_INVAL, "slora_kv_build_step: a sequence is named twice");
      const int64_t len = kv->seqs[seqs[i]].len;
      if (counts[i] < 0) return fail(SLORA_E_INVAL, "slora_kv_build_step: negative count");
      if (reread && counts[i] > len)
        return fail(SLORA_E_INVAL, "slora_kv_build_step: more rows than the sequence has tokens");
      if (!reread && len + counts[i] > kv->d.max_tokens)
        return fail(SLORA_E_INVAL, "slora_kv_build_step: a sequence would pass max_tokens");
      if (!reread && len + counts[i] + kv->seqs[seqs[i]].shift() > kMostPositions)
        return fail(SLORA_E_INVAL, "slora_kv_build_step: a sequence would pass position 2^30");
      rows += counts[i];
    }
    if (rows > INT32_MAX / 2) return fail(SLORA_E_INVAL, "slora_kv_build_step: too many rows");
    st = new slora_kv_step();
    st->kv = kv;
    st->reread = reread != 0;
    st->n_rows = (int32_t)rows;
    st->row_pos.reserve((size_t)rows);
    int64_t need = 0, patches = 0;
    int32_t row0 = 0;
    for (int32_t i = 0; i < n; ++i) {
      Seq& s = kv->seqs[seqs[i]];
      const int64_t end = reread ? s.len : s.len + counts[i];
      const int32_t start = (int32_t)(end - counts[i]), blocks = (int32_t)((end + kv->block - 1) / kv->block);
      st->seqs.push_back({seqs[i], start, counts[i], row0});
      st->gens.push_back(s.gen);
      st->ends.push_back(blocks);
      st->max_len = std::max(st->max_len, (int32_t)end);
      const int32_t shift = reread ? 0 : s.shift();              // (a reread step rotates nothing)
      if (counts[i]) st->n_positions = std::max(st->n_positions, (int32_t)end + shift);
      need += (blocks - s.blocks) * kv->per_block();
      patches += (blocks - s.entered) * kv->per_block();
      st->row_pos.resize((size_t)row0 + counts[i]);
      std::iota(st->row_pos.end() - counts[i], st->row_pos.end(), start + shift);
      for (int32_t b = start / kv->block; counts[i] && b < blocks; ++b)
        st->blocks.push_back({seqs[i], b, std::max(0, start - b * kv->block),
                              (int32_t)std::min<int64_t>(kv->block, end - (int64_t)b * kv->block),
                              row0 + std::max(0, b * kv->block - start), shift, {0, 0}});
      row0 += counts[i];
    }
    st->n_small = (int32_t)(std::stable_partition(st->blocks.begin(), st->blocks.end(), [](const KvBlock& b) {
                              return b.slot1 - b.slot0 == 1;
                            }) - st->blocks.begin());
    build_tiles(st, window, sinks);
    const int64_t kvh = kv->d.n_kv_heads;
    const int64_t append =
        2 * (int64_t)st->blocks.size() * kvh + (rows * kv->d.n_heads * (kv->d.head_dim / 16)) / kThreads + 1;
    if (std::max({append, (int64_t)st->prompts.size() * kvh, (int64_t)st->tiles.size() * kvh,
                  (int64_t)st->combine.size() * kvh * kKvRows}) > kMostGroups ||
        patches > INT32_MAX / 2 || rows * kv->d.n_heads > INT32_MAX / 2 || st->n_parts * kvh > INT32_MAX / 2) {
      delete st;
      return fail(SLORA_E_INVAL, "slora_kv_build_step: the step is too large for one launch");
    }
    if (need > slora_free_count(kv->pool, kv->d.cls)) {
      delete st;
      return fail(SLORA_E_NOMEM, "slora_kv_build_step: not enough free pages");
    }
    std::vector<int32_t> ids((size_t)need);
    st->patches.reserve((size_t)patches);
    kv->blocks.reserve(need / kv->per_block(), kv->per_block());
    for (int32_t i = 0; i < n; ++i) {
      std::vector<int32_t>& held = kv->seqs[seqs[i]].held;
      const size_t want = (size_t)st->ends[i];
      if (want > held.capacity()) held.reserve(std::max(want, 2 * held.capacity()));
      std::vector<int32_t>& stored = kv->seqs[seqs[i]].stored;
      stored.resize(std::max(stored.size(), (size_t)st->ends[i] * kv->d.n_layers), 0);
    }
    slora_status got = slora_alloc_pages(kv->pool, kv->d.cls, need, ids.data());
    if (got != SLORA_OK) {
      delete st;
      return got;
    }
    // nothing below can fail
    st->n_new_pages = need;
    size_t at = 0;
    for (int32_t i = 0; i < n; ++i) {
      Seq& s = kv->seqs[seqs[i]];
      for (; s.blocks < st->ends[i]; ++s.blocks, at += (size_t)kv->per_block())
        s.held.push_back(kv->blocks.add(ids.data() + at, kv->per_block()));
      if (!reread) s.len += counts[i];
      for (int32_t b = s.entered; b < s.blocks; ++b)
        for (int64_t x = 0; x < kv->per_block(); ++x) {
          const uint64_t entry = ((uint64_t)seqs[i] * kv->per_block() + x) * kv->max_blocks + b;
          const int32_t page = kv->pages_of(s.held[b])[x];
          st->patches.push_back({(uint32_t)entry, (uint32_t)(entry >> 32), page, 0});
        }
    }
  } catch (const std::bad_alloc&) {
    delete st;
    return fail(SLORA_E_NOMEM, "slora_kv_build_step: out of host memory");
  }
  *out = st;
  return SLORA_OK;
}

void slora_kv_step_destroy(slora_kv_step* st) { delete st; }

slora_status slora_kv_step_get_info(const slora_kv_step* st, slora_kv_step_info* info) {
  if (!st || !info) return fail(SLORA_E_INVAL, "slora_kv_step_get_info: NULL argument");
  *info = slora_kv_step_info{};
  info->n_seqs = (int32_t)st->seqs.size();
  info->n_rows = st->n_rows;
  info->max_len = st->max_len;
  info->n_blocks = (int32_t)st->blocks.size();
  info->n_new_pages = (int32_t)st->n_new_pages;
  info->n_row_tiles = (int32_t)st->tiles.size();
  info->n_prompt_tiles = (int32_t)st->prompts.size();
  info->meta_bytes = st->bytes();
  info->workspace_bytes = st->workspace();
  return SLORA_OK;
}

slora_status slora_kv_step_upload(slora_kv_step* st, void* dev_meta, size_t dev_meta_bytes, void* stream) {
  const std::string f = "slora_kv_step_upload";
  if (!st || !dev_meta) return fail(SLORA_E_INVAL, f + ": NULL argument");
  if (reinterpret_cast<uintptr_t>(dev_meta) & 15) return fail(SLORA_E_INVAL, f + ": dev_meta must be 16-byte aligned");
  if (dev_meta_bytes < st->bytes()) return fail(SLORA_E_NOMEM, f + ": dev_meta smaller than meta_bytes");
  slora_kv* kv = st->kv;
  slora_status ok = check_launch(f, kv, st, 0);
  if (ok != SLORA_OK) return ok;
  if (st->bytes() > 0) {
    std::vector<char> image;
    try {
      image.resize(st->bytes());
    } catch (const std::bad_alloc&) {
      return fail(SLORA_E_NOMEM, f + ": out of host memory");
    }
    auto put = [&](size_t off, const void* src, size_t bytes) {
      if (bytes) std::memcpy(image.data() + off, src, bytes);
    };
    put(0, st->blocks.data(), st->blocks.size() * sizeof(KvBlock));
    put(st->prompts_off(), st->prompts.data(), st->prompts.size() * sizeof(KvTile));
    put(st->tiles_off(), st->tiles.data(), st->tiles.size() * sizeof(KvTile));
    put(st->tiles_off() + st->tiles.size() * sizeof(KvTile), st->combine.data(), st->combine.size() * sizeof(KvTile));
    put(st->patches_off(), st->patches.data(), st->patches.size() * sizeof(KvPatch));
    put(st->row_pos_off(), st->row_pos.data(), st->row_pos.size() * sizeof(int32_t));
    UploadWith with;
    with.table = kv->table();
    with.patches_off = st->patches_off();
    with.n_patches = (int32_t)st->patches.size();
    ok = pool_upload(kv->pool, dev_meta, image.data(), image.size(), static_cast<hipStream_t>(stream), with);
    if (ok != SLORA_OK) return ok;
  }
  for (size_t i = 0; i < st->seqs.size(); ++i) {
    Seq& s = kv->seqs[st->seqs[i].seq];
    s.entered = std::max(s.entered, st->ends[i]);
  }
  st->dev = static_cast<const char*>(dev_meta);
  return SLORA_OK;
}

slora_status slora_kv_append(slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q, int64_t q_stride,
                             void* q_out, int64_t q_out_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const float* cos_sin, int64_t n_positions, void* stream) {
  return append("slora_kv_append", kv, st, layer, q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, nullptr,
                cos_sin, n_positions, stream);
}

slora_status slora_kv_append_norm(slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q, int64_t q_stride,
                                  void* q_out, int64_t q_out_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const slora_kv_norm* norm, const float* cos_sin,
                                  int64_t n_positions, void* stream) {
  const std::string f = "slora_kv_append_norm";
  if (!norm) return fail(SLORA_E_INVAL, f + ": NULL norm");
  if (!(norm->eps >= 0x1p-126f) || !std::isfinite(norm->eps))
    return fail(SLORA_E_INVAL, f + ": eps must be at least 2^-126 and finite");
  if (norm->per_head != 0 && norm->per_head != 1) return fail(SLORA_E_INVAL, f + ": per_head must be 0 or 1");
  if ((reinterpret_cast<uintptr_t>(norm->q_weight) | reinterpret_cast<uintptr_t>(norm->k_weight)) & 15)
    return fail(SLORA_E_INVAL, f + ": the weights must be 16-byte aligned");
  return append(f, kv, st, layer, q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, norm, cos_sin,
                n_positions, stream);
}

// Frequencies are found in more than 64 bits, as turns a position.
slora_status slora_kv_rotary_table(slora_kv* kv, const slora_kv_rotary* r, int64_t first, int64_t n, float* cos_sin,
                                   void* stream) {
  const std::string f = "slora_kv_rotary_table";
  if (!kv || !r || (!cos_sin && n != 0)) return fail(SLORA_E_INVAL, f + ": NULL argument");
  const int32_t rot = kv->d.rot_dim;
  if (!rot) return fail(SLORA_E_INVAL, f + ": the cache rotates nothing (rot_dim 0)");
  if (reinterpret_cast<uintptr_t>(cos_sin) & 15) return fail(SLORA_E_INVAL, f + ": cos_sin must be 16-byte aligned");
  if (first < 0 || n < 0 || first > kMostPositions || n > kMostPositions - first)
    return fail(SLORA_E_INVAL, f + ": positions must be 0 .. 2^30");
  if (r->reserved0 != 0) return fail(SLORA_E_INVAL, f + ": reserved0 must be 0");
  if (r->scaling < SLORA_KV_ROT_NONE || r->scaling > SLORA_KV_ROT_RAMP)
    return fail(SLORA_E_INVAL, f + ": unknown scaling");
  if (!(r->base > 1.) || !std::isfinite(r->base)) return fail(SLORA_E_INVAL, f + ": base must be above 1 and finite");
  if (!std::isfinite(r->amplitude)) return fail(SLORA_E_INVAL, f + ": amplitude must be finite");
  const bool scaled = r->scaling != SLORA_KV_ROT_NONE;
  if (scaled && (!(r->factor >= 1.) || !std::isfinite(r->factor)))
    return fail(SLORA_E_INVAL, f + ": factor must be at least 1 and finite");
  if (r->scaling == SLORA_KV_ROT_BANDS || r->scaling == SLORA_KV_ROT_RAMP) {
    if (!(r->trained >= 1.) || !std::isfinite(r->trained))
      return fail(SLORA_E_INVAL, f + ": trained must be at least 1 and finite");
    if (!(r->low > 0.) || !(r->high > r->low) || !std::isfinite(r->high))
      return fail(SLORA_E_INVAL, f + ": low and high must be finite, 0 < low < high");
  }
  if (n == 0) return SLORA_OK;
  typedef long double wide;
  const wide pi2 = 6.283185307179586476925286766559005768L, factor = scaled ? (wide)r->factor : 1.L;
  wide log_base = std::log((wide)r->base);
  if (r->scaling == SLORA_KV_ROT_BASE) log_base += std::log(factor) * rot / (rot - 2);
  auto pair_of = [&](double turns) { return rot * std::log((wide)r->trained / (pi2 * turns)) / (2 * log_base); };
  KvRotary R{};
  wide by16[8], by1[16];                                       // t_i = by16[i / 16] by1[i % 16]
  for (int32_t i = 0; i < 16; ++i) by1[i] = std::exp(-2 * i * log_base / rot);
  for (int32_t i = 0; i < 8; ++i) by16[i] = std::exp(-32 * i * log_base / rot);
  for (int32_t i = 0; i < rot / 2; ++i) {
    wide t = by16[i / 16] * by1[i % 16], keep = 1.L;
    if (r->scaling == SLORA_KV_ROT_LINEAR) keep = 0.L;
    if (r->scaling == SLORA_KV_ROT_BANDS)
      keep = (r->trained * t / pi2 - r->low) / ((wide)r->high - r->low);
    if (r->scaling == SLORA_KV_ROT_RAMP) {
      const wide high = std::max(std::floor(pair_of(r->high)), 0.L);
      const wide low = std::min(std::ceil(pair_of(r->low)), (wide)(rot - 1));
      keep = 1.L - (i - high) / std::max(low - high, 0.001L);
    }
    keep = std::min(std::max(keep, 0.L), 1.L);
    if (keep < 1.L) t *= keep + (1.L - keep) / factor;
    t /= pi2;
    R.turn_hi[i] = (double)t;
    R.turn_lo[i] = (double)(t - (wide)R.turn_hi[i]);
  }
  R.amplitude = r->amplitude;
  R.out = cos_sin;
  R.first = first;
  R.n = n;
  R.half = rot / 2;
  slora_status ok = pool_device_current(kv->pool);
  if (ok != SLORA_OK) return ok;
  return launched(f, launch_kv_rotary(R, static_cast<hipStream_t>(stream)));
}

slora_status slora_kv_attend(slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q, int64_t q_stride,
                             void* out, int64_t out_stride, float scale, int32_t window, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return attend("slora_kv_attend", kv, st, layer, q, q_stride, out, out_stride, scale, window, 0, workspace,
                workspace_bytes, stream);
}

slora_status slora_kv_attend_sinks(slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q,
                                   int64_t q_stride, void* out, int64_t out_stride, float scale, int32_t window,
                                   int32_t sinks, void* workspace, size_t workspace_bytes, void* stream) {
  return attend("slora_kv_attend_sinks", kv, st, layer, q, q_stride, out, out_stride, scale, window, sinks, workspace,
                workspace_bytes, stream);
}

size_t slora_kv_take_bytes(const slora_kv* kv, int32_t n, const int32_t* dst, const int32_t* src,
                           const int32_t* n_ranges, const int64_t* ranges) {
  const std::string f = "slora_kv_take_bytes: ";
  try {
    TakePlan plan;
    const char* why = plan_take(kv, n, dst, src, n_ranges, ranges, &plan);
    if (!why) return std::max<size_t>(16, plan.bytes());
    fail(SLORA_E_INVAL, f + why);
  } catch (const std::bad_alloc&) {
    fail(SLORA_E_NOMEM, f + "out of host memory");
  }
  return 0;
}

slora_status slora_kv_take(slora_kv* kv, int32_t n, const int32_t* dst, const int32_t* src, const int32_t* n_ranges,
                           const int64_t* ranges, void* dev_meta, size_t dev_meta_bytes, void* stream) {
  const std::string f = "slora_kv_take";
  try {
    TakePlan plan;
    if (const char* why = plan_take(kv, n, dst, src, n_ranges, ranges, &plan))
      return fail(SLORA_E_INVAL, f + ": " + why);
    const int64_t per = plan.per, need = (int64_t)plan.copies.size() * per;
    if (need > slora_free_count(kv->pool, kv->d.cls)) return fail(SLORA_E_NOMEM, f + ": not enough free pages");
    const bool works = !plan.rows.empty();
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (works) {
      if (!dev_meta || reinterpret_cast<uintptr_t>(dev_meta) & 15)
        return fail(SLORA_E_INVAL, f + ": dev_meta must be non-NULL and 16-byte aligned");
      if (dev_meta_bytes < plan.bytes()) return fail(SLORA_E_NOMEM, f + ": dev_meta smaller than slora_kv_take_bytes");
      slora_status ok = pool_device_current(kv->pool);
      if (ok != SLORA_OK) return ok;
    }
    if (n > 0) {
      // Also where nothing is launched: launches that the graph holds already would
      // read freed pages.  (Such a call needs no device, so asking for one may fail.)
      hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
      const hipError_t e = hipStreamIsCapturing(hs, &capture);
      if (e != hipSuccess && works) return fail(SLORA_E_HIP, f + ": hipStreamIsCapturing: " + hipGetErrorString(e));
      if (e != hipSuccess) (void)hipGetLastError();              // not for a later call to find
      if (e == hipSuccess && capture != hipStreamCaptureStatusNone)
        return fail(SLORA_E_INVAL, f + ": the stream is captured, which this call cannot be");
    }
    // everything that can run out of host memory
    std::vector<int32_t> ids((size_t)need);
    std::vector<char> image(works ? plan.bytes() : 0);
    std::vector<Seq> made(plan.parts.size());
    for (size_t i = 0; i < plan.parts.size(); ++i) {
      const TakePlan::Part& part = plan.parts[i];
      Seq& s = made[i];
      s.len = part.len;
      s.blocks = s.entered = (int32_t)part.from.size();
      s.gen = kv->seqs[part.dst].gen + 1;
      s.held.resize(part.from.size());
      s.stored.assign(part.from.size() * kv->d.n_layers, kv->block);
      if (part.len % kv->block)
        std::fill(s.stored.end() - kv->d.n_layers, s.stored.end(), (int32_t)(part.len % kv->block));
      s.runs = part.runs;
    }
    kv->blocks.reserve((int64_t)plan.copies.size(), per);
    slora_status ok = slora_alloc_pages(kv->pool, kv->d.cls, need, ids.data());
    if (ok != SLORA_OK) return ok;
    if (works) {
      auto put = [&](size_t off, const auto& v) {
        if (!v.empty()) std::memcpy(image.data() + off, v.data(), v.size() * sizeof(v[0]));
      };
      put(0, plan.rows);
      put(plan.copies_off(), plan.copies);
      put(plan.entries_off(), plan.entries);
      put(plan.tokens_off(), plan.tokens);
      put(plan.pages_off(), ids);
      ok = pool_upload(kv->pool, dev_meta, image.data(), image.size(), hs);
      if (ok == SLORA_OK) {
        const char* dev = static_cast<const char*>(dev_meta);
        KvTake A{};
        A.kv = kv->view();
        A.rows = reinterpret_cast<const KvTakeRow*>(dev);
        A.copies = reinterpret_cast<const KvCopy*>(dev + plan.copies_off());
        A.entries = reinterpret_cast<const int32_t*>(dev + plan.entries_off());
        A.tokens = reinterpret_cast<const int32_t*>(dev + plan.tokens_off());
        A.pages = reinterpret_cast<const int32_t*>(dev + plan.pages_off());
        A.n_rows = (int32_t)plan.rows.size();
        A.n_copies = (int32_t)plan.copies.size();
        ok = launched(f, launch_kv_take(A, plan.in_place, hs));
        if (ok != SLORA_OK) (void)hipStreamSynchronize(hs);     // nothing writes pages that are given back
      }
      if (ok != SLORA_OK) {
        pool_untake_pages(kv->pool, kv->d.cls, need, ids.data());
        return ok;
      }
    }
    // nothing below can fail: first what the new sequences hold, then what the old ones let go of
    int64_t copy = 0;
    for (size_t i = 0; i < plan.parts.size(); ++i) {
      const TakePlan::Part& part = plan.parts[i];
      for (size_t b = 0; b < part.from.size(); ++b) {
        if (part.from[b] < 0) {
          made[i].held[b] = kv->blocks.add(ids.data() + copy++ * per, per);
        } else {
          made[i].held[b] = kv->seqs[part.src].held[part.from[b]];
          ++kv->blocks.refs[made[i].held[b]];
        }
      }
    }
    for (size_t i = 0; i < plan.parts.size(); ++i) {
      Seq& s = kv->seqs[plan.parts[i].dst];
      for (int32_t record : s.held)
        if (kv->blocks.release(record)) pool_return_pages(kv->pool, kv->d.cls, per, kv->pages_of(record));
      s = std::move(made[i]);
    }
  } catch (const std::bad_alloc&) {
    return fail(SLORA_E_NOMEM, f + ": out of host memory");
  }
  return SLORA_OK;
}

slora_status slora_kv_read(slora_kv* kv, const slora_kv_step* st, int32_t layer, void* k, int64_t k_stride, void* v,
                           int64_t v_stride, void* stream) {
  const std::string f = "slora_kv_read";
  slora_status ok = check_launch(f, kv, st, layer);
  if (ok != SLORA_OK) return ok;
  if (!k && !v) return fail(SLORA_E_INVAL, f + ": NULL k and v");
  if (st->n_rows == 0) return SLORA_OK;
  if (k && (ok = check_rows(f, "k", kv, k, k_stride, kv->d.n_kv_heads)) != SLORA_OK) return ok;
  if (v && (ok = check_rows(f, "v", kv, v, v_stride, kv->d.n_kv_heads)) != SLORA_OK) return ok;
  if (!st->dev) return fail(SLORA_E_INVAL, f + ": step not uploaded (call slora_kv_step_upload)");
  if ((ok = pool_device_current(kv->pool)) != SLORA_OK) return ok;
  KvRead R{};
  R.kv = kv->view();
  R.blocks = reinterpret_cast<const KvBlock*>(st->dev);
  R.n_blocks = (int32_t)st->blocks.size();
  R.layer = layer;
  R.k = k;
  R.v = v;
  R.k_stride = k_stride;
  R.v_stride = v_stride;
  return launched(f, launch_kv_read(R, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
