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
  std::vector<int32_t> pages;   // [block][layer][head]
  std::vector<int32_t> stored;  // [block][layer] tokens that appends have been launched for
};

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
// the others, with their key splits, longest first.
void build_tiles(slora_kv_step* st) {
  const slora_kv_desc& d = st->kv->d;
  const int32_t G = d.n_heads / d.n_kv_heads;
  const bool half = st->kv->info.dtype == SLORA_F16;
  auto prompt = [&](const StepSeq& s) { return half && (int64_t)s.rows * G >= (s.start ? kPromptMin : kFreshMin); };
  // key groups that the tile of packed rows [r0, r0 + n) sees, without a window
  auto groups_of = [&](const StepSeq& s, int64_t r0, int64_t n) {
    return (s.start + (std::min<int64_t>(r0 + n, (int64_t)s.rows * G) - 1) / G) / kKvGroup + 1;
  };
  // groups of a workgroup: the fewest for which all row tiles' workgroups are at most kWantGroups
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
      if (wgs * d.n_kv_heads <= kWantGroups) high = mid;
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
  }
  return SLORA_OK;
}

slora_status launched(const std::string& f, hipError_t e) {
  if (e == hipSuccess) return SLORA_OK;
  return fail(SLORA_E_HIP, f + " launch: " + hipGetErrorString(e));
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
    slora_status st = slora_free_pages(kv->pool, kv->d.cls, (int64_t)s.pages.size(), s.pages.data());
    if (st != SLORA_OK) return st;
  } catch (const std::bad_alloc&) {
    return fail(SLORA_E_NOMEM, "slora_kv_drop: out of host memory");
  }
  s.pages.clear();
  s.pages.shrink_to_fit();
  s.stored.clear();
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
    ids[b] = s.pages[(size_t)(b * kv->per_block() + (int64_t)layer * kv->d.n_kv_heads + head)];
  *n = s.blocks;
  return SLORA_OK;
}

slora_status slora_kv_build_step(slora_kv* kv, int32_t n, const int32_t* seqs, const int32_t* counts, int32_t reread,
                                 slora_kv_step** out) {
  if (!kv || !out || n < 0 || (n > 0 && (!seqs || !counts)))
    return fail(SLORA_E_INVAL, "slora_kv_build_step: NULL argument");
  if (reread != 0 && reread != 1) return fail(SLORA_E_INVAL, "slora_kv_build_step: reread must be 0 or 1");
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
      if (counts[i]) st->n_positions = std::max(st->n_positions, (int32_t)end);
      need += (blocks - s.blocks) * kv->per_block();
      patches += (blocks - s.entered) * kv->per_block();
      for (int32_t p = start; p < end; ++p) st->row_pos.push_back(p);
      for (int32_t b = start / kv->block; counts[i] && b < blocks; ++b)
        st->blocks.push_back({seqs[i], b, std::max(0, start - b * kv->block),
                              (int32_t)std::min<int64_t>(kv->block, end - (int64_t)b * kv->block),
                              row0 + std::max(0, b * kv->block - start), {0, 0, 0}});
      row0 += counts[i];
    }
    st->n_small = (int32_t)(std::stable_partition(st->blocks.begin(), st->blocks.end(), [](const KvBlock& b) {
                              return b.slot1 - b.slot0 == 1;
                            }) - st->blocks.begin());
    build_tiles(st);
    // a launch holds fewer than 2^32 threads, and counts in the kernels are 31 bits
    constexpr int64_t kMostGroups = ((int64_t)1 << 32) / kThreads - 1;
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
    for (int32_t i = 0; i < n; ++i) {
      std::vector<int32_t>& pages = kv->seqs[seqs[i]].pages;
      const size_t want = (size_t)(st->ends[i] * kv->per_block());
      if (want > pages.capacity()) pages.reserve(std::max(want, 2 * pages.capacity()));
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
      const size_t more = (size_t)((st->ends[i] - s.blocks) * kv->per_block());
      s.pages.insert(s.pages.end(), ids.begin() + at, ids.begin() + at + more);
      at += more;
      s.blocks = st->ends[i];
      if (!reread) s.len += counts[i];
      for (int32_t b = s.entered; b < s.blocks; ++b)
        for (int64_t x = 0; x < kv->per_block(); ++x) {
          const uint64_t entry = ((uint64_t)seqs[i] * kv->per_block() + x) * kv->max_blocks + b;
          const int32_t page = s.pages[(size_t)(b * kv->per_block() + x)];
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
    hipStream_t hs = static_cast<hipStream_t>(stream);
    ok = pool_upload(kv->pool, dev_meta, image.data(), image.size(), hs);
    if (ok != SLORA_OK) return ok;
    const char* dev = static_cast<const char*>(dev_meta);
    ok = launched(f, launch_kv_patch(kv->table(), reinterpret_cast<const KvPatch*>(dev + st->patches_off()),
                                     (int32_t)st->patches.size(), hs));
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
  const std::string f = "slora_kv_append";
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
  ok = launched(f, launch_kv_append(A, static_cast<hipStream_t>(stream)));
  if (ok == SLORA_OK)
    for (const KvBlock& b : st->blocks) kv->seqs[b.seq].stored[(size_t)b.block * kv->d.n_layers + layer] = b.slot1;
  return ok;
}

slora_status slora_kv_attend(slora_kv* kv, const slora_kv_step* st, int32_t layer, const void* q, int64_t q_stride,
                             void* out, int64_t out_stride, float scale, int32_t window, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const std::string f = "slora_kv_attend";
  slora_status ok = check_launch(f, kv, st, layer);
  if (ok != SLORA_OK) return ok;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(SLORA_E_INVAL, f + ": scale times log2(e) must be finite in fp32");
  if (window < 0) return fail(SLORA_E_INVAL, f + ": window must be 0 (none) or positive");
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
  A.q = q;
  A.out = out;
  A.q_stride = q_stride;
  A.out_stride = out_stride;
  A.scale_log2 = scale_log2;
  A.part = static_cast<float*>(workspace);
  return launched(f, launch_kv_attend(A, static_cast<hipStream_t>(stream)));
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
