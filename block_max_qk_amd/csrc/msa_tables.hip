// Host side of msa_step_tables: argument validation (all of it before any HIP
// call) and one launch on the caller's stream, or two where the free list's
// count is updated in place.
#include "msa_index_score.h"

#include <algorithm>
#include <cstdint>

#include "msa_host.hpp"
#include "msa_tables.hpp"

namespace {

bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// Memory that a call reads or writes.
struct Range {
  const void* at;
  int64_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  const auto x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
         y < x + (uintptr_t)a.bytes;
}

}  // namespace

extern "C" msa_status_t msa_step_tables(
    const int32_t* new_tokens, const int32_t* ctx_len, const int32_t* rows, int32_t batch,
    int32_t* pool, int64_t pool_rows, int64_t pool_blocks, const int32_t* free_pages,
    int64_t free_size, const int32_t* free_count, int32_t* free_out, int64_t max_blocks, int64_t T,
    int32_t block_size, int32_t* cu_seqlens_q, int32_t* kv_len, int32_t* start_loc,
    int32_t* block_table, int32_t* positions, int64_t* slots, int32_t* cu_pages, void* stream) {
  if (!cu_seqlens_q || !cu_pages || !free_count || !free_out) return MSA_ERR_NULL;
  // (every workgroup adds up the lengths before its requests: 2^20 of them take
  // milliseconds, and as the square)
  if (batch < 0 || batch > (1 << 20) || T < 0 || T > INT32_MAX || block_size != msa::kP)
    return MSA_ERR_SHAPE;
  if (max_blocks < 1 || max_blocks > (1 << 24) || pool_blocks < max_blocks ||
      pool_blocks > INT32_MAX || pool_rows < 0 || pool_rows > INT32_MAX || free_size < 0 ||
      free_size > INT32_MAX || pool_rows * pool_blocks > ((int64_t)1 << 60))
    return MSA_ERR_SHAPE;
  if (batch > 0 && (!new_tokens || !ctx_len || !kv_len || !start_loc || !block_table ||
                    (pool_rows > 0 && !pool)))
    return MSA_ERR_NULL;
  if ((free_size > 0 && !free_pages) || (T > 0 && (!positions || !slots))) return MSA_ERR_NULL;
  for (const void* p : {(const void*)new_tokens, (const void*)ctx_len, (const void*)rows,
                        (const void*)pool, (const void*)free_pages, (const void*)free_count,
                        (const void*)free_out, (const void*)cu_seqlens_q, (const void*)kv_len,
                        (const void*)start_loc, (const void*)block_table, (const void*)positions,
                        (const void*)cu_pages})
    if (misaligned(p, 4)) return MSA_ERR_STRIDE;
  if (misaligned(slots, 8)) return MSA_ERR_STRIDE;

  // workgroups read lengths and pages while others write: nothing that is
  // written may be read elsewhere, or be written twice (but the counts: below)
  const Range read[] = {{new_tokens, 4 * (int64_t)batch}, {ctx_len, 4 * (int64_t)batch},
                        {rows, 4 * (int64_t)batch}, {free_pages, 4 * free_size}};
  const Range written[] = {{pool, 4 * pool_rows * pool_blocks},
                           {cu_seqlens_q, 4 * ((int64_t)batch + 1)},
                           {kv_len, 4 * (int64_t)batch},
                           {start_loc, 4 * (int64_t)batch},
                           {block_table, 4 * batch * max_blocks},
                           {positions, 4 * T},
                           {slots, 8 * T},
                           {cu_pages, 4 * ((int64_t)batch + 1)},
                           {free_out, 8}};
  constexpr int kWritten = sizeof(written) / sizeof(written[0]);
  for (int i = 0; i < kWritten; ++i) {
    for (const Range& r : read)
      if (overlap(written[i], r)) return MSA_ERR_STRIDE;
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return MSA_ERR_STRIDE;
    if (i + 1 < kWritten && overlap(written[i], Range{free_count, 8})) return MSA_ERR_STRIDE;
  }

  msa::TablesParams p{};
  p.fresh = new_tokens;
  p.ctx = ctx_len;
  p.rows = rows;
  p.pool = pool;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.cu_q = cu_seqlens_q;
  p.kv_len = kv_len;
  p.start_loc = start_loc;
  p.block_table = block_table;
  p.positions = positions;
  p.slots = slots;
  p.cu_pages = cu_pages;
  p.R = pool_rows;
  p.width = pool_blocks;
  p.T = T;
  p.free_size = (int32_t)free_size;
  p.B = batch;
  p.MB = (int32_t)max_blocks;
  // about 512 workgroups, two a CU: groups of requests where there are more, and
  // where there are fewer, several workgroups that share a request's blocks and
  // tokens, of 512 of the longest request's at least
  p.group = (int32_t)std::clamp<int64_t>((batch + 511) / 512, 1, 64);
  const int64_t groups = std::max<int64_t>((batch + (int64_t)p.group - 1) / p.group, 1);
  const int64_t most = std::max<int64_t>(max_blocks, T);
  const int64_t share =
      p.group > 1 ? 1 : std::clamp<int64_t>(512 / groups, 1, std::max<int64_t>(most / 512, 1));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)groups, (unsigned)share), block(64 * msa::kTableWaves);
  // every workgroup reads the count, so it is written behind them all if it is
  // the same memory (the two counts of free_out, or one of them)
  const bool one = groups * share == 1;
  if (one || !overlap(Range{free_count, 8}, Range{free_out, 8})) p.free_out = free_out;
  hipError_t e = msa::launch_kernel(msa::tables_kernel, grid, block, s, p);
  if (e == hipSuccess && !p.free_out) {
    p.free_out = free_out;
    p.count_only = 1;
    e = msa::launch_kernel(msa::tables_kernel, dim3(1), block, s, p);
  }
  return e == hipSuccess ? MSA_OK : MSA_ERR_HIP;
}
