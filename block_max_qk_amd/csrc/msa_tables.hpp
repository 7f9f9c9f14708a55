// The step tables kernel (gfx950 only): from the requests' lengths the prefix
// sums, block tables, positions and slots of one serving step, with pages from a
// free list for the blocks that the new tokens begin.
//
//   cu[b + 1] = sum of new[0..b],  kv[b] = ctx[b] + new[b],
//   need[b] = ceil(kv[b] / 128) - ceil(ctx[b] / 128)  (blocks below MB, of a row that exists)
//
// Bound by latency: a workgroup reads the lengths of every request before its own
// (8 bytes each, out of the L2), adds them up, and knows from the two sums where
// its requests' tokens begin and which pages of the free list are theirs; no
// workgroup waits for another, and one launch does it all (a scan of its own in
// front would be a second launch, 5 us, for less than that of reads).  The lengths
// of groups of `group` requests are scanned by one wave, so that there are about
// 512 workgroups up to 32768 requests (and the reads grow with their square).
//
// 64 decode requests over tables of 256 blocks 4 us, 300 of 1 to 200 tokens 5,
// 4096 over tables of 1024 blocks (19 MB) 10.5 to 11 (the profiler's figures; calls in
// a row take 9.8), 1.8 TB/s, 13.5 with one request's lengths in flight a lane and one
// loop for the blocks and the rest of a row.  A call takes 9 to 10 us of host time, so
// none of these waits for its kernel.  A long prompt among more than 256 requests does:
// no other workgroup shares its tokens then, and past 512 requests one wave takes them.
// 8192 tokens beside 255 single ones 6.5 us, beside 512 or 600 25.7; 30000 beside 600
// 87, beside 4095 89.
#pragma once

#include "msa_device.hpp"

namespace msa {

constexpr int kTableWaves = 4;

struct TablesParams {
  const int32_t* fresh;        // [B] new tokens
  const int32_t* ctx;          // [B] earlier tokens
  const int32_t* rows;         // [B] pool rows, or nullptr: row b
  int32_t* pool;               // [R, width]
  const int32_t* free_pages;   // [free_size]
  const int32_t* free_count;   // [2]
  int32_t* free_out;           // [2], or nullptr: written by a launch of its own
  int32_t* cu_q;               // [B+1]
  int32_t* kv_len;             // [B]
  int32_t* start_loc;          // [B]
  int32_t* block_table;        // [B, MB]
  int32_t* positions;          // [T]
  int64_t* slots;              // [T]
  int32_t* cu_pages;           // [B+1]
  int64_t R, width, T;
  int32_t free_size, B, MB;
  int32_t group;               // requests per workgroup, at most 64
  int32_t count_only;          // 1: only free_out is written (one workgroup)
};

__device__ __forceinline__ int clamp31(int64_t x) {
  return (int)min(x, (int64_t)INT32_MAX);
}

// What the step needs to know of a request's lengths.
struct TablesRequest {
  int64_t row;                 // of the pool, -1: none
  int32_t ctx, fresh, kv;      // never negative
  int32_t held, now;           // blocks below MB before and after the step
  int32_t need;                // pages that the step takes for it, if there are enough
};

__device__ __forceinline__ TablesRequest tables_request(const TablesParams& p, int b) {
  TablesRequest r;
  r.ctx = max(p.ctx[b], 0);
  r.fresh = max(p.fresh[b], 0);
  r.row = p.rows ? p.rows[b] : b;
  if (r.row < 0 || r.row >= p.R) r.row = -1;
  r.kv = clamp31((int64_t)r.ctx + r.fresh);
  r.held = min((int)(((uint32_t)r.ctx + kP - 1) / kP), p.MB);
  r.now = min((int)(((uint32_t)r.kv + kP - 1) / kP), p.MB);
  r.need = r.row >= 0 ? r.now - r.held : 0;
  return r;
}

__global__ __launch_bounds__(64 * kTableWaves) void tables_kernel(TablesParams p) {
  const int tid = threadIdx.x, l = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t base = p.count_only ? p.B : (int64_t)blockIdx.x * p.group;
  const int b0 = (int)min(base, (int64_t)p.B);
  const int n = min(p.group, p.B - b0);               // this workgroup's requests
  const int64_t count = min(max(p.free_count[0], 0), p.free_size);

  // tokens and pages of the requests before, and this group's own
  __shared__ int64_t sums[kTableWaves][2];
  int64_t tokens = 0, pages = 0;
  // (four requests a lane at a time, whose reads are in flight together)
  for (int64_t b = tid; b < b0; b += 4 * 64 * kTableWaves) {
    TablesRequest r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      r[u] = tables_request(p, (int)min(b + u * 64 * kTableWaves, (int64_t)b0 - 1));
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool is = b + u * 64 * kTableWaves < b0;
      tokens += is ? r[u].fresh : 0;
      pages += is ? r[u].need : 0;
    }
  }
  tokens = lane_at(wave_incl_scan(tokens), 63);
  pages = lane_at(wave_incl_scan(pages), 63);
  if (l == 0) {
    sums[wave][0] = tokens;
    sums[wave][1] = pages;
  }
  TablesRequest mine{-1, 0, 0, 0, 0, 0, 0};
  if (l < n) mine = tables_request(p, b0 + l);
  const int64_t t_incl = wave_incl_scan((int64_t)mine.fresh);
  const int64_t p_incl = wave_incl_scan((int64_t)mine.need);
  __syncthreads();
  tokens = pages = 0;
#pragma unroll
  for (int w = 0; w < kTableWaves; ++w) {
    tokens += sums[w][0];
    pages += sums[w][1];
  }
  // (lane i: where request b0 + i's tokens and pages begin)
  const int64_t t_first = tokens + t_incl - mine.fresh;
  const int64_t p_first = pages + p_incl - mine.need;
  const int64_t t_end = tokens + lane_at(t_incl, 63);     // of the whole group
  const int64_t p_end = pages + lane_at(p_incl, 63);

  const bool last = b0 + n == p.B;
  if (last && p.free_out && blockIdx.y == 0 && tid == 0) {
    p.free_out[0] = (int)(count - min(p_end, count));
    p.free_out[1] = clamp31(max(p_end - count, (int64_t)0));
  }
  if (p.count_only) return;
  if (blockIdx.y == 0 && wave == 0) {
    if (l < n) {
      p.cu_q[b0 + l + 1] = (int)min(t_first + mine.fresh, p.T);
      p.cu_pages[b0 + l + 1] = (int)min(p_first + mine.need, count);
      p.kv_len[b0 + l] = mine.kv;
      p.start_loc[b0 + l] = mine.ctx / kP;
    }
    if (b0 == 0 && l == 0) p.cu_q[0] = p.cu_pages[0] = 0;
  }

  // one request a workgroup: all waves of its row of the grid share it;
  // otherwise a wave each in turn
  const bool shared = p.group == 1;
  const int64_t at = 64 * (shared ? (int64_t)blockIdx.y * kTableWaves + wave : 0) + l;
  const int64_t step = 64 * (shared ? (int64_t)gridDim.y * kTableWaves : 1);
  for (int i = shared ? 0 : wave; i < n; i += shared ? 1 : kTableWaves) {
    const int64_t row = lane_at(mine.row, i);
    const int held = lane_at(mine.held, i), now = lane_at(mine.now, i);
    const int ctx = lane_at(mine.ctx, i);
    const int64_t pf = lane_at(p_first, i), tf = lane_at(t_first, i);
    int32_t* const pr = p.pool + row * p.width;
    // the page of block k < now (-1: none); pages are taken from the list's end
    auto page_of = [&](int k) -> int {
      if (row < 0) return -1;
      if (k < held) return pr[k];
      const int64_t nth = pf + (k - held);
      return nth < count ? p.free_pages[count - 1 - nth] : -1;
    };
    int64_t k = at;
    for (; k < now; k += step) {
      const int page = page_of((int)k);
      p.block_table[(int64_t)(b0 + i) * p.MB + k] = page;
      if (row >= 0 && k >= held) pr[k] = page;
    }
    for (; k < p.MB; k += step) p.block_table[(int64_t)(b0 + i) * p.MB + k] = -1;
    const int64_t te = min(tf + lane_at(mine.fresh, i), p.T);
    for (int64_t t = tf + at; t < te; t += step) {
      const int64_t pos = ctx + (t - tf);
      const int page = pos / kP < p.MB ? page_of((int)(pos / kP)) : -1;
      p.positions[t] = clamp31(pos);
      p.slots[t] = page >= 0 ? (int64_t)page * kP + pos % kP : -1;
    }
  }
  // rows behind the last token
  if (last) {
    const int64_t all = (int64_t)gridDim.y * 64 * kTableWaves;
    for (int64_t t = t_end + (int64_t)blockIdx.y * 64 * kTableWaves + tid; t < p.T; t += all) {
      p.positions[t] = 0;
      p.slots[t] = -1;
    }
  }
}

}  // namespace msa
