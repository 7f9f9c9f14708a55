// Attention kernels of the MSA layer (gfx950 only): dense attention of the new
// tokens over a paged or packed cache (msa_attention) and attention over the
// blocks that the top-k selection names (msa_block_attention).
//
//   S = c <q, k_j>, c = softmax_scale * log2(e), over the visible j
//   l = sum 2^(S - m),  out = sum 2^(S - m) v_j / l,  lse = ln 2 (m + log2 l)
//
// for any m near max S (kLift, kReach), in one pass over the keys with the
// running m and l.  Both products are taken transposed, with the keys (then the
// head elements) as the MFMA's M side and the rows -- (query token, head) pairs
// of one KV head -- as its N side:
// S^T = K Q^T leaves a lane with many keys of ONE row, so m and l are mostly
// in-register reductions, and O^T = V^T P^T takes the lane's own weights as
// its B operand without moving them: the order of the keys inside an MFMA's
// contraction is free, so V is read (transposed, ds_read_b64_tr_b16) in the
// order in which S^T left the keys.  The accumulators' columns are the rows
// too, so a row's rescaling factor is already in the lane that needs it.
// P is rounded to the operands' type (to nearest), which is what the MFMA
// takes; m, l and both accumulators are float32.
#pragma once

#include <type_traits>

#include "msa_device.hpp"

namespace msa {

struct AttnParams {
  const uint8_t* q;            // query rows, q_row_stride bytes per token
  const uint8_t* k;
  const uint8_t* v;
  const int32_t* block_table;  // [B, MB] (paged) or nullptr
  const int32_t* cu_q;         // [B+1]
  const int32_t* kv_len;       // [B]
  const int32_t* blocks;       // [T, Hkv, nsel] selected blocks, or nullptr
  uint8_t* out;                // [T, Hq, D], the query's type
  float* lse;                  // [T, Hq] or nullptr
  float* part_o;               // [nsplit, T, Hq, D], with nsplit > 1
  float2* part_ml;             // [nsplit, T, Hq]: m and l
  int64_t q_row_stride;        // bytes between query tokens
  int64_t k_page_stride, v_page_stride;   // bytes between pages (paged)
  int32_t k_row_stride, v_row_stride;     // bytes between key tokens
  int32_t k_head_stride, v_head_stride;   // bytes between KV heads
  int64_t keys;                // packed key tokens (T2)
  int64_t T;
  int32_t B, Hq, Hkv, g;
  int32_t MB, NP, nsel;
  int32_t paged, causal;
  float c;                     // softmax_scale * log2(e)
  int32_t hpt, tpt, hchunks, ntiles;      // as in Params
  int32_t nsplit;              // parts that a tile's blocks are split into, at most
  int32_t min_blocks;          // blocks per part at least
  int32_t join_rows;           // rows of a wave of attn_join_kernel
  int32_t balanced;            // dense tiles are split by attn_part
  float per_target;            // 1 / the parts per KV head that attn_part aims at
};

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A tile of query tokens of one request.
struct AttnTile {
  int valid;
  int t0, ntok, i0;            // first token, tokens, index of the first in the request
  int b, Lq, L;                // request, its new tokens, its keys that exist
  int len;                     // kv_len of the request (positions follow from it)
  int64_t koff;                // packed offset of the request's keys
};

// Keys that exist of a request's kv, packed ones from koff on.
__device__ __forceinline__ int keys_there(const AttnParams& p, int kv, int64_t koff) {
  return (int)(p.paged ? min((int64_t)kv, (int64_t)p.MB * kP)
                       : max(min((int64_t)kv, p.keys - koff), (int64_t)0));
}

// Tile `tin` of request b, which begins at token t0 with lq new tokens and kv
// keys.  Lengths that break the rules (negative, past the tensors) are cut to
// what the tensors hold, so that no address leaves them.
__device__ __forceinline__ void set_tile(const AttnParams& p, AttnTile& w, int b, int tin, int t0,
                                         int lq, int kv, int64_t koff) {
  w.b = b;
  w.Lq = lq;
  w.i0 = tin * p.tpt;
  w.t0 = t0 + w.i0;
  const int64_t room = p.T - (int64_t)w.t0;
  w.ntok = (int)min((int64_t)min(p.tpt, w.Lq - w.i0), w.t0 < 0 ? (int64_t)0 : room);
  w.koff = koff;
  w.len = kv;
  w.L = keys_there(p, kv, koff);
  w.valid = w.ntok > 0;
}

// The tile-th tile of tpt tokens: a prefix sum of the requests' tile counts,
// 64 requests at a time (every lane of the wave takes part).
__device__ __forceinline__ AttnTile attn_tile(const AttnParams& p, int tile) {
  AttnTile w;
  w.valid = 0;
  const int l = lane_id();
  int acc = 0;
  int64_t kacc = 0;
  for (int base = 0; base < p.B; base += 64) {
    const int b = base + l;
    int t0 = 0, lq = 0, kv = 0;
    if (b < p.B) {
      t0 = p.cu_q[b];
      lq = max(p.cu_q[b + 1] - t0, 0);
      kv = max(p.kv_len[b], 0);
    }
    int n = lq > 0;
    if (__ballot(lq > p.tpt)) n = (int)(((uint32_t)lq + p.tpt - 1) / (uint32_t)p.tpt);
    const int incl = wave_incl_scan(n);
    const int64_t kincl = p.paged ? kv : wave_incl_scan((int64_t)kv);
    const int total = lane_at(incl, 63);
    if (tile < acc + total) {
      const unsigned long long m = __ballot(acc + incl > tile);
      const int src = __builtin_amdgcn_readfirstlane(__ffsll((long long)m) - 1);
      const int tin = tile - (acc + lane_at(incl, src) - lane_at(n, src));
      set_tile(p, w, base + src, tin, lane_at(t0, src), lane_at(lq, src), lane_at(kv, src),
               kacc + lane_at(kincl, src) - lane_at(kv, src));
      return w;
    }
    acc += total;
    if (!p.paged) kacc += lane_at(kincl, 63);
  }
  return w;
}

// Part `unit` of a launch whose tiles are split by their own lengths: parts of
// at most a `target`-th of all blocks (of one head), min_blocks blocks or more,
// so that long requests get many and short ones stay whole.  The parts of up to
// 64 requests (one a lane) are handed out longest first, and the launch ends
// evenly whatever order the requests come in.  A request's tiles get as many
// parts each as its last one needs; there are at most target + 1 + ntiles parts.
struct AttnPart {
  AttnTile w;
  int split, parts;
};
__device__ __forceinline__ AttnPart attn_part(const AttnParams& p, int unit) {
  AttnPart r;
  r.w.valid = 0;
  const int l = lane_id();
  int t0 = 0, lq = 0, kv = 0, n = 0, nb = 0;     // of request base + l
  int64_t koff = 0, kacc = 0;
  auto load = [&](int base) {
    const int b = base + l;
    t0 = lq = kv = 0;
    if (b < p.B) {
      t0 = p.cu_q[b];
      lq = max(p.cu_q[b + 1] - t0, 0);
      kv = max(p.kv_len[b], 0);
    }
    n = lq > 0;
    if (__ballot(lq > p.tpt)) n = (int)(((uint32_t)lq + p.tpt - 1) / (uint32_t)p.tpt);
    if (!p.paged) {
      const int64_t incl = wave_incl_scan((int64_t)kv);
      koff = kacc + incl - kv;
      kacc += lane_at(incl, 63);
    }
    nb = (int)(((uint32_t)keys_there(p, kv, koff) + kP - 1) / kP);
  };
  // Sizes in float32, which spares the prologue integer divisions; they and the
  // quotients are taken low by more than what rounding adds, so that exact
  // quotients stay whole, and the bound has a part more for that.
  float total = 0.f;                             // of each lane, then of the wave
  if (p.nsplit > 1) {
    for (int base = 0; base < p.B; base += 64) {
      load(base);
      total += (float)n * (float)nb;
    }
    total = lane_at(wave_incl_scan(total), 63);
  }
  const float size = fmaxf(ceilf(total * p.per_target * 0.9999f), (float)p.min_blocks);
  const float per_size = 0.9999f * __builtin_amdgcn_rcpf(size);
  auto parts_of = [&]() -> int { return min((int)((float)nb * per_size) + 1, p.nsplit); };
  auto take = [&](int b, int src, int off, int parts) {
    r.parts = parts;
    // (a request's last tiles first)
    const int tin = parts == 1 ? off : (int)((uint32_t)off / (uint32_t)parts);
    r.split = off - tin * parts;
    set_tile(p, r.w, b, lane_at(n, src) - 1 - tin, lane_at(t0, src), lane_at(lq, src),
             lane_at(kv, src), lane_at(koff, src));
  };
  if (p.B <= 64) {
    if (p.nsplit == 1) load(0);
    const int parts = parts_of();
    // (the length of a part above the lane's number; lanes without a request
    // come last)
    const int len = n > 0 ? (int)((float)nb * __builtin_amdgcn_rcpf((float)parts)) : 0;
    const int key = l < p.B ? len << 6 | (63 - l) : -l;
    int rank = max(l - p.B, 0);
    for (int j = 0; j < p.B; ++j) rank += lane_at(key, j) > key;
    // lane i receives the number of the lane of rank i
    const int from = __builtin_amdgcn_ds_permute(rank << 2, l);
    const int units = __shfl(n * parts, from);
    const int incl = wave_incl_scan(units);
    if (unit >= lane_at(incl, 63)) return r;
    const int at = __builtin_amdgcn_readfirstlane(__ffsll((long long)__ballot(incl > unit)) - 1);
    const int src = lane_at(from, at);
    take(src, src, unit - (lane_at(incl, at) - lane_at(units, at)), lane_at(parts, src));
    return r;
  }
  int acc = 0;
  kacc = 0;
  for (int base = 0; base < p.B; base += 64) {
    load(base);
    const int parts = parts_of();
    const int units = n * parts;
    const int incl = wave_incl_scan(units);
    const int sum = lane_at(incl, 63);
    if (unit < acc + sum) {
      const int src =
          __builtin_amdgcn_readfirstlane(__ffsll((long long)__ballot(acc + incl > unit)) - 1);
      take(base + src, src, unit - (acc + lane_at(incl, src) - lane_at(units, src)),
           lane_at(parts, src));
      return r;
    }
    acc += sum;
  }
  return r;
}

// Last visible key of the request's i-th new token: kv_len - L_q + i under
// the causal mode, the last key without it.
__device__ __forceinline__ int attn_last(const AttnParams& p, const AttnTile& w, int i) {
  return min(p.causal ? w.len - w.Lq + i : w.L - 1, w.L - 1);
}

// Two floats -> one register of two 16-bit operands, rounded to nearest.
template <int KK>
__device__ __forceinline__ int pack2(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) float f32x2;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const f32x2 v = {a, b};
  if constexpr (KK == KBF16)
    return __builtin_bit_cast(int, __builtin_convertvector(v, bf16x2));
  else
    return __builtin_bit_cast(int, __builtin_convertvector(v, f16x2));
}

// ds_read_b64_tr_b16: within each 16 lanes, lane i gives the address of
// columns 4 (i % 4) .. + 3 of row i / 4 of a 4 x 16 block of 16-bit elements
// and receives the four rows of column i.
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
__device__ __forceinline__ i32x2 lds_read_tr(const uint8_t* p) {
  return __builtin_bit_cast(
      i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// x[l] + x[l ^ 32], x[l] + x[l ^ 16] (as max_xor32 and max_xor16)
__device__ __forceinline__ float sum_xor32(float x) {
  uint32_t a = __builtin_bit_cast(uint32_t, x), b = a;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1\n\tv_add_f32 %0, %0, %1"
               : "+v"(a), "+v"(b));
  return __builtin_bit_cast(float, a);
}
__device__ __forceinline__ float sum_xor16(float x) {
  uint32_t a = __builtin_bit_cast(uint32_t, x), b = a;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\ts_nop 1\n\tv_add_f32 %0, %0, %1"
               : "+v"(a), "+v"(b));
  return __builtin_bit_cast(float, a);
}

// Registers whose loads are waited for here, not at their first use inside a
// loop, where the wait would count the loop's own copies.
__device__ __forceinline__ void landed(i32x4& x) { asm volatile("" : "+v"(x)); }

// m, the power of two that a row's weights 2^(S - m) are taken against, follows
// the row's running maximum with a lag: it moves, and the accumulators are
// rescaled, only when a score passes m + kReach, and then to kLift below that
// score.  Almost every stage after the first skips the rescaling; m cancels in
// out and is put back in lse.  (A row's own scores alone decide when its m
// moves, so its bits do not depend on the rows it shares a tile with.)
//  - bf16 weights have float32's range: no lift, a lag of 2^8.
//  - f16 weights end at 2^-24, in steps of that below 2^-14.  Against a largest
//    weight of 1 the keys 17 nats below a row's largest score (a sink's, say)
//    would drop out of the sum of values and stay in l: 32768 keys 18 nats below
//    a sink came out as 0 for 5e-4.  So the row's largest weight lies in
//    [2^11, 2^15] (65504 is the type's largest), what rounds to 0 is 2^-36 of it,
//    and steps grow coarser than 2^-11 only 17 nats below it.  The lag is 2^4 so
//    that the lift may be that large.
template <int KK>
constexpr float kLift = KK == KF16 ? 11.f : 0.f;
template <int KK>
constexpr float kReach = KK == KF16 ? 15.f : 8.f;

// The row's m with the largest score so far, mx, in sight.
template <int KK>
__device__ __forceinline__ float moved(float m, float mx) {
  return mx > m + kReach<KK> ? mx - kLift<KK> : m;
}

// ln of the sum l 2^m, without the lift's cancelling digits.
template <int KK>
__device__ __forceinline__ float lse_of(float m, float l) {
  if (l == 0.f) return -__builtin_inff();
  return ((m + kLift<KK>) + __log2f(l * __builtin_exp2f(-kLift<KK>))) * kLn2;
}

// What the join needs to know of a row of a launch with split tiles, written by
// its first part: that the row is whole (a NaN that no m is: m never is one), or
// which parts there are not.  `lane` of `lanes` lanes.
constexpr uint32_t kWholeBits = 0x7FEBCDEFu;
__device__ __forceinline__ void mark_parts(const AttnParams& p, int64_t row, int parts, int lane,
                                           int lanes) {
  if (p.nsplit == 1) return;
  const int64_t rows = p.T * p.Hq;
  if (parts == 1) {
    if (lane == 0) p.part_ml[row].x = __builtin_bit_cast(float, kWholeBits);
    return;
  }
  for (int s = parts + lane; s < p.nsplit; s += lanes)
    p.part_ml[s * rows + row] = float2{-__builtin_inff(), 0.f};
}

// NI copies of 1 KB, a wave's lanes' pieces at the byte offsets `of` of a raw
// buffer of `bytes`; ONCE: rows that nobody else reads (the nontemporal hint).
template <int NI, bool ONCE = false>
__device__ __forceinline__ void copy_rows(uint8_t* dst, const uint8_t* src, int bytes,
                                          const uint32_t* of) {
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(src), 0, bytes, kBufferWord3);
#pragma unroll
  for (int i = 0; i < NI; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (__attribute__((address_space(3))) void*)(dst + 1024 * i), 16, of[i], 0, 0,
        ONCE ? 2 : 0);
}

// ---------------------------------------------------------------------------
// Few rows: 16 rows a tile, the keys split over waves and workgroups.
//
// A tile is tpt tokens x hpt heads (at most 16 rows) of one KV head.  Its
// blocks -- all visible ones, or the token's selected ones -- are split into
// nsplit parts, one workgroup each; within a workgroup wave w takes keys
// 32w .. 32w + 31 of every block, with its own m, l and accumulators, and the
// four waves' results are joined through LDS at the end.  The bound is the
// reading of keys and values: each wave copies its 16 KB of a block straight
// into its own part of the LDS, one block ahead, with no barrier in the loop.
// 64 requests of up to 8192 keys, 8 KV heads, 1.17 GB: 190 us, 6.2 TB/s, which is
// what a large read reaches.
// A request of one tile (and head chunk) is the only reader of its rows, and its
// copies say so with the nontemporal hint; other tiles' copies do not.  With the
// hint and without: 64 requests of one token, up to 8000 keys, 157 and 174 us, of
// two tokens 180 and 200; 63 of one token beside one of 900 over 32768 keys, 32
// heads of their own, 3822 and 2192 (tile by tile, as here).
// Stages of 16 keys with two workgroups a CU instead: 207 us against 199.
// ---------------------------------------------------------------------------

constexpr int kAttnRows = 16;
constexpr int kRowWaves = 4;
constexpr int kRowStage = 16384;     // 32 keys' K and V rows

template <int KK, bool SEL>
__global__ __launch_bounds__(256, 1) void attn_rows_kernel(AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRowWaves][2][kRowStage];
  int rest = blockIdx.x, split = 0, parts = 1;
  if constexpr (SEL) {
    split = rest % p.nsplit;
    rest /= p.nsplit;
  }
  const int hc = rest % p.hchunks;
  rest /= p.hchunks;
  const int hk = rest % p.Hkv;
  AttnTile w;
  if constexpr (SEL) {
    w = attn_tile(p, rest / p.Hkv);
  } else {
    const AttnPart part = attn_part(p, rest / p.Hkv);
    w = part.w;
    split = part.split;
    parts = part.parts;
  }
  if (!w.valid) return;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane_id();
  const int n = l & 15, G = l >> 4;

  // this lane's row (column n of every MFMA result)
  const int ti = n / p.hpt;
  const int hg = hc * p.hpt + (n - ti * p.hpt);
  const bool row_ok = ti < w.ntok && ti < p.tpt && hg < p.g;
  const int lim = row_ok ? attn_last(p, w, w.i0 + ti) : -1;
  const int lim_lo = attn_last(p, w, w.i0);
  const int lim_hi = attn_last(p, w, w.i0 + w.ntok - 1);
  const int nb = lim_hi >= 0 ? lim_hi / kP + 1 : 0;    // blocks with a visible key

  // the part's blocks: [b0, b1) of the visible ones, or of the selected list
  int sel = -1, total = nb;
  if constexpr (SEL) {
    // one entry per lane; entries outside the visible blocks and repeats of
    // an earlier entry count as none; the rest move to the front.  (The top-k
    // selection gives ascending entries in front of its -1 tail: nothing to
    // look for then.)
    int e = l < p.nsel ? p.blocks[((int64_t)w.t0 * p.Hkv + hk) * p.nsel + l] : -1;
    bool ok = e >= 0 && e < nb;
    const int prev = __shfl_up(e, 1);
    const unsigned long long front = __ballot(ok);
    if ((front & (front + 1)) || __ballot(ok && l > 0 && prev >= e)) {
      for (int i = 0; i + 1 < p.nsel; ++i) ok = ok && !(l > i && e == lane_at(e, i));
    }
    const unsigned long long m = __ballot(ok);
    total = __popcll(m);
    // lane i receives the i-th entry: every kept lane sends its own to its rank
    const int rank = __popcll(m & ((1ull << l) - 1));
    sel = __builtin_amdgcn_ds_permute((ok ? rank : 63) << 2, e);
    if (l >= total) sel = -1;
  }
  if constexpr (SEL) parts = max(1, min(p.nsplit, (total + p.min_blocks - 1) / p.min_blocks));
  const int b0 = (int)((int64_t)total * split / parts);
  const int b1 = split < parts ? (int)((int64_t)total * (split + 1) / parts) : b0;
  if (SEL && split >= parts) return;
  const int nst = max(b1 - b0, 0);

  const int64_t out_row = ((int64_t)(w.t0 + ti) * p.Hq + hk * p.g + hg);

  // query fragments: k step s of group G is elements 32 s + 8 G .. + 7
  i32x4 qv[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) qv[s] = i32x4{0, 0, 0, 0};
  if (row_ok) {
    const uint8_t* qr = p.q + (int64_t)(w.t0 + ti) * p.q_row_stride + (hk * p.g + hg) * (2 * kD);
#pragma unroll
    for (int s = 0; s < 4; ++s) qv[s] = ld16(qr + 64 * s + 16 * G);
  }

  // page numbers, one per lane, 64 blocks at a time (-1: no page)
  int pidx = -1, pbase = 0;
  auto page_of = [&](int blk) -> int {
    const int pg = p.block_table[(int64_t)w.b * p.MB + blk];
    return pg >= 0 && pg < p.NP ? pg : -1;
  };
  auto load_pages = [&](int from) {
    pbase = from;
    const int i = b0 + from + l;
    if constexpr (!SEL) {
      pidx = consumed(p.paged && from + l < nst ? page_of(i) : -1);
    }
  };
  if constexpr (SEL) {
    // (selected blocks: at most 64, all at once)
    if (l < total) pidx = p.paged ? page_of(sel) : -1;
  } else {
    load_pages(0);
  }

  // copies of one block's 32 keys: instruction i brings rows 4 i .. 4 i + 3
  // (16 lanes to a row), the 16-byte chunks of row r permuted by the XORs
  // that the reads below undo
  const int cr = l >> 4, cc = l & 15;
  uint8_t* const mine = &ring[wave][0][0];
  struct Block { int beta, page; };
  auto block_at = [&](int s) -> Block {
    Block x;
    if constexpr (SEL) {
      x.beta = lane_at(sel, b0 + s);
      x.page = lane_at(pidx, b0 + s);
    } else {
      x.beta = b0 + s;
      x.page = lane_at(pidx, s - pbase);
    }
    return x;
  };
  struct Rows { const uint8_t *k, *v; int n; };
  auto rows_of = [&](const Block& x) -> Rows {
    const int j0 = x.beta * kP + 32 * wave;
    const bool there = !p.paged || x.page >= 0;
    const int64_t pg = max(x.page, 0);
    const int64_t kb = p.paged ? pg * p.k_page_stride + (int64_t)(32 * wave) * p.k_row_stride
                               : (w.koff + j0) * p.k_row_stride;
    const int64_t vb = p.paged ? pg * p.v_page_stride + (int64_t)(32 * wave) * p.v_row_stride
                               : (w.koff + j0) * p.v_row_stride;
    return Rows{p.k + uniform64(kb + (int64_t)hk * p.k_head_stride),
                p.v + uniform64(vb + (int64_t)hk * p.v_head_stride),
                __builtin_amdgcn_readfirstlane(there ? max(0, min(32, lim_hi + 1 - j0)) : 0)};
  };
  uint32_t kof[8], vof[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + cr;
    kof[i] = (uint32_t)(r * p.k_row_stride + 16 * (cc ^ (r & 15)));
    vof[i] = (uint32_t)(r * p.v_row_stride + 16 * (cc ^ ((r & 7) << 1)));
  }

  const bool once = __builtin_amdgcn_readfirstlane(w.Lq <= p.tpt && p.hchunks == 1);
  auto copy = [&](uint8_t* dst, const Rows& r) __attribute__((always_inline)) {
    if (once) {
      copy_rows<8, true>(dst, r.k, r.n * p.k_row_stride, kof);
      copy_rows<8, true>(dst + 8192, r.v, r.n * p.v_row_stride, vof);
    } else {
      copy_rows<8>(dst, r.k, r.n * p.k_row_stride, kof);
      copy_rows<8>(dst + 8192, r.v, r.n * p.v_row_stride, vof);
    }
  };

  f32x4 o[8];
  float m, lsum;

  // One block's keys and values at kt; with CAREFUL as in attn_tile_kernel.
  // (kt is one half of the ring while copies into the other are in flight, and
  // the parameters say that the two do not overlap: reads of LDS that may
  // alias a copy in flight would wait for all copies.)
  auto step = [&](const uint8_t* __restrict kt, uint8_t* __restrict dst, const Block& cur,
                  const Rows& next, bool more, auto careful) __attribute__((always_inline)) {
    if constexpr (!decltype(careful)::value) {
      if (more) {
        copy(dst, next);
        asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
    }
    const uint8_t* vt = kt + 8192;
    const int j0 = cur.beta * kP + 32 * wave;
    const bool there = !p.paged || cur.page >= 0;

    // S^T: tile a holds keys j0 + 4 G + r, tile b keys j0 + 16 + 4 G + r of row n
    f32x4 sa = {0.f, 0.f, 0.f, 0.f}, sb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = ((4 * k + G) ^ n) << 4;
      sa = mfma16x16x32<KK>(*reinterpret_cast<const i32x4*>(kt + n * 256 + ch), qv[k], sa);
      sb = mfma16x16x32<KK>(*reinterpret_cast<const i32x4*>(kt + (16 + n) * 256 + ch), qv[k], sb);
    }
    if (!there || j0 + 31 > lim_lo) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = j0 + 4 * G + r;
        sa[r] = there && j <= lim ? sa[r] : -__builtin_inff();
        sb[r] = there && j + 16 <= lim ? sb[r] : -__builtin_inff();
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(sa[0], sa[1]), fmaxf(sa[2], sa[3])),
                     fmaxf(fmaxf(sb[0], sb[1]), fmaxf(sb[2], sb[3])));
    mx = max_xor32(max_xor16(mx)) * p.c;
    if (__ballot(mx > m + kReach<KK>)) {
      const float mn = moved<KK>(m, mx);
      const float alpha = exp2_hw(m - (mn == -__builtin_inff() ? 0.f : mn));
      m = mn;
      lsum *= alpha;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] *= alpha;
    }
    const float ms = m == -__builtin_inff() ? 0.f : m;
    float pa[4], pb[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      pa[r] = exp2_hw(__builtin_fmaf(sa[r], p.c, -ms));
      pb[r] = exp2_hw(__builtin_fmaf(sb[r], p.c, -ms));
    }
    lsum += ((pa[0] + pa[1]) + (pa[2] + pa[3])) + ((pb[0] + pb[1]) + (pb[2] + pb[3]));
    const i32x4 pf = {pack2<KK>(pa[0], pa[1]), pack2<KK>(pa[2], pa[3]), pack2<KK>(pb[0], pb[1]),
                      pack2<KK>(pb[2], pb[3])};
    auto value = [&](int d) -> i32x4 {
      const int r = 4 * G + (n >> 2);
      const int ch = ((2 * d + ((n >> 1) & 1)) ^ ((r & 7) << 1)) * 16 + (n & 1) * 8;
      const i32x2 v0 = lds_read_tr(vt + r * 256 + ch);
      const i32x2 v1 = lds_read_tr(vt + (r + 16) * 256 + ch);
      return i32x4{v0[0], v0[1], v1[0], v1[1]};
    };
    if constexpr (!decltype(careful)::value) {
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] = mfma16x16x32<KK>(value(d), pf, o[d]);
    } else {
      for (int tk = 0; tk < w.ntok; ++tk) {
        const int end = attn_last(p, w, w.i0 + tk);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          i32x4 v = value(d);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + 16 * (e >> 1) + 4 * G + 2 * (e & 1);
            v[e] = j + 1 <= end ? v[e] : j <= end ? v[e] & 0xFFFF : 0;
          }
          const f32x4 x = mfma16x16x32<KK>(v, pf, o[d]);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[d][r] = ti == tk ? x[r] : o[d][r];
        }
      }
    }
  };

#pragma unroll
  for (int s = 0; s < 4; ++s) landed(qv[s]);
  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = -__builtin_inff();
    lsum = 0.f;
    if (nst <= 0) return;
    if (!SEL && pbase > 0) load_pages(0);
    Block cur = block_at(0);
    Rows r = rows_of(cur);
    if constexpr (!decltype(careful)::value) {
      copy(mine, r);
    }
    for (int s = 0; s < nst; ++s) {
      Block next = cur;
      if constexpr (decltype(careful)::value) {
        if (!SEL && s - pbase >= 64) load_pages(s);
        cur = block_at(s);
        r = rows_of(cur);
        wave_lds_sync();
        for (int i = 0; i < 8; ++i) {
          const bool ok = 4 * i + cr < r.n;
          const i32x4 zero = {0, 0, 0, 0};
          *reinterpret_cast<i32x4*>(mine + 1024 * i + 16 * l) = ok ? ld16(r.k + kof[i]) : zero;
          *reinterpret_cast<i32x4*>(mine + 8192 + 1024 * i + 16 * l) =
              ok ? ld16(r.v + vof[i]) : zero;
        }
        wave_lds_sync();
        step(mine, mine + kRowStage, cur, r, false, careful);
      } else {
        if (s + 1 < nst) {
          if (!SEL && s + 1 - pbase >= 64) load_pages(s + 1);
          next = block_at(s + 1);
          r = rows_of(next);
        }
        // (the reads of the half that is written next are done)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        step(mine + (s & 1) * kRowStage, mine + ((s + 1) & 1) * kRowStage, cur, r, s + 1 < nst,
             careful);
        cur = next;
      }
    }
  };

  pass(std::false_type{});
  if (w.ntok > 1) {
    float odd = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) odd += o[d][r] - o[d][r];
    if (__ballot(row_ok && odd != 0.f)) pass(std::true_type{});
  }

  // join the four waves: each writes its accumulators, m and l, then wave w
  // joins head elements 32 w .. 32 w + 31
  lsum = sum_xor32(sum_xor16(lsum));
  __syncthreads();
  float* const ol = reinterpret_cast<float*>(&ring[0][0][0]);    // [wave][row][132]
  constexpr int OS = 132;                                        // (row stride: no bank conflicts)
  float* const mls = ol + kRowWaves * kAttnRows * OS;            // [wave][row][2]
#pragma unroll
  for (int d = 0; d < 8; ++d)
    *reinterpret_cast<f32x4*>(ol + (wave * kAttnRows + n) * OS + 16 * d + 4 * G) = o[d];
  if (G == 0) {
    mls[(wave * kAttnRows + n) * 2] = m;
    mls[(wave * kAttnRows + n) * 2 + 1] = lsum;
  }
  __syncthreads();
  float mt = -__builtin_inff();
#pragma unroll
  for (int u = 0; u < kRowWaves; ++u) mt = fmaxf(mt, mls[(u * kAttnRows + n) * 2]);
  const float ms = mt == -__builtin_inff() ? 0.f : mt;
  float lt = 0.f;
  f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < kRowWaves; ++u) {
    const float a = exp2_hw(mls[(u * kAttnRows + n) * 2] - ms);
    lt += a * mls[(u * kAttnRows + n) * 2 + 1];
    const float* src = ol + (u * kAttnRows + n) * OS + 32 * wave + 8 * G;
    s0 += a * *reinterpret_cast<const f32x4*>(src);
    s1 += a * *reinterpret_cast<const f32x4*>(src + 4);
  }
  if (!row_ok) return;
  const int64_t rows = p.T * p.Hq;
  if (wave == 0 && split == 0) mark_parts(p, out_row, parts, G, 4);
  if (parts > 1) {
    const int64_t pr = split * rows + out_row;
    if (wave == 0 && G == 0) p.part_ml[pr] = float2{mt, lt};
    if (nst > 0) {
      float* dst = p.part_o + pr * kD + 32 * wave + 8 * G;
      *reinterpret_cast<f32x4*>(dst) = s0;
      *reinterpret_cast<f32x4*>(dst + 4) = s1;
    }
    return;
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  const i32x4 res = {pack2<KK>(s0[0] * inv, s0[1] * inv), pack2<KK>(s0[2] * inv, s0[3] * inv),
                     pack2<KK>(s1[0] * inv, s1[1] * inv), pack2<KK>(s1[2] * inv, s1[3] * inv)};
  *reinterpret_cast<i32x4*>(p.out + out_row * (2 * kD) + 64 * wave + 16 * G) = res;
  if (p.lse && wave == 0 && G == 0)
    p.lse[out_row] = lse_of<KK>(mt, lt);
}

// ---------------------------------------------------------------------------
// The join of a split tile's parts: a wave takes join_rows rows, of which it
// passes over those that were not split, one by one with half a wave per part
// (32 lanes of 16 bytes are a part's row), two pairs of parts in flight.  Bound by
// latency and then memory: 4096 whole rows 2.8 us, 4096 in 3 parts 4.7, 22624
// rows in up to 6 parts 9.4; in 3 parts (41 MB) 9.7 us against 11.7 with a whole
// wave per part, one after the other.  Rows that no request holds are left as
// they are.
// ---------------------------------------------------------------------------

template <int KK>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  const int l = lane_id();
  const int64_t rows = p.T * p.Hq;
  const int64_t end = min(rows, (int64_t)max(p.cu_q[p.B], 0) * p.Hq);
  const int64_t from = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * p.join_rows;
  // which of the wave's rows are in parts
  bool open = false;
  if (l < p.join_rows && from + l < end && from + l >= (int64_t)p.cu_q[0] * p.Hq)
    open = __builtin_bit_cast(uint32_t, p.part_ml[from + l].x) != kWholeBits;
  for (unsigned long long todo = __ballot(open); todo; todo &= todo - 1) {
    const int64_t row = from + (__ffsll((long long)todo) - 1);
    // parts that the tile did not need, or that saw nothing, hold no sums: l = 0
    // (NaN where anything seen was no number)
    float2 ml = {-__builtin_inff(), 0.f};
    if (l < p.nsplit) ml = p.part_ml[l * rows + row];
    float mt = max_xor32(max_xor16(ml.x));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
    const float ms = mt == -__builtin_inff() ? 0.f : mt;
    const float a = ml.y == 0.f ? 0.f : exp2_hw(ml.x - ms);
    float lt = sum_xor32(sum_xor16(a * ml.y));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) lt += __shfl_xor(lt, d);
    const int half = l >> 5;
    const unsigned long long filled = __ballot(ml.y != 0.f);
    auto part = [&](int s) -> f32x4 {      // its share of elements 4 (l % 32) .. + 3
      const f32x4 none = {0.f, 0.f, 0.f, 0.f};
      if (!(filled >> s & 1)) return none;
      return *reinterpret_cast<const f32x4*>(p.part_o + (s * rows + row) * kD + 4 * (l & 31));
    };
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.nsplit; s += 4) {
      if (!(filled >> s)) break;
      const int s0 = s + half, s1 = s + 2 + half;      // (at most 66: tested before use)
      const f32x4 x0 = s0 < p.nsplit ? part(s0) : f32x4{0.f, 0.f, 0.f, 0.f};
      const f32x4 x1 = s1 < p.nsplit ? part(s1) : f32x4{0.f, 0.f, 0.f, 0.f};
      o += __shfl(a, s0 & 63) * x0 + __shfl(a, s1 & 63) * x1;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = sum_xor32(o[r]);
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    if (half == 0)
      *reinterpret_cast<i32x2*>(p.out + row * (2 * kD) + 8 * l) =
          i32x2{pack2<KK>(o[0] * inv, o[1] * inv), pack2<KK>(o[2] * inv, o[3] * inv)};
    if (p.lse && l == 0)
      p.lse[row] = lse_of<KK>(mt, lt);
  }
}

// ---------------------------------------------------------------------------
// What the two kernels of many rows share: stages of 64 keys, two per block,
// and where their rows come from.
// ---------------------------------------------------------------------------

constexpr int kTileKeys = 64;
constexpr int kNoPage = 1 << 30;

// A block of the walk: its number, whether it is on a page, the places of its rows.
struct Entry {
  int beta;
  bool there;
  int64_t k, v;
};

// Entries of the walk, their numbers (kNoPage: on no page) and places held one
// per lane, 64 at a time, so that a stage takes a few readlanes and no address
// arithmetic (scalar multiplications per stage held up every wave for hundreds
// of cycles).
struct BlockList {
  int bidx = 0, base = 0;
  int64_t kat = 0, vat = 0;

  // Entries from .. from + 63 of `count`; number(i) is the number of entry i.
  template <typename F>
  __device__ __forceinline__ void load(const AttnParams& p, const AttnTile& w, int hk, int from,
                                       int count, F number) {
    const int l = lane_id();
    base = from;
    bidx = kNoPage;
    kat = vat = 0;
    if (from + l < count) {
      bidx = number(from + l);
      if (p.paged) {
        const int pg = p.block_table[(int64_t)w.b * p.MB + bidx];
        if (pg >= 0 && pg < p.NP) {
          kat = pg * p.k_page_stride;
          vat = pg * p.v_page_stride;
        } else {
          bidx |= kNoPage;
        }
      } else {
        kat = (w.koff + (int64_t)bidx * kP) * p.k_row_stride;
        vat = (w.koff + (int64_t)bidx * kP) * p.v_row_stride;
      }
    }
    bidx = consumed(bidx);
    kat += (int64_t)hk * p.k_head_stride;
    vat += (int64_t)hk * p.v_head_stride;
  }
  __device__ __forceinline__ Entry at(int e) const {
    const int x = lane_at(bidx, e - base);
    return Entry{x & (kNoPage - 1), x < kNoPage, lane_at(kat, e - base), lane_at(vat, e - base)};
  }
};

// Where the keys of half `in` of a block lie, and how many bytes of them there
// are to the tile's last visible one, lim_hi.
struct StageRows {
  const uint8_t *k, *v;
  int kb, vb;
};
__device__ __forceinline__ StageRows stage_rows(const AttnParams& p, int lim_hi, const Entry& x,
                                                int in) {
  const int left = x.there ? max(0, min(kTileKeys, lim_hi + 1 - x.beta * kP - in * kTileKeys)) : 0;
  return StageRows{p.k + x.k + in * kTileKeys * p.k_row_stride,
                   p.v + x.v + in * kTileKeys * p.v_row_stride,
                   __builtin_amdgcn_readfirstlane(left * p.k_row_stride),
                   __builtin_amdgcn_readfirstlane(left * p.v_row_stride)};
}

// A wave's NI copies of a stage's rows through registers, for the careful pass
// (whose copies need not overlap anything); kof, vof as for copy_rows.
template <int NI>
__device__ __forceinline__ void copy_plain(const AttnParams& p, uint8_t* kring, uint8_t* vring,
                                           int wave, const StageRows& r, const uint32_t* kof,
                                           const uint32_t* vof) {
  const int l = lane_id();
  for (int i = 0; i < NI; ++i) {
    const int row = (wave * NI + i) * 4 + (l >> 4);
    const int at = (wave * NI + i) * 1024 + 16 * l;
    const i32x4 zero = {0, 0, 0, 0};
    *reinterpret_cast<i32x4*>(kring + at) =
        row * p.k_row_stride < r.kb ? ld16(r.k + kof[i]) : zero;
    *reinterpret_cast<i32x4*>(vring + at) =
        row * p.v_row_stride < r.vb ? ld16(r.v + vof[i]) : zero;
  }
}

// ---------------------------------------------------------------------------
// Many rows: 32 rows a wave, NW waves a workgroup, every wave reading the same
// stages of 64 keys from the LDS.
//
// The stages' K and V rows are copied straight into two-deep LDS rings one
// stage ahead, through raw buffers that end at the tile's last visible key, so
// rows past it read zeros (a stored NaN there cannot reach a sum).
//
// Bound by the matrix units and, before they are full, by the card's power: 2048
// tokens over 32768 keys, 32 heads on 4 KV heads, take 907 to 988 us by card
// (1.08 to 1.17 PFLOP/s; 8192^3 products of the library reach 1.24), with the MFMA
// busy in 56% of the cycles, vector instructions in 40%, the LDS in 25% without
// bank conflicts.  32 rows a wave, because a fragment of K or V out of the LDS
// then feeds the largest MFMA; 8 waves a workgroup share a stage's copies (4
// where 256 rows would leave CUs without work).  Two waves a SIMD fill the gaps
// between one wave's MFMAs and its weights.  Without effect within 1%: the next
// stage's scores beside this one's weights by hand (spills: slower), wave
// priorities, tiles handed out by weight, leaving out a last half block that no
// row sees.
//
// A weight of 0 does not hide an infinity or NaN in the value of a key that
// only other rows of the tile see.  So a tile that ends with an accumulator
// that is not finite is taken again with the second product formed token by
// token, from values with the unseen rows cleared (careful); a tile of finite
// inputs costs only the look at its accumulators.
// ---------------------------------------------------------------------------

template <int KK, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_tile_kernel(AttnParams p) {
  constexpr int SB = kTileKeys * 256;          // bytes of a stage's K (or V) rows
  constexpr int NI = SB / 1024 / NW;           // copies of each per wave and stage
  // One LDS object, cut up by hand: with several, the compiler attaches alias
  // scopes to the copies into the ring and then waits for them before every
  // read of it.
  constexpr int kFlagAt = 4 * SB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFlagAt + 16];
  uint8_t* const kring = lds;                                       // [2][64 K rows]
  uint8_t* const vring = lds + 2 * SB;                              // [2][64 V rows]
  int* const flag = reinterpret_cast<int*>(lds + kFlagAt);
  // heavy tiles (the last tokens of a request see the most keys) first; the
  // KV head changes fastest, so that with 8 XCDs taking workgroups in turn an
  // XCD's L2 holds the keys of few heads
  int rest = blockIdx.x, split = 0;
  if (!p.balanced) {
    split = rest % p.nsplit;
    rest /= p.nsplit;
  }
  const int hc = rest % p.hchunks;
  rest /= p.hchunks;
  const int hk = rest % p.Hkv;
  rest /= p.Hkv;
  AttnTile w;
  int parts = p.nsplit;
  if (p.balanced) {
    const AttnPart part = attn_part(p, rest);
    w = part.w;
    split = part.split;
    parts = part.parts;
  } else {
    w = attn_tile(p, p.ntiles - 1 - rest);
  }
  if (!w.valid) return;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane_id();
  const int n = l & 31, h = l >> 5;
  const int row = wave * 32 + n;
  const int ti = row / p.hpt;
  const int hg = hc * p.hpt + (row - ti * p.hpt);
  const bool row_ok = row < p.hpt * p.tpt && ti < w.ntok && hg < p.g;
  const int lim = row_ok ? attn_last(p, w, w.i0 + ti) : -1;
  const int lim_lo = attn_last(p, w, w.i0);
  const int lim_hi = attn_last(p, w, w.i0 + w.ntok - 1);
  const int total = lim_hi >= 0 ? lim_hi / kP + 1 : 0;
  parts = max(1, min(parts, (total + p.min_blocks - 1) / p.min_blocks));
  if (split >= parts) return;
  const int b0 = (int)((int64_t)total * split / parts);
  const int b1 = (int)((int64_t)total * (split + 1) / parts);

  i32x4 qv[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) qv[s] = i32x4{0, 0, 0, 0};
  if (row_ok) {
    const uint8_t* qr = p.q + (int64_t)(w.t0 + ti) * p.q_row_stride + (hk * p.g + hg) * (2 * kD);
#pragma unroll
    for (int s = 0; s < 8; ++s) qv[s] = ld16(qr + 16 * (2 * s + h));
  }

  const int count = b1 - b0;
  BlockList list;
  auto load_entries = [&](int from) __attribute__((always_inline)) {
    list.load(p, w, hk, from, count, [&](int i) { return b0 + i; });
  };
  auto entry_at = [&](int e) __attribute__((always_inline)) -> Entry {
    if (e - list.base >= 64) load_entries(e);
    return list.at(e);
  };

  const int cr = l >> 4, cc = l & 15;
  uint32_t kof[NI], vof[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = (wave * NI + i) * 4 + cr;
    kof[i] = (uint32_t)(r * p.k_row_stride + 16 * (cc ^ (r & 15)));
    vof[i] = (uint32_t)(r * p.v_row_stride + 16 * (cc ^ ((r & 3) << 2)));
  }
  auto rows_of = [&](const Entry& x, int in) __attribute__((always_inline)) -> StageRows {
    return stage_rows(p, lim_hi, x, in);
  };

  f32x16 o[4];
  float m, lsum;

  // A stage in two parts: its scores from the K rows at kt, and what follows
  // from them with the V rows at vt.  (The copies that may be in flight go to
  // other parts of the rings, and the parameters say so, as in
  // attn_rows_kernel.)
  f32x16 st[2];
  auto scores = [&](const uint8_t* __restrict kt) __attribute__((always_inline)) {
    // S^T, two tiles of 32 keys: register r of tile t is key
    // j0 + 32 t + 8 (r / 4) + 4 h + r % 4 of row n
    st[0] = st[1] = f32x16{};
    // (K fragments are read KLEAD ahead of their MFMAs and pinned there: left to
    // itself the compiler read each right before its use, and every MFMA waited
    // for the LDS)
    constexpr int KLEAD = 4;
    i32x4 kf[16];
    auto key_frag = [&](int i) -> i32x4 {
      const int jj = 32 * (i >> 3) + n;
      return *reinterpret_cast<const i32x4*>(kt + jj * 256 +
                                             (((2 * (i & 7) + h) ^ (jj & 15)) << 4));
    };
#pragma unroll
    for (int i = 0; i < KLEAD; ++i) kf[i] = key_frag(i);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + KLEAD < 16) kf[i + KLEAD] = key_frag(i + KLEAD);
      st[i >> 3] = mfma32x32x16<KK>(kf[i], qv[i & 7], st[i >> 3]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto absorb = [&](const uint8_t* __restrict vt, const Entry& cur, int in, auto careful)
      __attribute__((always_inline)) {
    const int j0 = cur.beta * kP + in * kTileKeys;
    const bool there = cur.there;
    if (!there || j0 + kTileKeys - 1 > lim_lo) {
      // (compared as constants against one value per lane: the keys' numbers
      // themselves would take 32 registers through the whole loop)
      const int rel = there ? lim - j0 - 4 * h : -1;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          st[t][r] = 32 * t + 8 * (r >> 2) + (r & 3) <= rel ? st[t][r] : -__builtin_inff();
    }
    float mx = st[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, st[t][r]);
    mx = max_xor32(mx) * p.c;
    if (__ballot(mx > m + kReach<KK>)) {
      const float mn = moved<KK>(m, mx);
      const float alpha = exp2_hw(m - (mn == -__builtin_inff() ? 0.f : mn));
      m = mn;
      lsum *= alpha;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= alpha;
    }
    const float ms = m == -__builtin_inff() ? 0.f : m;
    float add = 0.f;
    i32x4 pf[4];
    // weights 2 i and 2 i + 1 of this lane's 32, rounded and packed
    auto weigh = [&](int i) __attribute__((always_inline)) {
      const float a = exp2_hw(__builtin_fmaf(st[i >> 3][2 * (i & 7)], p.c, -ms));
      const float b = exp2_hw(__builtin_fmaf(st[i >> 3][2 * (i & 7) + 1], p.c, -ms));
      add += a + b;
      pf[i >> 2][i & 3] = pack2<KK>(a, b);
    };
    // O^T += V^T P^T, 16 keys a step: registers 8 u .. 8 u + 7 of a tile are
    // keys 16 u + 4 h + {0..3} and 16 u + 8 + 4 h + {0..3}
    const int vi = l & 15;
    auto value = [&](int i) __attribute__((always_inline)) -> i32x4 {
      const int r = 16 * (i >> 2) + 4 * h + (vi >> 2);
      const int ch = ((4 * (i & 3) + 2 * ((l >> 4) & 1) + ((vi >> 1) & 1)) ^ ((r & 3) << 2)) * 16 +
                     (vi & 1) * 8;
      const i32x2 v0 = lds_read_tr(vt + r * 256 + ch);
      const i32x2 v1 = lds_read_tr(vt + (r + 8) * 256 + ch);
      return i32x4{v0[0], v0[1], v1[0], v1[1]};
    };
    if constexpr (!decltype(careful)::value) {
      // (a step's MFMAs run beside the next step's weights, each with one pair
      // of them and the read of a later operand, pinned)
      constexpr int VLEAD = 3;
      i32x4 vf[16];
#pragma unroll
      for (int i = 0; i < VLEAD; ++i) vf[i] = value(i);
#pragma unroll
      for (int i = 0; i < 4; ++i) weigh(i);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i + VLEAD < 16) vf[i + VLEAD] = value(i + VLEAD);
        o[i & 3] = mfma32x32x16<KK>(vf[i], pf[i >> 2], o[i & 3]);
        if (i < 12) weigh(i + 4);
        __builtin_amdgcn_sched_barrier(0);
      }
      lsum += add;
    } else {
      // token by token: the values of keys that it does not see cleared, its
      // rows' sums kept
#pragma unroll
      for (int i = 0; i < 16; ++i) weigh(i);
      lsum += add;
      const int first = wave * 32 / p.hpt, last = min((wave * 32 + 31) / p.hpt, w.ntok - 1);
      for (int tk = first; tk <= last; ++tk) {
        if (!__ballot(row_ok && ti == tk)) continue;
        const int end = attn_last(p, w, w.i0 + tk);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          f32x16 x = o[d];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            i32x4 v = value(4 * u + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + 16 * u + 8 * (e >> 1) + 4 * h + 2 * (e & 1);
              v[e] = j + 1 <= end ? v[e] : j <= end ? v[e] & 0xFFFF : 0;
            }
            x = mfma32x32x16<KK>(v, pf[u], x);
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] = ti == tk ? x[r] : o[d][r];
        }
      }
    }
  };

  // the stages, two per block
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    if (count <= 0) return;
    load_entries(0);
    if constexpr (decltype(careful)::value) {
      for (int s = 0; s < 2 * count; ++s) {
        const Entry x = entry_at(s >> 1);
        __syncthreads();
        copy_plain<NI>(p, kring, vring, wave, rows_of(x, s & 1), kof, vof);
        __syncthreads();
        scores(kring);
        absorb(vring, x, s & 1, careful);
      }
      return;
    }
    Entry x = entry_at(0);
    StageRows r = rows_of(x, 0);
    // one half of an entry: the copies of the next into `kd` and `vd`, then its
    // own work on the rows at kt and vt
    auto half = [&](const uint8_t* __restrict kt, const uint8_t* __restrict vt,
                    uint8_t* __restrict kd, uint8_t* __restrict vd, int in)
        __attribute__((always_inline)) {
      copy_rows<NI>(kd + wave * NI * 1024, r.k, r.kb, kof);
      copy_rows<NI>(vd + wave * NI * 1024, r.v, r.vb, vof);
      scores(kt);
      absorb(vt, x, in, careful);
    };
    copy_rows<NI>(kring + wave * NI * 1024, r.k, r.kb, kof);
    copy_rows<NI>(vring + wave * NI * 1024, r.v, r.vb, vof);
    for (int e = 0; e < count; ++e) {
      // at each half: this wave's copies of the stage have landed; after the
      // barrier everyone's have, and everyone has read the stage before
      r = rows_of(x, 1);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      half(kring, vring, kring + SB, vring + SB, 0);
      Entry xn = x;
      if (e + 1 < count) {
        xn = entry_at(e + 1);
        r = rows_of(xn, 0);
      } else {
        r.kb = r.vb = 0;       // (nothing is read: the last copies bring zeros)
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      half(kring + SB, vring + SB, kring, vring, 1);
      x = xn;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };

  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = f32x16{};
    m = -__builtin_inff();
    lsum = 0.f;
    walk(careful);
  };

#pragma unroll
  for (int s = 0; s < 8; ++s) landed(qv[s]);
  pass(std::false_type{});
  if (w.ntok > 1) {
    // (x - x is 0 for a finite x only; the products add no rounding of their own)
    float odd = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) odd += o[d][r] - o[d][r];
    __syncthreads();
    if (tid == 0) *flag = 0;
    __syncthreads();
    if (row_ok && odd != 0.f) *flag = 1;
    __syncthreads();
    if (*flag) pass(std::true_type{});
  }

  lsum = sum_xor32(lsum);
  if (!row_ok) return;
  const int64_t out_row = ((int64_t)(w.t0 + ti) * p.Hq + hk * p.g + hg);
  // register r of o[d] is head element 32 d + 8 (r / 4) + 4 h + r % 4
  if (split == 0) mark_parts(p, out_row, parts, h, 2);
  if (parts > 1) {
    const int64_t pr = (int64_t)split * p.T * p.Hq + out_row;
    if (h == 0) p.part_ml[pr] = float2{m, lsum};
    if (b0 < b1) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4*>(p.part_o + pr * kD + 32 * d + 8 * q + 4 * h) =
              f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
    }
    return;
  }
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<i32x2*>(p.out + out_row * (2 * kD) + 2 * (32 * d + 8 * q + 4 * h)) =
          i32x2{pack2<KK>(o[d][4 * q] * inv, o[d][4 * q + 1] * inv),
                pack2<KK>(o[d][4 * q + 2] * inv, o[d][4 * q + 3] * inv)};
  if (p.lse && h == 0)
    p.lse[out_row] = lse_of<KK>(m, lsum);
}

// ---------------------------------------------------------------------------
// Selected blocks, many tokens: 16 rows a wave, NW waves a workgroup.
//
// The workgroup walks the union of its tokens' blocks in ascending order: a
// block is copied into the LDS once for all of them, a wave none of whose
// tokens selected it skips its products, and a row of another token gets
// weight 0.  With one workgroup per token the copying bounds it (64 KB per
// token, KV head and selected block out of the L2); neighbouring tokens share
// most of their blocks, and even unrelated lists share them once the tile's
// tokens name more blocks than there are.  Tiles of 16 rows, because a wave
// takes the union of its own tokens' lists, which for few tokens is little
// longer than one list, and because four waves fit a SIMD, which hides what
// the barriers of unequally busy waves cost.
//
// 4096 tokens of 8 heads a group over 16 blocks each of 32768 keys, lists that
// overlap in part (23 blocks for two tokens together, 51 for sixteen): 328 to 354
// us by card, 0.38 to 0.41 PFLOP/s of the selected products; where that took 328,
// 374 us with 32 rows a wave and half as many waves, 1058 us with a workgroup per
// token.  With one list for each tile's tokens it takes 183 us: the rest is the
// wave's own union, and waiting at the stages' barriers for waves that have more
// of the blocks.  Where K and V come from hardly matters (325 us with every block
// on one of 16 pages), and no unit
// is full: MFMA 23%, vector 34%, LDS 24% of the cycles.
// ---------------------------------------------------------------------------

template <int KK, int NW>
__global__ __launch_bounds__(64 * NW, 4) void attn_union_kernel(AttnParams p) {
  constexpr int SB = kTileKeys * 256;          // bytes of a stage's K (or V) rows
  constexpr int NI = SB / 1024 / NW;           // copies of each per wave and stage
  constexpr int kSelBits = 8192 * NW;          // (token, block) marks of a workgroup
  constexpr int kSelSpan = 256 * NW;           // blocks marked at a time, at most
  // One LDS object, cut up by hand: with several, the compiler attaches alias
  // scopes to the copies into the ring and then waits for them before every
  // read of it.
  constexpr int kMarksAt = 4 * SB, kNamedAt = kMarksAt + kSelBits / 8;
  constexpr int kFlagAt = kNamedAt + 2 * kSelSpan;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFlagAt + 16];
  uint8_t* const kring = lds;                                       // [2][64 K rows]
  uint8_t* const vring = lds + 2 * SB;                              // [2][64 V rows]
  // [token][block of the span], and the span's blocks in ascending order
  uint32_t* const marks = reinterpret_cast<uint32_t*>(lds + kMarksAt);
  uint16_t* const named = reinterpret_cast<uint16_t*>(lds + kNamedAt);
  int* const flag = reinterpret_cast<int*>(lds + kFlagAt);
  // an XCD takes runs of 8 consecutive tiles of one KV head, which have most
  // of their blocks in common
  const int per = gridDim.x / p.nsplit;      // (a multiple of 64)
  const int split = blockIdx.x / per;
  const int id = blockIdx.x - split * per;
  const int run = (id >> 6) * 8 + (id & 7);
  const int tile = (run / (p.Hkv * p.hchunks)) * 8 + ((id >> 3) & 7);
  const int unit = run % (p.Hkv * p.hchunks);
  const int hc = unit % p.hchunks;
  const int hk = unit / p.hchunks;
  if (tile >= p.ntiles) return;
  const AttnTile w = attn_tile(p, tile);
  if (!w.valid) return;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane_id();
  const int n = l & 15, G = l >> 4;
  const int row = wave * 16 + n;
  const int ti = row / p.hpt;
  const int hg = hc * p.hpt + (row - ti * p.hpt);
  const bool row_ok = row < p.hpt * p.tpt && ti < w.ntok && hg < p.g;
  const int lim = row_ok ? attn_last(p, w, w.i0 + ti) : -1;
  const int lim_lo = attn_last(p, w, w.i0);
  const int lim_hi = attn_last(p, w, w.i0 + w.ntok - 1);
  const int total = lim_hi >= 0 ? lim_hi / kP + 1 : 0;
  const int parts = max(1, min(p.nsplit, (total + p.min_blocks - 1) / p.min_blocks));
  if (split >= parts) return;
  const int b0 = (int)((int64_t)total * split / parts);
  const int b1 = (int)((int64_t)total * (split + 1) / parts);

  i32x4 qv[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) qv[s] = i32x4{0, 0, 0, 0};
  if (row_ok) {
    const uint8_t* qr = p.q + (int64_t)(w.t0 + ti) * p.q_row_stride + (hk * p.g + hg) * (2 * kD);
#pragma unroll
    for (int s = 0; s < 4; ++s) qv[s] = ld16(qr + 64 * s + 16 * G);
  }

  // the blocks come as a list of `count` entries, the marked ones of a span
  int base = b0, count = b1 - b0;
  const int span = min(kSelSpan, kSelBits / p.tpt & ~31);
  BlockList list;
  auto load_entries = [&](int from) __attribute__((always_inline)) {
    list.load(p, w, hk, from, count, [&](int i) { return base + named[i]; });
  };
  auto entry_at = [&](int e) __attribute__((always_inline)) -> Entry {
    if (e - list.base >= 64) load_entries(e);
    return list.at(e);
  };

  const int cr = l >> 4, cc = l & 15;
  uint32_t kof[NI], vof[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = (wave * NI + i) * 4 + cr;
    kof[i] = (uint32_t)(r * p.k_row_stride + 16 * (cc ^ (r & 15)));
    vof[i] = (uint32_t)(r * p.v_row_stride + 16 * (cc ^ ((r & 7) << 1)));
  }
  auto rows_of = [&](const Entry& x, int in) __attribute__((always_inline)) -> StageRows {
    return stage_rows(p, lim_hi, x, in);
  };

  f32x4 o[8];
  float m, lsum;

  // A stage in two parts: its scores from the K rows at kt, and what follows
  // from them with the V rows at vt.  `mine`: this lane's row's token selected
  // the block.  (The copies that may be in flight go to other parts of the
  // rings, and the parameters say so, as in attn_rows_kernel.)
  f32x4 st[4];
  auto scores = [&](const uint8_t* __restrict kt) __attribute__((always_inline)) {
    // S^T, four tiles of 16 keys: register r of tile t is key
    // j0 + 16 t + 4 G + r of row n (fragments read ahead and pinned, as there)
    constexpr int KLEAD = 3;
    i32x4 kf[16];
    // (k step k's chunk is 4 k + G with the row's swizzle: 64 k flipped into one
    // offset, made afresh for each stage -- as loop invariants the operands'
    // addresses alone would take the registers that make four waves fit)
    uint32_t kat0 = n * 256 + ((G ^ n) << 4);
    asm volatile("" : "+v"(kat0));
    auto key_frag = [&](int i) __attribute__((always_inline)) -> i32x4 {
      return *reinterpret_cast<const i32x4*>(kt + 4096 * (i >> 2) + (kat0 ^ (64 * (i & 3))));
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KLEAD; ++i) kf[i] = key_frag(i);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i + KLEAD < 16) kf[i + KLEAD] = key_frag(i + KLEAD);
      st[i >> 2] = mfma16x16x32<KK>(kf[i], qv[i & 3], st[i >> 2]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto absorb = [&](const uint8_t* __restrict vt, const Entry& cur, int in, bool mine, auto careful)
      __attribute__((always_inline)) {
    const int j0 = cur.beta * kP + in * kTileKeys;
    if (!cur.there || j0 + kTileKeys - 1 > lim_lo) {
      const int rel = cur.there ? lim - j0 - 4 * G : -1;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t][r] = 16 * t + r <= rel ? st[t][r] : -__builtin_inff();
    }
    float mx = st[0][0];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, st[t][r]);
    mx = max_xor32(max_xor16(mx)) * p.c;
    mx = mine ? mx : -__builtin_inff();
    if (__ballot(mx > m + kReach<KK>)) {
      const float mn = moved<KK>(m, mx);
      const float alpha = exp2_hw(m - (mn == -__builtin_inff() ? 0.f : mn));
      m = mn;
      lsum *= alpha;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] *= alpha;
    }
    const float ms = m == -__builtin_inff() ? 0.f : m;
    float add = 0.f;
    i32x4 pf[2];
    // weights 2 i and 2 i + 1 of this lane's 16, rounded and packed
    auto weigh = [&](int i) __attribute__((always_inline)) {
      const float a = exp2_hw(__builtin_fmaf(st[i >> 1][2 * (i & 1)], p.c, -ms));
      const float b = exp2_hw(__builtin_fmaf(st[i >> 1][2 * (i & 1) + 1], p.c, -ms));
      add += a + b;
      const int pk = pack2<KK>(a, b);
      pf[i >> 2][i & 3] = mine ? pk : 0;
    };
    // O^T += V^T P^T, 32 keys a step u, in S^T's order: 32 u + 4 G + {0..3} and
    // 32 u + 16 + 4 G + {0..3}; fragment i is step i / 8, elements 16 (i % 8) on
    const int vr = 4 * G + (n >> 2);
    uint32_t vat0 = vr * 256 + (((n >> 1) & 1) ^ ((vr & 7) << 1)) * 16 + (n & 1) * 8;
    asm volatile("" : "+v"(vat0));
    auto value = [&](int i) __attribute__((always_inline)) -> i32x4 {
      const uint8_t* at = vt + 8192 * (i >> 3) + (vat0 ^ (32 * (i & 7)));
      const i32x2 v0 = lds_read_tr(at), v1 = lds_read_tr(at + 4096);
      return i32x4{v0[0], v0[1], v1[0], v1[1]};
    };
    if constexpr (!decltype(careful)::value) {
      constexpr int VLEAD = 2;
      i32x4 vf[16];
#pragma unroll
      for (int i = 0; i < VLEAD; ++i) vf[i] = value(i);
#pragma unroll
      for (int i = 0; i < 4; ++i) weigh(i);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i + VLEAD < 16) vf[i + VLEAD] = value(i + VLEAD);
        o[i & 7] = mfma16x16x32<KK>(vf[i], pf[i >> 3], o[i & 7]);
        if (i < 4) weigh(i + 4);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) weigh(i);
      const int first = wave * 16 / p.hpt, last = min((wave * 16 + 15) / p.hpt, w.ntok - 1);
      for (int tk = first; tk <= last; ++tk) {
        if (!__ballot(row_ok && ti == tk && mine)) continue;
        const int end = attn_last(p, w, w.i0 + tk);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          f32x4 x = o[d];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            i32x4 v = value(8 * u + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + 32 * u + 16 * (e >> 1) + 4 * G + 2 * (e & 1);
              v[e] = j + 1 <= end ? v[e] : j <= end ? v[e] & 0xFFFF : 0;
            }
            x = mfma16x16x32<KK>(v, pf[u], x);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) o[d][r] = ti == tk ? x[r] : o[d][r];
        }
      }
    }
    lsum += mine ? add : 0.f;
  };

  // the list's stages, two per block
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    if (count <= 0) return;
    load_entries(0);
    auto selected = [&](const Entry& e) -> bool {
      const int at = e.beta - base;
      return row_ok && (marks[ti * (span >> 5) + (at >> 5)] >> (at & 31)) & 1;
    };
    auto some = [&](bool mine) -> bool { return __ballot(mine && row_ok) != 0; };
    if constexpr (decltype(careful)::value) {
      for (int s = 0; s < 2 * count; ++s) {
        const Entry x = entry_at(s >> 1);
        __syncthreads();
        copy_plain<NI>(p, kring, vring, wave, rows_of(x, s & 1), kof, vof);
        __syncthreads();
        const bool mine = selected(x);
        if (some(mine)) {
          scores(kring);
          absorb(vring, x, s & 1, mine, careful);
        }
      }
      return;
    }
    Entry x = entry_at(0);
    StageRows r = rows_of(x, 0);
    // one half of an entry: the copies of the next into `kd` and `vd`, then its
    // own work on the rows at kt and vt
    auto half = [&](const uint8_t* __restrict kt, const uint8_t* __restrict vt,
                    uint8_t* __restrict kd, uint8_t* __restrict vd, int in, bool mine, bool any)
        __attribute__((always_inline)) {
      copy_rows<NI>(kd + wave * NI * 1024, r.k, r.kb, kof);
      copy_rows<NI>(vd + wave * NI * 1024, r.v, r.vb, vof);
      if (any) {
        scores(kt);
        absorb(vt, x, in, mine, careful);
      }
    };
    copy_rows<NI>(kring + wave * NI * 1024, r.k, r.kb, kof);
    copy_rows<NI>(vring + wave * NI * 1024, r.v, r.vb, vof);
    for (int e = 0; e < count; ++e) {
      const bool mine = selected(x);
      const bool any = some(mine);
      // at each half: this wave's copies of the stage have landed; after the
      // barrier everyone's have, and everyone has read the stage before
      r = rows_of(x, 1);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      half(kring, vring, kring + SB, vring + SB, 0, mine, any);
      Entry xn = x;
      if (e + 1 < count) {
        xn = entry_at(e + 1);
        r = rows_of(xn, 0);
      } else {
        r.kb = r.vb = 0;       // (nothing is read: the last copies bring zeros)
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      half(kring + SB, vring + SB, kring, vring, 1, mine, any);
      x = xn;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };

  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = -__builtin_inff();
    lsum = 0.f;
    const int words = span >> 5;
    for (base = b0; base < b1; base += span) {
      const int end = min(base + span, b1);
      __syncthreads();
      for (int i = tid; i < w.ntok * words; i += 64 * NW) marks[i] = 0;
      __syncthreads();
      for (int i = tid; i < w.ntok * p.nsel; i += 64 * NW) {
        const int tk = i / p.nsel;
        const int e = p.blocks[((int64_t)(w.t0 + tk) * p.Hkv + hk) * p.nsel + (i - tk * p.nsel)];
        if (e >= base && e < end && (int64_t)e * kP <= attn_last(p, w, w.i0 + tk))
          atomicOr(&marks[tk * words + ((e - base) >> 5)], 1u << ((e - base) & 31));
      }
      __syncthreads();
      if (wave == 0) {
        // a word a lane at a time, the marked blocks' places by a prefix sum
        int n0 = 0;
        for (int wd = 0; wd < words; wd += 64) {
          uint32_t u = 0;
          if (wd + l < words)
            for (int tk = 0; tk < w.ntok; ++tk) u |= marks[tk * words + wd + l];
          const int incl = wave_incl_scan((int)__popc(u));
          int at = n0 + incl - __popc(u);
          for (; u; u &= u - 1) named[at++] = (uint16_t)(32 * (wd + l) + __ffs(u) - 1);
          n0 += lane_at(incl, 63);
        }
        if (l == 0) *flag = n0;
      }
      __syncthreads();
      count = __builtin_amdgcn_readfirstlane(*flag);
      walk(careful);
    }
  };

#pragma unroll
  for (int s = 0; s < 4; ++s) landed(qv[s]);
  pass(std::false_type{});
  if (w.ntok > 1) {
    // (x - x is 0 for a finite x only; the products add no rounding of their own)
    float odd = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) odd += o[d][r] - o[d][r];
    __syncthreads();
    if (tid == 0) *flag = 0;
    __syncthreads();
    if (row_ok && odd != 0.f) *flag = 1;
    __syncthreads();
    if (*flag) pass(std::true_type{});
  }

  lsum = sum_xor32(sum_xor16(lsum));
  if (!row_ok) return;
  const int64_t out_row = ((int64_t)(w.t0 + ti) * p.Hq + hk * p.g + hg);
  // register r of o[d] is head element 16 d + 4 G + r
  if (split == 0) mark_parts(p, out_row, parts, G, 4);
  if (parts > 1) {
    const int64_t pr = (int64_t)split * p.T * p.Hq + out_row;
    if (G == 0) p.part_ml[pr] = float2{m, lsum};
    if (b0 < b1) {
#pragma unroll
      for (int d = 0; d < 8; ++d)
        *reinterpret_cast<f32x4*>(p.part_o + pr * kD + 16 * d + 4 * G) = o[d];
    }
    return;
  }
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
  for (int d = 0; d < 8; ++d)
    *reinterpret_cast<i32x2*>(p.out + out_row * (2 * kD) + 2 * (16 * d + 4 * G)) =
        i32x2{pack2<KK>(o[d][0] * inv, o[d][1] * inv), pack2<KK>(o[d][2] * inv, o[d][3] * inv)};
  if (p.lse && G == 0)
    p.lse[out_row] = lse_of<KK>(m, lsum);
}

}  // namespace msa
