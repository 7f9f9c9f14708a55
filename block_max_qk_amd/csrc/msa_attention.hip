// Host side of msa_attention and msa_block_attention: argument validation (all
// of it before any HIP call), the split of the work, and the launch of one
// gfx950 kernel, or two where the keys are split, on the caller's stream.
// Nothing is allocated or kept between calls.
#include "msa_index_score.h"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "msa_attention.hpp"
#include "msa_attention_forms.hpp"
#include "msa_host.hpp"

namespace {

using msa::AttnParams;

constexpr int64_t kMaxSplit = 64;      // one lane per part in the join

struct Plan {
  int rows;          // rows per tile: 16 (attn_rows_kernel), 128 or 256 (attn_tile_kernel;
                     // 128 with selected blocks: attn_union_kernel)
  int hpt, tpt, hchunks;
  int64_t ntiles;
  int nsplit, min_blocks, target;
  bool balanced;
  int64_t units;     // workgroups (attn_union_kernel: tiles x parts)
};

// The tile and the split, from the sizes alone.
//
// Dense: tiles of 16 rows where the requests' new tokens fill no more on
// average, 128 rows otherwise, and 256 where requests average three quarters
// of that and such tiles, or their parts of 8 blocks, fill the chip's 256 CUs
// (2048 tokens over 32768 keys, 8 heads a group: 911 us with 256 rows, 951 with
// 128, 3130 with 16; 9 requests of 2 to 258 tokens: 81, 74 and 163 us; one
// prompt of 1000 tokens: 35, 27 and 59 us; 64 requests of one token: 193 with
// 16, 240 with 128).  The average is all that the sizes tell: where few chunks
// stand among many decode tokens, it chooses 16 rows for both (63 tokens beside
// a chunk of 65 over 32768 keys: 510 us with 16 rows, 174 with 128; beside one of
// 900, 32 heads of their own: 2190 and 800).
// Selected blocks: one workgroup per token and KV head (16 rows), or tiles of
// 128 rows that walk the union of their tokens' blocks once tokens can share
// them and fill the chip (16 blocks of 16000 keys, 4 KV heads: 60 tokens 21 us
// against 43, 200 tokens 69 against 60, 1600 tokens 411 against 152; 64
// requests of 2 tokens 85 against 89).
//
// Few tiles are split over the keys until there are about `want` parts, of
// min_blocks blocks at least; a split pays a second kernel and the traffic of
// its partial sums.  (64 x 4 with 16 selected blocks: 44 us unsplit, 52 in two
// parts; 512 tokens over 8000 keys, 128 rows: 87 us in 512 parts, 96 in 256,
// 149 unsplit; 256 rows, 1024 tokens over 16000 keys: 264 us in 256 parts, 272
// in 512; 800 tokens over selected blocks: 99 us in 256 parts, 114 in 512; one
// prompt of 1000 tokens: 27 us unsplit, 39 in two parts of 4 blocks.)
//
// Dense tiles of 16 rows, and larger ones of more than one request, are split
// by their own lengths (attn_part), aiming at 192 parts, three quarters of the
// CUs, which leaves the rounding up room in one round of workgroups, and at
// twice as many of 128 rows, of which a CU holds two.
//  - 16 rows: 24 requests of one token, 8 KV heads; all of 1024 keys, of up to
//    4096, or of 1024 and one of 8192: 23, 42 and 32 us; aiming at 128 parts
//    23, 48 and 37, at 256 30, 47 and 30, at 512 29, 50 and 36; every tile in
//    the same number of parts, 1536 in all, 29, 53 and 58.  64 requests of up
//    to 8192 keys: 194 us, 196 in 1536 even parts.
//  - 128 rows: 100, 300, 40 and 20 tokens over 32768, 400, 900 and 20 keys: 87
//    us, 94 aiming at 192, 155 in even parts; 9 requests of 2 to 258 tokens: 66
//    us, 74 in even parts.
//  - 256 rows: 8 requests of 200 tokens over 2048 keys: 69 us, 94 aiming at
//    384, 90 in even parts.
// Not split are caches of fewer than 8 blocks (16 for the larger tiles; 4 blocks
// 8.2 us, 9.1 in two parts), what would write partial sums of more than 2^18 rows
// (136 MB), and 1024 items (tile, KV head, chunk) and more: there every workgroup
// would go over the whole batch before it knows a part's length, and an even
// batch pays for that (requests of 512 keys, 64 heads on 8: 256 of them 103 us,
// 111 in parts; 1024 of them 454 and 544; 4096 of 16 heads on 2 664 and 1109),
// while one request far longer than the rest then holds the launch up (one of
// 131072 keys beside 127, 255 or 1023 of 512: 1380, 1430 and 1790 us, in parts
// 167, 246 and 890).
Plan plan_for(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t MB, int64_t nsel,
              int most_rows = 256, int64_t most_split = kMaxSplit, int least_blocks = 8) {
  Plan p{};
  const int64_t g = Hq / Hkv;
  const bool few = nsel > 0 ? T < 8 * B || T * Hkv < 640 : T * std::min<int64_t>(g, 16) <= 16 * B;
  p.rows = few ? msa::kAttnRows : 128;
  if (!few && nsel == 0) {
    const int64_t rows = T * std::min<int64_t>(g, 256);
    const int64_t big = (rows + 255) / 256 * Hkv;
    if (rows >= 192 * B && big >= 128 && big * std::max<int64_t>(MB / 8, 1) >= 256)
      p.rows = most_rows;
  }
  p.hpt = (int)std::min<int64_t>(g, p.rows);
  p.tpt = few && nsel > 0 ? 1 : p.rows / p.hpt;
  p.hchunks = (int)((g + p.hpt - 1) / p.hpt);
  p.ntiles = std::min<int64_t>(T, (T + B * (p.tpt - 1)) / p.tpt);
  const int64_t items = std::max<int64_t>(p.ntiles * Hkv * p.hchunks, 1);
  const int64_t blocks = std::max<int64_t>(few && nsel > 0 ? std::min(nsel, MB) : MB, 1);
  p.min_blocks = few ? 2 : p.rows == 256 ? 8 : least_blocks;
  const int64_t want = nsel > 0 ? (few ? 128 : 256) : few ? 1536 : p.rows == 128 ? 512 : 256;
  int64_t n = items >= want ? 1 : (want + items - 1) / items;
  p.target = 1;
  if (nsel == 0 && (few || B > 1)) {
    const int64_t heads = Hkv * p.hchunks;
    p.target = (int)std::max<int64_t>((p.rows == 128 ? 384 : 192) / heads, 1);
    n = items >= 1024 || MB < (few ? 8 : 2 * p.min_blocks) ? 1
        : std::min<int64_t>(p.target, std::max<int64_t>((1 << 18) / (T * Hq), 1));
    p.balanced = true;
  }
  n = std::min(n, (blocks + p.min_blocks - 1) / p.min_blocks);
  p.nsplit = (int)std::max<int64_t>(1, std::min(n, most_split));
  p.units = p.ntiles * Hkv * p.hchunks * p.nsplit;
  if (p.balanced && p.nsplit > 1) p.units = (p.target + 1 + p.ntiles) * Hkv * p.hchunks;
  return p;
}

// Bytes of one part's sums.
int64_t part_bytes(int64_t T, int64_t Hq) {
  return T * Hq * (int64_t)(msa::kD * sizeof(float) + sizeof(float2));
}

int64_t workspace_for(const Plan& p, int64_t T, int64_t Hq) {
  return p.nsplit > 1 ? p.nsplit * part_bytes(T, Hq) : 0;
}

// The plan of a call in another form, in at most `room` parts.  128 rows take the
// place of 256 below 128 blocks, and where a causal range narrows the keys, as
// documents do (32 heads on 4, us with 128 and 256 rows: 2048 tokens over 4096 keys
// biased 127 and 138, over 16384 553 and 540, over 32768 capped 1363 and 1294; 16
// requests of 300 over 2000 keys capped 222 and 256; one prompt of 4096 biased 170
// and 159; 4 requests of 1000 in documents of 1024 tokens 72 and 86).  Tiles of 128
// rows are split down to 4 blocks a part, as a stage takes longer and a range
// leaves fewer of them: us with parts of 8, 4 and 2 blocks or more, 50 tokens over
// 2992 keys capped 44, 30 and 26; 2 requests of 40 over 13600 46, 35 and 39; 5
// prompts of 1750 tokens in all with images 55, 44 and 42; one of 1233 tokens with
// images 46, 48 and 53; 5 requests of 976 over 1089 in documents 55, 58 and 58.  (All
// as the rules were chosen; capped ones take 2 to 4% less now, biased ones 0 to 2%
// more.)  Neither rule is the better one for every size: the prompt of 4096 biased has
// as many blocks as the chunk over 4096 keys and is 7% slower with 128 rows, and the
// documents are 5% slower in parts of 4.
Plan plan_form(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t MB, bool narrow,
               int64_t room) {
  Plan p = plan_for(T, B, Hq, Hkv, MB, 0, 256, room, 4);
  if (p.rows == 256 && (MB < 128 || narrow)) p = plan_for(T, B, Hq, Hkv, MB, 0, 128, room, 4);
  return p;
}

// Sizes that a plan is asked for without a call.
bool sizes_ok(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv, int64_t max_blocks,
              int32_t num_blocks) {
  return T >= 1 && T <= INT32_MAX && batch >= 1 && batch <= (1 << 30) && Hq >= 1 &&
         Hq <= (1 << 16) && Hkv >= 1 && Hq % Hkv == 0 && max_blocks >= 0 &&
         max_blocks <= (1 << 24) && num_blocks >= 0 && num_blocks <= 64;
}

template <int KK>
hipError_t launch(const AttnParams& p, const Plan& plan, int form, int64_t grid, hipStream_t s) {
  hipError_t e;
  const dim3 gr((unsigned)grid);
  if (form != 0) {
    e = msa::launch_form<KK>(p, plan.rows, form, gr, s);
  } else if (plan.rows == msa::kAttnRows) {
    e = msa::launch_kernel(p.blocks ? msa::attn_rows_kernel<KK, true>
                                    : msa::attn_rows_kernel<KK, false>,
                           gr, dim3(256), s, p);
  } else if (p.blocks) {
    e = msa::launch_kernel(msa::attn_union_kernel<KK, 8>, gr, dim3(512), s, p);
  } else if (plan.rows == 256) {
    e = msa::launch_kernel(msa::attn_tile_kernel<KK, 8>, gr, dim3(512), s, p);
  } else {
    e = msa::launch_kernel(msa::attn_tile_kernel<KK, 4>, gr, dim3(256), s, p);
  }
  if (e == hipSuccess && p.nsplit > 1)
    e = msa::launch_kernel(msa::attn_join_kernel<KK>,
                           dim3((unsigned)((p.T * p.Hq + 4 * p.join_rows - 1) / (4 * p.join_rows))),
                           dim3(256), s, p);
  return e;
}

// Forms of the scores, as the entry points take them.
struct Forms {
  float softcap;            // 0: none
  const float* slopes;      // or NULL
  const int32_t* visible;   // or NULL
};

// The forms in the kernels' terms; a sum of ScoreForms.
int set_forms(const Forms& f, float scale, AttnParams& p) {
  int form = 0;
  p.slopes = f.slopes;
  p.visible = reinterpret_cast<const int2*>(f.visible);
  p.per_scale = 1.f / scale;
  if (f.slopes) form |= msa::kBias;
  if (f.softcap > 0.f) {
    form |= msa::kCap;
    // tanh(x) = x (1 + c1 x^2 + .. + c4 x^8) for |x| <= 5/8, off by 1.22e-7 of itself
    // at most (two of float32's half steps)
    constexpr double kTanh[5] = {1.0, -0.333323412, 0.133081751, -0.0519479045, 0.0151953732};
    constexpr double kNear = 0.625;
    double a = (double)scale / f.softcap, unit = (double)scale * msa::kLog2e;
    // A cap so large or small that a coefficient of the products' square has no
    // float32 of full precision (at a scale of 1/sqrt(128), above 2170): the products
    // are scaled by a power of two in front (2^-110 at the least, so that those above
    // 2^-16 keep their digits), which changes no other rounding.
    const double a4 = a * a * (a * a), c4 = kTanh[4] * unit * a4 * a4;
    p.cap_unit = 1.f;
    if (!(c4 >= FLT_MIN && c4 <= FLT_MAX)) {
      const int e = std::clamp(std::ilogb(a) + 1, -110, 127);
      p.cap_unit = std::ldexp(1.f, e);
      a = std::ldexp(a, -e);
      unit = std::ldexp(unit, -e);
    }
    p.cap_top = f.softcap * msa::kLog2e;
    p.cap_twice = (float)(2.0 * msa::kLog2e * a);
    p.cap_near = (float)std::min(kNear / a, (double)FLT_MAX);
    for (int i = 0; i < 5; ++i, unit *= a * a) p.cap_poly[i] = (float)(kTanh[i] * unit);
    // Such caps go to the kernels of a cap and a bias (no slopes: 0), which spares the
    // others a look at cap_unit a stage (the chunk 1279 -> 1265 us).  So do caps past
    // 2^20: the others' weights' exponents are scores to all their digits less the
    // largest one rounded, with scores of 10^9 more than an exponent holds.
    if (p.cap_unit != 1.f || p.cap_top > 0x1p20f) form |= msa::kBias;
  }
  if (f.visible || form) form |= msa::kRange;
  return form;
}

msa_status_t run(const msa_tensor_t* query, const msa_tensor_t* key, const msa_tensor_t* value,
                 const int32_t* blocks, int64_t num_blocks, bool selected,
                 const int32_t* block_table, int64_t max_blocks, const int32_t* cu_seqlens_q,
                 const int32_t* kv_len, int32_t batch, int32_t block_size, int32_t layout,
                 int32_t sparse_mode, float softmax_scale, const Forms& forms, void* out,
                 float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!query || !key || !value || !cu_seqlens_q) return MSA_ERR_NULL;
  if (batch > 0 && !kv_len) return MSA_ERR_NULL;
  if (query->ndim == 3 && query->shape[0] > 0 && !out) return MSA_ERR_NULL;
  if (layout != MSA_LAYOUT_TND && layout != MSA_LAYOUT_BBND && layout != MSA_LAYOUT_BNBD)
    return MSA_ERR_LAYOUT;
  const bool paged = layout != MSA_LAYOUT_TND;
  if (query->dtype != MSA_DTYPE_F16 && query->dtype != MSA_DTYPE_BF16) return MSA_ERR_DTYPE;
  if (key->dtype != query->dtype || value->dtype != query->dtype) return MSA_ERR_DTYPE;

  // query [T, Hq, D]: rows of a wider projection's rows
  if (query->ndim != 3) return MSA_ERR_SHAPE;
  const int64_t T = query->shape[0], Hq = query->shape[1], D = query->shape[2];
  if (T < 0 || Hq < 1 || D != msa::kD || block_size != msa::kP) return MSA_ERR_SHAPE;
  const int64_t q_row = T > 1 ? query->stride[0] : Hq * D;
  if (!msa::compact_axis(D, query->stride[2], 1) || !msa::compact_axis(Hq, query->stride[1], D) ||
      q_row < Hq * D || (q_row * 2) % 16)
    return MSA_ERR_STRIDE;

  msa::CacheView kv, vv;
  msa_status_t st = msa::cache_view(*key, layout, msa::kD, msa::kP, true, kv);
  if (st != MSA_OK) return st;
  st = msa::cache_view(*value, layout, msa::kD, msa::kP, true, vv);
  if (st != MSA_OK) return st;
  if (kv.pages != vv.pages || kv.heads != vv.heads || Hq % kv.heads) return MSA_ERR_SHAPE;
  const int64_t Hkv = kv.heads;

  if (max_blocks < 0 || batch < 0) return MSA_ERR_SHAPE;
  if (paged) {
    if (!block_table && batch > 0) return MSA_ERR_NULL;
    if (max_blocks < 1) return MSA_ERR_SHAPE;
  } else if (block_table) {
    return MSA_ERR_SHAPE;   // packed keys take no block table
  }
  if (batch == 0 && T > 0) return MSA_ERR_SHAPE;
  if (sparse_mode != 0 && sparse_mode != 3) return MSA_ERR_ATTR;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale * msa::kLog2e)) return MSA_ERR_ATTR;
  if (!(forms.softcap >= 0.f) || !std::isfinite(forms.softcap * msa::kLog2e)) return MSA_ERR_ATTR;
  if (forms.softcap > 0.f && !std::isfinite(2.f * msa::kLog2e * softmax_scale / forms.softcap))
    return MSA_ERR_ATTR;
  if (forms.slopes && !std::isfinite(1.f / softmax_scale)) return MSA_ERR_ATTR;
  if ((reinterpret_cast<uintptr_t>(forms.slopes) & 3u) ||
      (reinterpret_cast<uintptr_t>(forms.visible) & 7u))
    return MSA_ERR_STRIDE;
  if (selected) {
    if (num_blocks < 1 || num_blocks > 64) return MSA_ERR_ATTR;
    if (T > 0 && !blocks) return MSA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(blocks) & 3u) return MSA_ERR_STRIDE;
  }
  // sizes the kernels index with 32-bit integers
  if (max_blocks > (1 << 24) || Hq > (1 << 16) || batch > (1 << 30) || T > INT32_MAX)
    return MSA_ERR_SHAPE;
  if (!msa::aligned16(query->data) || !msa::aligned16(out) || !msa::aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MSA_ERR_STRIDE;
  if (T == 0) return MSA_OK;
  if (!query->data || (kv.pages > 0 && (!key->data || !value->data))) return MSA_ERR_NULL;

  Plan plan = plan_for(T, batch, Hq, Hkv, max_blocks, selected ? num_blocks : 0);
  const int64_t need = workspace_for(plan, T, Hq);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MSA_ERR_WORKSPACE;
  if (forms.softcap > 0.f || forms.slopes || forms.visible) {
    const int64_t room = workspace ? workspace_bytes / part_bytes(T, Hq) : 1;
    plan = plan_form(T, batch, Hq, Hkv, max_blocks, forms.visible && sparse_mode == 3,
                     std::clamp<int64_t>(room, 1, kMaxSplit));
  }
  int64_t grid = plan.units;
  if (selected && plan.rows != msa::kAttnRows) {   // runs of 8 tiles, 8 runs at a time
    const int64_t runs = (plan.ntiles + 7) / 8 * Hkv * plan.hchunks;
    grid = (runs + 7) / 8 * 64 * plan.nsplit;
  }
  // (a launch holds less than 2^32 threads)
  const int64_t threads = plan.rows == 256 || (selected && plan.rows == 128) ? 512 : 256;
  if (grid * threads > UINT32_MAX ||
      (plan.nsplit > 1 && T * Hq * 64 > (int64_t)UINT32_MAX))
    return MSA_ERR_SHAPE;

  AttnParams p{};
  p.q = static_cast<const uint8_t*>(query->data);
  p.k = static_cast<const uint8_t*>(key->data);
  p.v = static_cast<const uint8_t*>(value->data);
  p.block_table = paged ? block_table : nullptr;
  p.cu_q = cu_seqlens_q;
  p.kv_len = kv_len;
  p.blocks = selected ? blocks : nullptr;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<float*>(workspace) +
                                        (plan.nsplit > 1 ? plan.nsplit * T * Hq * msa::kD : 0));
  p.q_row_stride = q_row * 2;
  p.k_page_stride = kv.page;
  p.v_page_stride = vv.page;
  p.k_row_stride = (int32_t)kv.row;
  p.v_row_stride = (int32_t)vv.row;
  p.k_head_stride = (int32_t)kv.head;
  p.v_head_stride = (int32_t)vv.head;
  p.keys = paged ? 0 : kv.pages;
  p.T = T;
  p.B = batch;
  p.Hq = (int32_t)Hq;
  p.Hkv = (int32_t)Hkv;
  p.g = (int32_t)(Hq / Hkv);
  p.MB = (int32_t)std::max<int64_t>(max_blocks, 1);
  p.NP = paged ? (int32_t)kv.pages : 0;
  p.nsel = selected ? (int32_t)num_blocks : 0;
  p.paged = paged ? 1 : 0;
  p.causal = sparse_mode == 3 ? 1 : 0;
  p.c = softmax_scale * msa::kLog2e;
  p.hpt = plan.hpt;
  p.tpt = plan.tpt;
  p.hchunks = plan.hchunks;
  p.ntiles = (int32_t)plan.ntiles;
  p.nsplit = plan.nsplit;
  p.min_blocks = plan.min_blocks;
  p.balanced = plan.balanced ? 1 : 0;
  p.join_rows = (int32_t)std::clamp<int64_t>(T * Hq / 8192, 1, 64);   // the chip holds 8192 waves
  p.per_target = 1.f / plan.target;
  const int form = set_forms(forms, softmax_scale, p);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = query->dtype == MSA_DTYPE_BF16 ? launch<msa::KBF16>(p, plan, form, grid, s)
                                                      : launch<msa::KF16>(p, plan, form, grid, s);
  return e == hipSuccess ? MSA_OK : MSA_ERR_HIP;
}

}  // namespace

extern "C" {

msa_status_t msa_attention(const msa_tensor_t* query, const msa_tensor_t* key,
                           const msa_tensor_t* value, const int32_t* block_table,
                           int64_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* kv_len,
                           int32_t batch, int32_t block_size, int32_t layout, int32_t sparse_mode,
                           float softmax_scale, void* out, float* lse, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  return run(query, key, value, nullptr, 0, false, block_table, max_blocks, cu_seqlens_q, kv_len,
             batch, block_size, layout, sparse_mode, softmax_scale, Forms{}, out, lse, workspace,
             workspace_bytes, stream);
}

msa_status_t msa_attention_ex(const msa_tensor_t* query, const msa_tensor_t* key,
                              const msa_tensor_t* value, const int32_t* block_table,
                              int64_t max_blocks, const int32_t* cu_seqlens_q,
                              const int32_t* kv_len, int32_t batch, int32_t block_size,
                              int32_t layout, int32_t sparse_mode, float softmax_scale,
                              float softcap, const float* slopes, const int32_t* visible,
                              void* out, float* lse, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  return run(query, key, value, nullptr, 0, false, block_table, max_blocks, cu_seqlens_q, kv_len,
             batch, block_size, layout, sparse_mode, softmax_scale,
             Forms{softcap, slopes, visible}, out, lse, workspace, workspace_bytes, stream);
}

msa_status_t msa_block_attention(const msa_tensor_t* query, const msa_tensor_t* key,
                                 const msa_tensor_t* value, const int32_t* blocks,
                                 int32_t num_blocks, const int32_t* block_table,
                                 int64_t max_blocks, const int32_t* cu_seqlens_q,
                                 const int32_t* kv_len, int32_t batch, int32_t block_size,
                                 int32_t layout, int32_t sparse_mode, float softmax_scale,
                                 void* out, float* lse, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  return run(query, key, value, blocks, num_blocks, true, block_table, max_blocks, cu_seqlens_q,
             kv_len, batch, block_size, layout, sparse_mode, softmax_scale, Forms{}, out, lse,
             workspace, workspace_bytes, stream);
}

int64_t msa_attention_workspace(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                int64_t max_blocks, int32_t num_blocks) {
  if (!sizes_ok(T, batch, Hq, Hkv, max_blocks, num_blocks)) return 0;
  return workspace_for(plan_for(T, batch, Hq, Hkv, max_blocks, num_blocks), T, Hq);
}

int64_t msa_attention_ex_workspace(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                   int64_t max_blocks) {
  if (!sizes_ok(T, batch, Hq, Hkv, max_blocks, 0)) return 0;
  int64_t most = msa_attention_workspace(T, batch, Hq, Hkv, max_blocks, 0);
  for (const bool narrow : {false, true})
    most = std::max(most, workspace_for(plan_form(T, batch, Hq, Hkv, max_blocks, narrow, kMaxSplit),
                                        T, Hq));
  return most;
}

int32_t msa_attention_tile_rows(int64_t T, int32_t batch, int32_t Hq, int32_t Hkv,
                                int64_t max_blocks, int32_t num_blocks) {
  if (!sizes_ok(T, batch, Hq, Hkv, max_blocks, num_blocks)) return 0;
  return plan_for(T, batch, Hq, Hkv, max_blocks, num_blocks).rows;
}

}  // extern "C"
