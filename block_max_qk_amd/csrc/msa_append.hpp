// The cache append kernel (gfx950 only): rows of new tokens rotated by their
// positions, encoded in the destination's type and stored in their pages.
//
// Bound by memory: every row is read once and written once, the angles of a
// token once per wave.  A wave takes one token and a run of steps; a step is
// four head rows of one item, 16 lanes to a row and 8 elements to a lane
// (16-byte loads, whole lines per row).  The step's item is the same for the
// whole wave, so its type, layout and pointers are scalars and nothing
// diverges.  Loads run three steps ahead.
//
// 14000 tokens of 64 query, 8 key and 8 value rows and an e4m3 index branch: 140
// us, 4.5 TB/s of reads and writes together (a copy reaches 4.95); 4096 tokens
// with an MXFP4 index branch 37 us, 2.9 TB/s; a decode step of 64 tokens 5.8 us:
// its three dependent reads and the launch.  20 rows of 8192 tokens alone, by the
// destination's type: 16-bit 20.3 us (4.3 TB/s), e4m3 25.9 (2.6), MXFP4 30.4 (1.9),
// int8 37.2 (1.8).  What the encoded types take longer is arithmetic and fewer
// waves: with the rotation in float32 they take 21.9, 25.5 and 32.6 us, int8 with
// a reciprocal for its quotients too 26.5, but codes next to a border are then
// not the nearest.
//
// With several position axes the angles of a pair stand in the row of its own
// axis's position.  A lane reads its part of every axis's row, 16 bytes at a time,
// and picks by the pairs' axes (two bits each, in scalars): up to four times the
// angles, out of the L2, once per wave.  The axes' positions are read beside the
// search for the token's request, which hides them.  The 14000 tokens take 151 us
// so (154 with the positions read behind the search), 64 tokens 6.9.
#pragma once

#include "msa_device.hpp"

namespace msa {

constexpr int kAppendItems = 8;
constexpr int kAppendWaves = 4;
constexpr int kLayoutRows = 3;        // MSA_LAYOUT_ROWS

struct AppendItem {
  const uint8_t* src;
  uint8_t* dst;
  uint8_t* scale;
  int64_t src_row, src_head;          // bytes between tokens, between heads
  int64_t page, row, head;            // dst bytes (ROWS: row per token)
  int64_t s_page, s_row, s_head;      // scale bytes
  int64_t limit;                      // pages, or packed tokens
  int32_t heads, steps;               // steps = ceil(heads / 4)
  int32_t kind;                       // KeyKind of dst
  int32_t layout, rotate;
};

struct AppendParams {
  AppendItem item[kAppendItems];
  const float* cos;
  const float* sin;
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* axis_pos;            // [axes, T] positions that the angles go by
  uint64_t pair_axis[2];              // the axis of each rotated pair, two bits a pair
  int64_t positions;                  // rows of the angle table
  int64_t T;
  int32_t B, MB;
  int32_t steps;                      // of all items
  int32_t per_wave, groups;           // steps per wave, waves per token
  int32_t half;                       // rotary_dim / 2 (0: no rotation)
  int32_t interleaved, packed;        // packed: some item is TND
  int32_t axes;                       // 0: the angles go by the token's position
};

// The request of token t: the largest b with cu[b] <= t, found 64 bounds at a
// time (one load per factor 64 of the batch); -1 if no request holds t.
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int64_t t) {
  const int l = lane_id();
  int lo = 0, hi = B;                 // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    // (64-bit: lo + 64 step passes 2^31 for the largest batches)
    const int64_t at = (int64_t)lo + (int64_t)(l + 1) * step;
    const bool below = at < hi && (int64_t)cu[at < hi ? at : hi] <= t;
    const int k = __popcll(__ballot(below));
    lo += k * step;
    hi = min(lo + step, hi);
  }
  return (int64_t)cu[lo] <= t && t < (int64_t)cu[lo + 1] ? lo : -1;
}

__device__ __forceinline__ float elem16(uint32_t w, int hi, bool bf) {
  const uint32_t x = hi ? w >> 16 : w & 0xFFFFu;
  if (bf) return __builtin_bit_cast(float, x << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)x);
}

// The float32 that a rounding to fewer bits takes where it would take y: the bits
// that a float32 has no room for leave the last one set, which keeps a value next
// to a border of the narrower type on its own side.  (To the nearest float32
// instead, 1 rotated row element in 2 million lands on the border and goes to the
// even code.  Below float32's normal range the cast rounds, far from any border.)
__device__ __forceinline__ float to_odd(double y) {
  const uint64_t u = __builtin_bit_cast(uint64_t, y);
  const uint32_t lo = (uint32_t)u;
  // (the sum carries into bit 29 if any of the 29 bits below is set)
  const uint32_t kept = (lo | ((lo & 0x1FFFFFFFu) + 0x1FFFFFFFu)) & 0xE0000000u;
  return (float)__builtin_bit_cast(double, (u >> 32 << 32) | kept);
}

// max over the 16 lanes of a row (or 4 of a group), in float64
template <int LANES>
__device__ __forceinline__ double lanes_max(double x) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) x = fmax(x, __shfl_xor(x, d));
  return x;
}
template <int LANES>
__device__ __forceinline__ bool lanes_any(bool x) {
  const int l = lane_id();
  const unsigned long long m = __ballot(x) >> (l & ~(LANES - 1));
  return (m & ((1ull << LANES) - 1)) != 0;
}

// Interleaved pairs of a lane's 8 elements, rotated by their 4 angles in type F.
template <typename F>
__device__ __forceinline__ void rotate_pairs(F* x, const float* c, const float* s) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const F a = x[2 * k], b = x[2 * k + 1];
    x[2 * k] = a * (F)c[k] - b * (F)s[k];
    x[2 * k + 1] = b * (F)c[k] + a * (F)s[k];
  }
}

// AXES: the angles go by position axes (compiled apart, as the test of it and its
// registers cost the plain form 1 us of 140).
template <bool BF, bool AXES>
__global__ __launch_bounds__(64 * kAppendWaves) void append_kernel(AppendParams p) {
  const int64_t wid = (int64_t)blockIdx.x * kAppendWaves +
                      __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = wid / p.groups;
  if (t >= p.T) return;
  int step = (int)(wid - t * p.groups) * p.per_wave;
  const int step_end = min(step + p.per_wave, p.steps);

  // (a token's angle rows by axis, read beside the search for its request)
  [[maybe_unused]] int turn[4];
  if constexpr (AXES) {
#pragma unroll
    for (int k = 0; k < 4; ++k) turn[k] = k < p.axes ? p.axis_pos[k * p.T + t] : 0;
  }
  const int b = __builtin_amdgcn_readfirstlane(request_of(p.cu_q, p.B, t));
  if (b < 0) return;
  const int q0 = p.cu_q[b];
  const int lq = p.cu_q[b + 1] - q0;
  const int64_t pos = (int64_t)p.kv_len[b] - lq + (t - q0);
  if (pos < 0 || (!AXES && p.half > 0 && pos >= p.positions)) return;
  if constexpr (AXES) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < p.axes && (turn[k] < 0 || turn[k] >= p.positions)) return;
  }
  const int l = lane_id();
  const int i = l & 15, rr = l >> 4;

  // where the token lives: its page and slot, or its packed row
  const int64_t blk = pos / kP;
  const int slot = (int)(pos - blk * kP);
  int page = -1;
  if (p.block_table && blk < p.MB) page = p.block_table[(int64_t)b * p.MB + blk];
  int64_t packed = 0;
  if (p.packed) {
    for (int base = 0; base < b; base += 64)
      packed += lane_at(wave_incl_scan(base + l < b ? (int64_t)max(p.kv_len[base + l], 0) : 0), 63);
    packed += pos;
  }

  // this lane's angles: of its 8 elements (halves, whose partners lie p.half
  // elements away in another lane) or of its 4 pairs (interleaved)
  float c[8], s[8];
  if constexpr (AXES) {
    // (a row of angles per axis; a lane reads those that its pairs belong to)
    const int at = 8 * i < 2 * p.half ? (p.interleaved ? 4 * i : (8 * i) % p.half) : 0;
    // two bits a pair from bit 2 at on: at is a multiple of 4, so 8 pairs lie in
    // one word unless at % 32 is 28, where only the 4 pairs of an interleaved lane begin
    const uint32_t mine = (uint32_t)(p.pair_axis[at >> 5] >> (2 * (at & 31)));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x >= p.axes) break;
      const float* cr = p.cos + (int64_t)turn[x] * p.half + at;
      const float* sr = p.sin + (int64_t)turn[x] * p.half + at;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        if (p.interleaved && k > 0) break;
        const f32x4 cv = *reinterpret_cast<const f32x4*>(cr + k);
        const f32x4 sv = *reinterpret_cast<const f32x4*>(sr + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool is = x == 0 || (mine >> (2 * (k + e)) & 3) == (uint32_t)x;
          c[k + e] = is ? cv[e] : c[k + e];
          s[k + e] = is ? sv[e] : s[k + e];
        }
      }
    }
  } else if (p.half > 0) {
    const float* cr = p.cos + pos * p.half;
    const float* sr = p.sin + pos * p.half;
    const int at = 8 * i < 2 * p.half ? (p.interleaved ? 4 * i : (8 * i) % p.half) : 0;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const int a = p.interleaved ? at : at + k;
      const f32x4 cv = *reinterpret_cast<const f32x4*>(cr + a);
      const f32x4 sv = *reinterpret_cast<const f32x4*>(sr + a);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[k + e] = cv[e];
        s[k + e] = sv[e];
      }
    }
  }
  // halves: the partner's lane and this lane's sign of the sine
  const int hc = p.half / 8;                       // lanes of one half
  const bool rot_lane = i < 2 * hc;
  const int partner = (l & 48) | (rot_lane ? (i < hc ? i + hc : i - hc) : i);

  // a step's item and its first step: kept once for the step at work and once
  // for the loads, which run DEPTH steps ahead
  constexpr int DEPTH = 3;
  struct Place { int item, first; };
  auto move_to = [&](Place& at, int st) {
    while (st >= at.first + p.item[at.item].steps) at.first += p.item[at.item++].steps;
  };
  Place at{0, 0}, ahead{0, 0};
  auto load = [&](int st) -> i32x4 {
    const i32x4 none = {0, 0, 0, 0};
    if (st >= step_end) return none;
    move_to(ahead, st);
    const AppendItem& a = p.item[ahead.item];
    const int h = 4 * (st - ahead.first) + rr;
    return h < a.heads ? ld16(a.src + t * a.src_row + (int64_t)h * a.src_head + 16 * i) : none;
  };
  i32x4 next[DEPTH];
#pragma unroll
  for (int k = 0; k < DEPTH; ++k) next[k] = load(step + k);
  for (; step < step_end; ++step) {
    move_to(at, step);
    const int cur = at.item, st = step - at.first;
    i32x4 raw = next[0];
#pragma unroll
    for (int k = 0; k + 1 < DEPTH; ++k) next[k] = next[k + 1];
    next[DEPTH - 1] = load(step + DEPTH);
    const AppendItem& a = p.item[cur];
    const int h = 4 * st + rr;
    int64_t off, soff;
    bool ok = h < a.heads;
    if (a.layout == kLayoutRows) {
      off = t * a.row;
      soff = t * a.s_row;
    } else if (a.layout == 0) {
      ok = ok && packed < a.limit;
      off = packed * a.row;
      soff = packed * a.s_row;
    } else {
      ok = ok && page >= 0 && page < a.limit;
      off = page * a.page + slot * a.row;
      soff = page * a.s_page + slot * a.s_row;
    }
    uint8_t* const dst = a.dst + off + (int64_t)h * a.head;
    uint8_t* const scl = a.scale + soff + (int64_t)h * a.s_head;

    if (a.kind == KF16 || a.kind == KBF16) {
      if (a.rotate) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = elem16((uint32_t)raw[k >> 1], k & 1, BF);
        if (p.interleaved) {
          if (rot_lane) rotate_pairs(x, c, s);
        } else {
          // (every lane takes part in the exchange)
          i32x4 other;
#pragma unroll
          for (int e = 0; e < 4; ++e) other[e] = __shfl(raw[e], partner);
          if (rot_lane) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float y = elem16((uint32_t)other[k >> 1], k & 1, BF);
              x[k] = i < hc ? x[k] * c[k] - y * s[k] : x[k] * c[k] + y * s[k];
            }
          }
        }
        typedef __attribute__((ext_vector_type(8))) float f32x8;
        f32x8 v;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = x[k];
        if constexpr (BF)
          raw = __builtin_bit_cast(i32x4, __builtin_convertvector(v, bf16x8));
        else
          raw = __builtin_bit_cast(i32x4, __builtin_convertvector(v, f16x8));
      }
      if (ok) *reinterpret_cast<i32x4*>(dst + 16 * i) = raw;
      continue;
    }

    // encoded types: in float64 up to the one rounding
    double y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = elem16((uint32_t)raw[k >> 1], k & 1, BF);
    if (a.rotate) {
      if (p.interleaved) {
        if (rot_lane) rotate_pairs(y, c, s);
      } else {
        i32x4 other;
#pragma unroll
        for (int e = 0; e < 4; ++e) other[e] = __shfl(raw[e], partner);
        if (rot_lane) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const double z = elem16((uint32_t)other[k >> 1], k & 1, BF);
            y[k] = i < hc ? y[k] * c[k] - z * s[k] : y[k] * c[k] + z * s[k];
          }
        }
      }
    }
    if (a.kind == KF8E4M3 || a.kind == KF8E5M2) {
      const float top = a.kind == KF8E4M3 ? 448.f : 57344.f;
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = to_odd(y[k]);
        f[k] = v != v ? v : fminf(fmaxf(v, -top), top);
      }
      int w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (a.kind == KF8E4M3) {
          w[e] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e], f[4 * e + 1], 0, false);
          w[e] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e + 2], f[4 * e + 3], w[e], true);
        } else {
          w[e] = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * e], f[4 * e + 1], 0, false);
          w[e] = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * e + 2], f[4 * e + 3], w[e], true);
        }
      }
      if (ok) *reinterpret_cast<int2*>(dst + 8 * i) = int2{w[0], w[1]};
      continue;
    }
    if (a.kind == KI8) {
      double top = 0.0;
      bool odd = false;                // an infinity or NaN
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double m = fabs(y[k]);
        odd = odd || !(m < __builtin_inf());
        top = fmax(top, m);
      }
      odd = lanes_any<16>(odd);
      top = lanes_max<16>(top);
      const float sc = (float)(top / 127.0);
      uint32_t w[2] = {0, 0};
      if (!odd && sc > 0.f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int q = (int)fmin(fmax(rint(y[k] / (double)sc), -127.0), 127.0);
          w[k >> 2] |= (uint32_t)(q & 255) << (8 * (k & 3));
        }
      }
      if (ok) {
        *reinterpret_cast<uint2*>(dst + 8 * i) = uint2{w[0], w[1]};
        if (i == 0) *reinterpret_cast<float*>(scl) = odd ? __builtin_nanf("") : sc;
      }
      continue;
    }
    // MXFP4: groups of 32 elements are 4 lanes.  In integer steps on the
    // float64's bits but for one addition: floor(log2) of the group's largest
    // magnitude is the exponent field of the largest high word, dividing by
    // the power of two lowers the exponent field, and adding 1.5 * 2^52 steps
    // of the E2M1 grid leaves the value's steps, rounded to nearest even, in the
    // low bits.
    uint32_t hi[8], top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      hi[k] = (uint32_t)(__builtin_bit_cast(uint64_t, y[k]) >> 32);
      top = max(top, hi[k] & 0x7FFFFFFFu);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const bool odd = top >= 0x7FF00000u;
    const int e8 = top == 0 ? 0 : min(max((int)(top >> 20) - 1023 - 2 + 127, 0), 254);
    const double inv = __builtin_bit_cast(double, (uint64_t)(127 - e8 + 1023) << 52);
    uint32_t w = 0;
    if (!odd) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // E2M1: steps of 1/2 below 2, 1 below 4, 2 above; codes 0..4, 4..6, 6..7
        const double m = fabs(y[k]) * inv;
        const uint32_t mh = (uint32_t)(__builtin_bit_cast(uint64_t, m) >> 32);
        const int seg = mh < 0x40000000u ? 0 : mh < 0x40100000u ? 1 : 2;   // below 2, below 4
        // 1.5 * 2^52 * (1/2, 1, 2)
        const double grid = __builtin_bit_cast(double, (uint64_t)(0x43280000u + (seg << 20)) << 32);
        const uint32_t r = (uint32_t)__builtin_bit_cast(uint64_t, m + grid);
        uint32_t code = min((r & 15u) + 2 * seg, 7u);
        if (code) code |= (hi[k] >> 28) & 8u;
        w |= code << (4 * k);
      }
    }
    if (ok) {
      *reinterpret_cast<uint32_t*>(dst + 4 * i) = w;
      if ((i & 3) == 0) scl[i >> 2] = odd ? 255 : (uint8_t)e8;
    }
  }
}

}  // namespace msa
