// Device helpers shared by the state space kernels (gfx950 only).
#pragma once

#include "common.hpp"
#include "ssm.hpp"
#include "wkv.h"

namespace wkv {

// The value of the lane that DPP control CTRL selects (every lane of the row is active).
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // lane ^1, ^2, ^7, ^15

// The sum of x over the wave, in every lane: four steps within the rows of 16, then the rows' sums.
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kXor1, 0xf, 0xf, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kXor2, 0xf, 0xf, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kHalfMirror, 0xf, 0xf, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kMirror, 0xf, 0xf, true);
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 0) + (uint32_t)__builtin_amdgcn_readlane((int)x, 16) +
         (uint32_t)__builtin_amdgcn_readlane((int)x, 32) + (uint32_t)__builtin_amdgcn_readlane((int)x, 48);
}

// One sequence of a call, the same in every lane of the wave that asked for it.
struct Sequence {
  long off;  // first token row
  int len;
  int row_in, row_out;  // state rows
  bool ok;              // false: rejected, nothing may be written
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long uniform(long x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (long)(((uint64_t)hi << 32) | lo);
}

// The sequence of `unit`, for a whole wave (lane = its lane).  A varlen call reads every length:
// an invalid one anywhere makes all offsets meaningless and rejects every slot; two slots of
// one state row, a row outside the table and tokens past the packed arrays reject the slot.
__device__ __forceinline__ Sequence find_sequence(const SeqParams &p, int unit, int lane) {
  Sequence q;
  int status = 0;
  if (!p.lengths) {
    q.off = (long)unit * p.T;
    q.len = p.T;
    q.row_in = p.state_map ? p.state_map[unit] : (p.n_state == 1 ? 0 : unit);
    q.row_out = unit;
    if (p.state_in && (q.row_in < 0 || q.row_in >= p.n_state)) status = WKV_DEV_BAD_STATE_MAP;
  } else {
    const int len = p.lengths[unit];
    const int row = p.state_map ? p.state_map[unit] : unit;
    uint32_t lo = 0, hi = 0;  // the sum of the lengths before this slot, of their halves of 16 bits: at most 65535 slots
    bool bad = false, dup = false;
    for (int i = lane; i < p.units; i += 64) {
      const int L = p.lengths[i];
      if (i < unit) {
        lo += (uint32_t)L & 0xffffu;
        hi += (uint32_t)L >> 16;
      }
      bad |= L < 0 || L > p.T;
      if (p.state_map && i != unit && p.state_map[i] == row) dup = true;
    }
    const long sum = (long)wave_sum(lo) + ((long)wave_sum(hi) << 16);
    if (__any(bad)) status |= WKV_DEV_BAD_LENGTH;
    if (row < 0 || row >= p.n_state) status |= WKV_DEV_BAD_STATE_MAP;
    if (__any(dup)) status |= WKV_DEV_DUPLICATE_ROW;
    if (!(status & WKV_DEV_BAD_LENGTH) && sum + len > p.total_tokens) status |= WKV_DEV_TOKEN_OVERFLOW;
    q.off = sum;
    q.len = uniform(len);
    q.row_in = q.row_out = uniform(row);
  }
  q.ok = status == 0;
  if (!q.ok && lane == 0 && p.dev_status) atomicOr(p.dev_status, status);
  return q;
}

// V consecutive elements of a token array, widened; the address is aligned to the whole load.
template <bool BF16, int V>
__device__ __forceinline__ void loadv(const void *base, long idx, float (&out)[V]) {
  if constexpr (BF16) {
    const uint16_t *p = static_cast<const uint16_t *>(base) + idx;
    if constexpr (V == 1) {
      out[0] = bf16_lo(*p);
    } else if constexpr (V == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
      out[0] = bf16_lo(w); out[1] = bf16_hi(w);
    } else if constexpr (V == 4) {
      const uint2 w = *reinterpret_cast<const uint2 *>(p);
      out[0] = bf16_lo(w.x); out[1] = bf16_hi(w.x); out[2] = bf16_lo(w.y); out[3] = bf16_hi(w.y);
    } else {
      const uint4 w = *reinterpret_cast<const uint4 *>(p);
      out[0] = bf16_lo(w.x); out[1] = bf16_hi(w.x); out[2] = bf16_lo(w.y); out[3] = bf16_hi(w.y);
      out[4] = bf16_lo(w.z); out[5] = bf16_hi(w.z); out[6] = bf16_lo(w.w); out[7] = bf16_hi(w.w);
    }
  } else {
    const float *p = static_cast<const float *>(base) + idx;
    if constexpr (V == 1) {
      out[0] = *p;
    } else if constexpr (V == 2) {
      const float2 w = *reinterpret_cast<const float2 *>(p);
      out[0] = w.x; out[1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(p + i);
        out[i] = w.x; out[i + 1] = w.y; out[i + 2] = w.z; out[i + 3] = w.w;
      }
    }
  }
}

// V consecutive results, rounded to nearest even when the array is bf16.
template <bool BF16, int V>
__device__ __forceinline__ void storev(void *base, long idx, const float (&v)[V]) {
  if constexpr (BF16) {
    uint16_t *p = static_cast<uint16_t *>(base) + idx;
    if constexpr (V == 1) *p = bf16_bits(v[0]);
    else if constexpr (V == 2) *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[1]);
    else if constexpr (V == 4)
      *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else
      *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                 pack_bf16(v[6], v[7]));
  } else {
    float *p = static_cast<float *>(base) + idx;
    if constexpr (V == 1) *p = v[0];
    else if constexpr (V == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    else {
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
}

__device__ __forceinline__ void store1(void *base, long idx, bool bf16, float v) {
  if (bf16) static_cast<uint16_t *>(base)[idx] = bf16_bits(v);
  else static_cast<float *>(base)[idx] = v;
}

__device__ __forceinline__ float load1_rt(const void *base, long idx, bool bf16) {
  return bf16 ? load1<true>(base, idx) : load1<false>(base, idx);
}

__device__ __forceinline__ float sigmoid_f(float v) { return fast_rcp(1.f + fast_exp(-v)); }

// ln(1 + e^v) = max(v, 0) + ln(1 + e) with e = e^-|v| in (0, 1].  ln(1 + e) / e is a polynomial of degree
// 8 (a least-squares fit on [0, 1], reweighted until its relative error was level at 2^-25): no
// cancellation, so a small step keeps its relative accuracy (under 2^-22 with its own roundings).
__device__ __forceinline__ float softplus_e(float v, float e) {
  float r = 0.005232690833508968f;
  r = fmaf(r, e, -0.029505230486392975f);
  r = fmaf(r, e, 0.07822594791650772f);
  r = fmaf(r, e, -0.13663245737552643f);
  r = fmaf(r, e, 0.19106008112430573f);
  r = fmaf(r, e, -0.2484298199415207f);
  r = fmaf(r, e, 0.3331909775733948f);
  r = fmaf(r, e, -0.4999949336051941f);
  r = fmaf(r, e, 0.9999999403953552f);
  return fmaf(e, r, fmaxf(v, 0.f));
}

__device__ __forceinline__ float softplus_f(float v) {
  return softplus_e(v, __builtin_amdgcn_exp2f(fabsf(v) * -1.4426950408889634f));
}

// The same with its slope, 1 / (1 + e^-v): 1 or e over 1 + e, as v is positive or not.
__device__ __forceinline__ float softplus_f(float v, float &slope) {
  const float e = __builtin_amdgcn_exp2f(fabsf(v) * -1.4426950408889634f);
  slope = (v >= 0.f ? 1.f : e) * fast_rcp(1.f + e);
  return softplus_e(v, e);
}

// A window of a token array for buffer loads and stores: `rows` rows from `row` on, columns from c
// on.  Accesses past its last row read 0 and write nothing; columns that a lane does not have are
// sent there by adding kOutside to their offset.  Offsets are 32-bit: at most 127 rows, of row strides
// up to kMaxStride.
constexpr uint32_t kOutside = 0x80000000u;
template <int ELEM>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void *base, long stride, long row, int rows, long c, int cols) {
  const char *at = static_cast<const char *>(base) + (row * stride + c) * ELEM;
  const uint32_t n = rows > 0 ? (uint32_t)(((rows - 1) * stride + cols) * ELEM) : 0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, (int)n, 0x00020000);
}

constexpr float kLog2e = 1.4426950408889634f;

// The sum of v over the L adjacent lanes that share a channel, in every one of them.
template <int L>
__device__ __forceinline__ float sum_all(float v) {
  if constexpr (L >= 2) v += dpp<kXor1>(v);
  if constexpr (L >= 4) v += dpp<kXor2>(v);
  if constexpr (L >= 8) v += dpp<kHalfMirror>(v);
  if constexpr (L >= 16) v += dpp<kMirror>(v);
  return v;
}

}  // namespace wkv
