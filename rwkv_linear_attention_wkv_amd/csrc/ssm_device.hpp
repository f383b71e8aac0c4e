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

// The slot whose length is the `rank`-th longest (ties by index), for a whole wave: the slots that take
// longest are then dispatched first.  Every lane ranks its slots against all others, whose lengths
// are uniform loads; calls of more slots keep their order.
constexpr int kRankedSlots = 256;
__device__ __forceinline__ int slot_by_length(const SeqParams &p, int rank, int lane) {
  if (!p.lengths || p.units > kRankedSlots) return rank;
  int slot = 0;
  for (int first = 0; first < p.units; first += 64) {
    const int mine = first + lane;
    const int len = mine < p.units ? p.lengths[mine] : -1;
    int above = 0;
    for (int j = 0; j < p.units; ++j) {
      const int other = p.lengths[j];
      above += other > len || (other == len && j < mine);
    }
    const uint64_t hit = __ballot(mine < p.units && above == rank);
    if (hit) slot = first + __builtin_ctzll(hit);
  }
  return uniform(slot);
}

// Vectors that need only their element's alignment: the memory unit takes loads and stores of up to 16
// bytes at any address (the mode that the compiler assumes for this target).
template <int BYTES>
struct Words;
template <> struct Words<2> { typedef uint16_t type; };
template <> struct Words<4> { typedef uint32_t type __attribute__((aligned(2))); };
template <> struct Words<8> { typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2))); };
template <> struct Words<16> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };

// V consecutive elements, widened.
template <bool BF16, int V>
__device__ __forceinline__ void loadv(const void *base, long idx, float (&out)[V]) {
  if constexpr (!BF16 && (V == 3 || V > 4)) {
#pragma unroll
    for (int i = 0; i + 4 <= V; i += 4) {
      float part[4];
      loadv<false>(base, idx + i, part);
#pragma unroll
      for (int k = 0; k < 4; ++k) out[i + k] = part[k];
    }
#pragma unroll
    for (int i = V / 4 * 4; i < V; ++i) out[i] = static_cast<const float *>(base)[idx + i];
  } else {
    constexpr int EL = BF16 ? 2 : 4;
    typedef typename Words<V * EL>::type W;
    const W w = *reinterpret_cast<const W *>(static_cast<const char *>(base) + idx * EL);
    if constexpr (BF16 && V == 1) {
      out[0] = bf16_lo(w);
    } else if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint32_t x;
        if constexpr (V == 2) x = w;
        else x = w[i / 2];
        out[i] = i & 1 ? bf16_hi(x) : bf16_lo(x);
      }
    } else if constexpr (V == 1) {
      out[0] = __uint_as_float(w);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = __uint_as_float(w[i]);
    }
  }
}

// V consecutive results, rounded to nearest even when the array is bf16.
template <bool BF16, int V>
__device__ __forceinline__ void storev(void *base, long idx, const float (&v)[V]) {
  if constexpr (!BF16 && (V == 3 || V > 4)) {
#pragma unroll
    for (int i = 0; i + 4 <= V; i += 4) {
      const float part[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
      storev<false>(base, idx + i, part);
    }
#pragma unroll
    for (int i = V / 4 * 4; i < V; ++i) static_cast<float *>(base)[idx + i] = v[i];
  } else {
    constexpr int EL = BF16 ? 2 : 4;
    typedef typename Words<V * EL>::type W;
    W w;
    if constexpr (BF16 && V == 1) {
      w = bf16_bits(v[0]);
    } else if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        if constexpr (V == 2) w = pack_bf16(v[i], v[i + 1]);
        else w[i / 2] = pack_bf16(v[i], v[i + 1]);
      }
    } else if constexpr (V == 1) {
      w = __float_as_uint(v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    }
    *reinterpret_cast<W *>(static_cast<char *>(base) + idx * EL) = w;
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
  return fmaf(e, r, __int_as_float(max(__float_as_int(v), 0)));  // max(v, 0) in one instruction; a NaN comes with e
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
