// Parts shared by the tiled scan kernels, forward and backward: rows of token arrays as the staging
// waves load and store them, states and sums as the scan waves hold them.
#pragma once

#include "ssm_device.hpp"

namespace wkv {

// Four state values of one channel: values 4q .. 4q + 3 of the N a row holds (zero beyond N).
__device__ __forceinline__ void load_state4(const float *row, int q, int N, bool whole, float (&h)[4]) {
  if (whole) {
    loadv<false>(row, 4 * q, h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = 4 * q + i < N ? row[4 * q + i] : 0.f;
  }
}

// A value of A, scaled for the base-2 exponential, and finite, so that a step of zero (a token past
// a sequence's end, too) is a decay of one also where A or its scaled value is an infinity.
__device__ __forceinline__ float decay_rate(float A) {
  constexpr float kMost = 3.4028234663852886e38f;
  A *= kLog2e;
  return A < -kMost ? -kMost : A > kMost ? kMost : A;  // NaN stays
}

__device__ __forceinline__ void load_decay4(const float *row, int q, int N, bool whole, float (&A)[4]) {
  load_state4(row, q, N, whole, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = decay_rate(A[i]);
}

__device__ __forceinline__ void store_state4(float *row, int q, int N, bool whole, const float (&h)[4]) {
  if (whole) {
    storev<false>(row, 4 * q, h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < N) row[4 * q + i] = h[i];
  }
}

// How a tile's rows are read and written VW channels at a time.  Whole: the blocks of channels divide
// by VW (addresses need no alignment: see Words).  Overlap: they do not; the last thread of a block's
// row moves back onto its neighbour's channels, which both then hold alike.  Single: a block has fewer
// than VW channels; one by one.  (48 slots of up to 700 tokens, two groups of 775 channels, fp32: 62 us with
// overlaps, 101 one by one.)
enum class Rows { kWhole, kOverlap, kSingle };

template <int CH, int VW>
Rows rows_of(int per_group) {
  if (VW == 1) return Rows::kSingle;
  if (per_group % VW == 0) return Rows::kWhole;
  const int last = (per_group - 1) % CH + 1;  // channels of the last block
  return last >= VW ? Rows::kOverlap : Rows::kSingle;
}

// VW adjacent elements as loaded: widened when they are used, so that no load is waited for early.
template <bool BF16, bool VEC, int VW>
struct RawRow {
  static_assert(!VEC || VW == 2 || VW == 4 || (BF16 && VW == 8), "whole loads are of 4, 8 or 16 bytes");
  uint32_t w[VEC && BF16 ? (VW + 1) / 2 : VW];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, const uint32_t (&col)[VEC ? 1 : VW]) {
    if constexpr (VEC) {
      if constexpr (sizeof w == 16) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(row + col[0]), 0, 0);
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
      } else if constexpr (sizeof w == 8) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)(row + col[0]), 0, 0);
        w[0] = v[0]; w[1] = v[1];
      } else {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)(row + col[0]), 0, 0);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        if constexpr (BF16) w[e] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)(row + col[e]), 0, 0);
        else w[e] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)(row + col[e]), 0, 0);
      }
    }
  }
  // Keeps every use behind this point, so that the wait for the loads stays there.
  __device__ __forceinline__ void arrive() {
#pragma unroll
    for (auto &x : w) asm volatile("" : "+v"(x));
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (VEC && BF16) return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else if constexpr (BF16) return bf16_lo(w[e]);
    else return __uint_as_float(w[e]);
  }
};

// Which of two or three sets of registers a tile uses, as a type.
template <int V>
struct Set { static constexpr int value = V; };

// VW adjacent results through a window.
template <bool BF16, bool VEC, int VW>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, uint32_t row, const uint32_t (&col)[VEC ? 1 : VW], const float (&v)[VW]) {
  static_assert(!VEC || VW == 2 || VW == 4 || VW == 8, "whole stores are of 2, 4 or 8 elements");
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      if constexpr (BF16) __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(v[e]), r, (int)(row + col[e]), 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), r, (int)(row + col[e]), 0, 0);
    }
  } else if constexpr (BF16) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    if constexpr (VW == 8)
      __builtin_amdgcn_raw_buffer_store_b128(u4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}, r,
                                             (int)(row + col[0]), 0, 0);
    else if constexpr (VW == 4) __builtin_amdgcn_raw_buffer_store_b64(u2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, r, (int)(row + col[0]), 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(v[0], v[1]), r, (int)(row + col[0]), 0, 0);
  } else {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    if constexpr (VW == 8) {
#pragma unroll
      for (int k = 0; k < 8; k += 4)
        __builtin_amdgcn_raw_buffer_store_b128(u4{__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])},
                                               r, (int)(row + col[0] + 4 * k), 0, 0);
    } else if constexpr (VW == 4)
      __builtin_amdgcn_raw_buffer_store_b128(u4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, r,
                                             (int)(row + col[0]), 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b64(u2{__float_as_uint(v[0]), __float_as_uint(v[1])}, r, (int)(row + col[0]), 0, 0);
  }
}

// v[i] of the LN lanes of a channel (lane bits 2 ..), summed over them: lane q of them returns the sum
// of v[q].  Each step halves the values: a lane keeps those that its own bit selects.
template <int LN>
__device__ __forceinline__ float spread4(const float (&v)[LN], int q) {
  if constexpr (LN == 1) {
    return v[0];
  } else {
    constexpr int half = LN / 2;
    float r[half];
#pragma unroll
    for (int i = 0; i < half; ++i) {
      if constexpr (LN >= 8) {  // the rows of 16 (halves of 32) trade places: one's own and the partner's values meet
        const uint32_t a = __float_as_uint(v[i]), b = __float_as_uint(v[i + half]);
        const auto w = LN == 16 ? __builtin_amdgcn_permlane32_swap(a, b, false, false) : __builtin_amdgcn_permlane16_swap(a, b, false, false);
        r[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
      } else {
        constexpr int kDown = LN == 4 ? 0x128 : 0x104, kUp = LN == 4 ? 0x128 : 0x114;  // lane ^ 8 by rotation; lane + 4, lane - 4
        const float lo = v[i] + dpp<kDown>(v[i]), hi = v[i + half] + dpp<kUp>(v[i + half]);
        r[i] = q & half ? hi : lo;
      }
    }
    return spread4<half>(r, q);
  }
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

}  // namespace wkv
