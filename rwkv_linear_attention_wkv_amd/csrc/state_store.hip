// The 8-bit store of carried states.  A row of `row` fp32 values is kept in groups of 64 (one key
// row of a WKV head, a few channels of a scan state): scale = max|v| / 127 (int8) or / 448 (e4m3),
// code = nearest to v / scale, ties to even; the last group may be short.  Both quotients are the
// fp32 ones, correctly rounded, so that codes do not depend on the kernel.  A group of zeros has
// scale 0; a group that holds an infinity or NaN has scale NaN and reads back as NaN throughout.
//
// Bound by memory (4 bytes in, 1 + 1/16 out, or the reverse): 16 lanes share a group, four values
// each, so a wave reads 1 KiB in one load; the group's largest magnitude is four DPP steps.  A set of
// lanes takes four groups at once, for loads enough in flight.  Writing 64 rows of 131072 values: 8.7 us,
// 4.9 TB/s (13.9 us with a group at a time and divisions).
#include "ssm_device.hpp"

namespace wkv {
namespace {

constexpr int kGroup = 64;

// Whether item `item`'s destination row `to` is also another item's, for a whole wave.
__device__ __forceinline__ bool shared_row(const int32_t *rows, int count, int item, int to, int lane) {
  bool dup = false;
  if (rows)
    for (int i = lane; i < count; i += 64) dup |= i != item && rows[i] == to;
  return __any(dup);
}

__device__ __forceinline__ bool store_item(const StoreParams &p, int item, int lane, bool to_store, long &cached, long &state) {
  const int c = p.store_rows ? p.store_rows[item] : item, s = p.state_rows ? p.state_rows[item] : item;
  int status = 0;
  if (c < 0 || c >= p.n_store || s < 0 || s >= p.n_state) status |= WKV_DEV_BAD_STATE_MAP;
  if (shared_row(to_store ? p.store_rows : p.state_rows, p.count, item, to_store ? c : s, lane)) status |= WKV_DEV_DUPLICATE_ROW;
  if (status && lane == 0 && p.dev_status) atomicOr(p.dev_status, status);
  cached = c;
  state = s;
  return status == 0;
}

constexpr int kRounds = 4;  // groups that a set of 16 lanes takes, all loaded before the first is used

// Four adjacent values of a row of `n`, from e on, that fit or are 0 beyond it.
template <bool VEC>
__device__ __forceinline__ void load_row4(const float *row, long e, long n, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = 0.f;
  if constexpr (VEC) {
    if (e < n) loadv<false>(row, e, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < n) v[i] = row[e + i];
  }
}

// v / scale, correctly rounded.  With y the correctly rounded 1 / scale (the hardware's and one Newton
// step: that is it for every mantissa but all ones) and q = v y, the remainder v - q scale is exact and
// q + remainder y rounds to the quotient (Markstein's theorem); two multiplies and an fma a value where
// a division takes ten instructions.  Only where neither leaves the normal range: see plain_division().
__device__ __forceinline__ float quotient(float v, float scale, float y) {
  const float q = v * y;
  return fmaf(fmaf(-q, scale, v), y, q);
}

__device__ __forceinline__ bool plain_division(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return (b & 0x7fffffu) == 0x7fffffu || b < (67u << 23) || b > (227u << 23);  // outside 2^-60 .. 2^100
}

template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(256) store_write_kernel(StoreParams p) {
  const int lane = threadIdx.x & 63;
  long cached, state;
  if (!store_item(p, blockIdx.y, lane, true, cached, state)) return;
  const long groups = (p.row + kGroup - 1) / kGroup;
  const float *src = p.states + state * p.row;
  uint8_t *dst = static_cast<uint8_t *>(p.data) + cached * p.row;
  const int set = threadIdx.x / 16, sub = 4 * (threadIdx.x & 15);
  for (long first = (long)blockIdx.x * 16 * kRounds; first < groups; first += (long)gridDim.x * 16 * kRounds) {
    float v[kRounds][4];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) load_row4<VEC>(src, (first + k * 16 + set) * kGroup + sub, p.row, v[k]);
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const long g = first + k * 16 + set, e = g * kGroup + sub;
      // magnitudes compare as their bits do, with infinities and NaN above every number
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7fffffffu);
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, kXor1, 0xf, 0xf, true));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, kXor2, 0xf, 0xf, true));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, kHalfMirror, 0xf, 0xf, true));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, kMirror, 0xf, 0xf, true));
      const float limit = E4M3 ? 448.f : 127.f;
      const bool finite = top < 0x7f800000u;
      const float scale = finite ? __uint_as_float(top) / limit : __uint_as_float(0x7fc00000u);
      float c[4];
      if (plain_division(scale)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = scale > 0.f ? v[k][i] / scale : 0.f;
      } else {
        const float y0 = fast_rcp(scale), y = fmaf(fmaf(-scale, y0, 1.f), y0, y0);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = quotient(v[k][i], scale, y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(c[i], -limit), limit);
      uint32_t code;
      if constexpr (E4M3) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        code = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
      } else {
        code = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) code |= ((uint32_t)(int)rintf(c[i]) & 0xffu) << (8 * i);
      }
      if constexpr (VEC) {
        if (e < p.row) *reinterpret_cast<uint32_t *>(dst + e) = code;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < p.row) dst[e + i] = (uint8_t)(code >> (8 * i));
      }
      if (sub == 0 && g < groups) p.scale[cached * groups + g] = scale;
    }
  }
}

template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(256) store_read_kernel(StoreParams p) {
  const int lane = threadIdx.x & 63;
  long cached, state;
  if (!store_item(p, blockIdx.y, lane, false, cached, state)) return;
  const long groups = (p.row + kGroup - 1) / kGroup;
  const uint8_t *src = static_cast<const uint8_t *>(p.data) + cached * p.row;
  float *dst = p.states + state * p.row;
  const int set = threadIdx.x / 16, sub = 4 * (threadIdx.x & 15);
  for (long first = (long)blockIdx.x * 16 * kRounds; first < groups; first += (long)gridDim.x * 16 * kRounds) {
    uint32_t code[kRounds];
    float scale[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const long g = first + k * 16 + set, e = g * kGroup + sub;
      code[k] = 0;
      if constexpr (VEC) {
        if (e < p.row) code[k] = *reinterpret_cast<const uint32_t *>(src + e);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < p.row) code[k] |= (uint32_t)src[e + i] << (8 * i);
      }
      scale[k] = g < groups ? p.scale[cached * groups + g] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const long e = (first + k * 16 + set) * kGroup + sub;
      float v[4];
      if constexpr (E4M3) {
        v[0] = __builtin_amdgcn_cvt_f32_fp8((int)code[k], 0); v[1] = __builtin_amdgcn_cvt_f32_fp8((int)code[k], 1);
        v[2] = __builtin_amdgcn_cvt_f32_fp8((int)code[k], 2); v[3] = __builtin_amdgcn_cvt_f32_fp8((int)code[k], 3);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(code[k] >> (8 * i));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= scale[k];
      if constexpr (VEC) {
        if (e < p.row) storev<false>(dst, e, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < p.row) dst[e + i] = v[i];
      }
    }
  }
}

dim3 store_grid(const StoreParams &p) {
  const long per_block = 16 * kRounds, blocks = ((p.row + kGroup - 1) / kGroup + per_block - 1) / per_block;
  return dim3((unsigned)(blocks < 4096 ? blocks : 4096), p.count);
}

}  // namespace

hipError_t launch_store_write(const StoreParams &p, hipStream_t s) {
  const bool vec = p.row % 4 == 0;  // the tables are 16-byte aligned
  if (p.e4m3) {
    if (vec) hipLaunchKernelGGL((store_write_kernel<true, true>), store_grid(p), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((store_write_kernel<true, false>), store_grid(p), dim3(256), 0, s, p);
  } else {
    if (vec) hipLaunchKernelGGL((store_write_kernel<false, true>), store_grid(p), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((store_write_kernel<false, false>), store_grid(p), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

hipError_t launch_store_read(const StoreParams &p, hipStream_t s) {
  const bool vec = p.row % 4 == 0;
  if (p.e4m3) {
    if (vec) hipLaunchKernelGGL((store_read_kernel<true, true>), store_grid(p), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((store_read_kernel<true, false>), store_grid(p), dim3(256), 0, s, p);
  } else {
    if (vec) hipLaunchKernelGGL((store_read_kernel<false, true>), store_grid(p), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((store_read_kernel<false, false>), store_grid(p), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace wkv
