// The selective state space scan.  Per channel d and state n, with delta = softplus(dt + dt_bias):
//   h[n] <- e^(delta A[d][n]) h[n] + delta x B[n],   y = sum_n C[n] h[n] + skip[d] x,  y *= z sigmoid(z)
// States and sums are fp32; a bf16 y is the fp32 result rounded to nearest even.
#include "ssm_device.hpp"

namespace wkv {
namespace {

// Four state values of one channel: values 4q .. 4q + 3 of the N a row holds (zero beyond N).
__device__ __forceinline__ void load_state4(const float *row, int q, int N, bool whole, float (&h)[4]) {
  if (whole) {
    loadv<false>(row, 4 * q, h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = 4 * q + i < N ? row[4 * q + i] : 0.f;
  }
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

// LN adjacent lanes share a channel, four states each; the tokens are walked one by one.
template <bool BF16, int LN>
__global__ void __launch_bounds__(256) ssm_scan_short_kernel(ScanSsmParams p) {
  constexpr int CH = 256 / LN;  // channels of a workgroup
  const int lane = threadIdx.x & 63, q = threadIdx.x % LN;
  const Sequence sq = find_sequence(p.seq, blockIdx.y, lane);
  if (!sq.ok) return;
  const int per_group = p.D / p.G, blocks = (per_group + CH - 1) / CH;
  const int g = blockIdx.x / blocks, in_group = (blockIdx.x % blocks) * CH + threadIdx.x / LN;
  const bool live = in_group < per_group;
  const long d = (long)g * per_group + (live ? in_group : 0);
  const int N = p.N;
  const bool whole = (N & 3) == 0 && 4 * q < N;
  float A[4], h[4] = {0.f, 0.f, 0.f, 0.f};
  load_state4(p.A + d * N, q, N, whole, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
  if (p.seq.state_in) load_state4(p.seq.state_in + ((long)sq.row_in * p.D + d) * N, q, N, whole, h);
  const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
  for (int t = 0; t < sq.len; ++t) {
    const long r = sq.off + t;
    const float x = load1<BF16>(p.x.base, r * p.x.stride + d);
    const float raw = load1<BF16>(p.dt.base, r * p.dt.stride + d) + bias;
    const float delta = p.softplus ? softplus_f(raw) : raw, dx = delta * x;
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 4 * q + i;
      const float b = n < N ? load1<BF16>(p.Bm.base, r * p.Bm.stride + g * N + n) : 0.f;
      const float c = n < N ? load1<BF16>(p.Cm.base, r * p.Cm.stride + g * N + n) : 0.f;
      h[i] = fmaf(__builtin_amdgcn_exp2f(delta * A[i]), h[i], dx * b);
      part = fmaf(c, h[i], part);
    }
    float y = fmaf(skip, x, sum_all<LN>(part));
    if (p.z.base) {
      const float z = load1<BF16>(p.z.base, r * p.z.stride + d);
      y *= z * sigmoid_f(z);
    }
    if (live && q == 0) store1(p.y, r * p.D + d, p.y_bf16, y);
  }
  if (live && p.seq.state_out && !(sq.len == 0 && p.seq.state_out == p.seq.state_in))
    store_state4(p.seq.state_out + ((long)sq.row_out * p.D + d) * N, q, N, whole, h);
}

template <bool BF16, int LN>
hipError_t go_short(const ScanSsmParams &p, hipStream_t s) {
  constexpr int CH = 256 / LN;
  const int per_group = p.D / p.G;
  const dim3 grid(p.G * ((per_group + CH - 1) / CH), p.seq.units);
  hipLaunchKernelGGL((ssm_scan_short_kernel<BF16, LN>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_states(const ScanSsmParams &p, hipStream_t s) {
  if (p.N <= 4) return go_short<BF16, 1>(p, s);
  if (p.N <= 8) return go_short<BF16, 2>(p, s);
  if (p.N <= 16) return go_short<BF16, 4>(p, s);
  if (p.N <= 32) return go_short<BF16, 8>(p, s);
  return go_short<BF16, 16>(p, s);
}

}  // namespace

hipError_t launch_ssm_scan(const ScanSsmParams &p, bool bf16, hipStream_t s) {
  return bf16 ? by_states<true>(p, s) : by_states<false>(p, s);
}

}  // namespace wkv
