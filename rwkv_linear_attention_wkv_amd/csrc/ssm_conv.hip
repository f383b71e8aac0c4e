// The short causal convolution over the channels of a token array, W = 2 .. 4 taps:
//   pre_t[d] = bias[d] + sum_j weight[d][j] x_(t-W+1+j)[d],   y = pre or pre * sigmoid(pre)
// with the W - 1 inputs before a sequence held as its state (oldest first).  RWKV's token shift
// x + mu (x_(t-1) - x) is the form with W = 2 and taps (mu, 1 - mu).
//
// Bound by memory: one read of x and one write of y.  A lane owns V adjacent channels (one load of
// up to 16 bytes) and walks a segment of the sequence with the last W - 1 inputs in registers, so
// that an input is read once but for the W - 1 before each segment.  Lane 0's segment also owns
// the state: it reads it, and writes the new one, so that a call may update it in place.
#include "ssm_device.hpp"

namespace wkv {
namespace {

template <bool BF16, bool YBF16, int W, int V>
__global__ void __launch_bounds__(256) ssm_conv_kernel(ConvParams p) {
  const int lane = threadIdx.x & 63, seg = blockIdx.y;
  const Sequence q = find_sequence(p.seq, blockIdx.z, lane);
  const int t0 = seg * p.seg_len;
  if (!q.ok || (seg && t0 >= q.len)) return;
  const long c = ((long)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= p.D) return;

  float w[W][V], bias[V], prev[W - 1][V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = p.weight[(c + e) * W + j];
    bias[e] = p.bias ? p.bias[c + e] : 0.f;
  }
  if (seg == 0) {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) prev[i][e] = 0.f;
      if (p.seq.state_in) loadv<false>(p.seq.state_in, ((long)q.row_in * (W - 1) + i) * p.D + c, prev[i]);
    }
    // an empty slot's state stays as it is; elsewhere an empty sequence hands its state on
    if (p.seq.state_out && !(q.len == 0 && p.seq.state_out == p.seq.state_in)) {
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int pos = q.len - (W - 1) + i;
        float v[V];
        if (pos >= 0) {
          loadv<BF16>(p.x.base, (q.off + pos) * p.x.stride + c, v);
        } else {
#pragma unroll
          for (int k = 0; k < W - 1; ++k)
            if (k == pos + W - 1) {
#pragma unroll
              for (int e = 0; e < V; ++e) v[e] = prev[k][e];
            }
        }
        storev<false>(p.seq.state_out, ((long)q.row_out * (W - 1) + i) * p.D + c, v);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) loadv<BF16>(p.x.base, (q.off + t0 - (W - 1) + i) * p.x.stride + c, prev[i]);
  }

  const int t1 = min(t0 + p.seg_len, q.len);
  constexpr int U = 4;
  for (int t = t0; t < t1; t += U) {
    float x[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u < t1) loadv<BF16>(p.x.base, (q.off + t + u) * p.x.stride + c, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u < t1) {
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float a = bias[e];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], prev[j][e], a);
          a = fmaf(w[W - 1][e], x[u][e], a);
          y[e] = p.silu ? a * sigmoid_f(a) : a;
#pragma unroll
          for (int j = 0; j < W - 2; ++j) prev[j][e] = prev[j + 1][e];
          prev[W - 2][e] = x[u][e];
        }
        storev<YBF16>(p.y, (q.off + t + u) * p.D + c, y);
      }
    }
  }
}

// Backward.  With d_t = dy_t act'(pre_t) (0 outside the sequence):
//   dx_s = sum_j weight[j] d_(s+W-1-j), plus the final state's gradient for the last W - 1 inputs (the
//   state before the first token is such an input too);  dweight[j] = sum_t d_t x_(t-W+1+j), dbias = sum_t d_t
// One read of x and dy, one write of dx: a lane walks its segment once with the last W - 1 inputs and d
// in registers, W - 1 tokens past its end.  The sums over tokens leave one row per segment, which a
// second kernel adds in order.
template <bool BF16, int W, int V>
__global__ void __launch_bounds__(256) ssm_conv_backward_kernel(ConvParams p) {
  const int lane = threadIdx.x & 63, seg = blockIdx.y;
  const Sequence q = find_sequence(p.seq, blockIdx.z, lane);
  const long c = ((long)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= p.D) return;
  float dw[W + 1][V];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.f;
  const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, q.len);
  if (q.ok) {
    float w[W][V], bias[V], x[W][V], d[W][V];  // x, d: tokens t - W + 1 .. t
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = p.weight[(c + e) * W + j];
      bias[e] = p.bias ? p.bias[c + e] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) x[i][e] = d[i][e] = 0.f;
      const int t = t0 - W + i;  // one place early: the loop shifts before it uses them
      if (i > 0) {
        if (t >= 0) loadv<BF16>(p.x.base, (q.off + t) * p.x.stride + c, x[i]);
        else if (p.seq.state_in) loadv<false>(p.seq.state_in, ((long)q.row_in * (W - 1) + t + W - 1) * p.D + c, x[i]);
      }
    }
    constexpr int U = 4;
    const int end = t1 + W - 1;
    for (int tb = t0; tb < end; tb += U) {
      float nx[U][V], ny[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (tb + u < min(end, q.len)) {
          loadv<BF16>(p.x.base, (q.off + tb + u) * p.x.stride + c, nx[u]);
          if (p.dy_bf16) loadv<true>(p.dy.base, (q.off + tb + u) * p.dy.stride + c, ny[u]);
          else loadv<false>(p.dy.base, (q.off + tb + u) * p.dy.stride + c, ny[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u;
        if (t < end) {
          const bool in = t < q.len;
          float g[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) { x[i][e] = x[i + 1][e]; d[i][e] = d[i + 1][e]; }
            x[W - 1][e] = in ? nx[u][e] : 0.f;
            float grad = in ? ny[u][e] : 0.f;
            if (p.silu) {
              float a = bias[e];
#pragma unroll
              for (int j = 0; j < W; ++j) a = fmaf(w[j][e], x[j][e], a);
              const float sg = sigmoid_f(a);
              grad *= sg * fmaf(a, 1.f - sg, 1.f);
              grad = in ? grad : 0.f;
            }
            d[W - 1][e] = grad;
            if (t < t1) {
#pragma unroll
              for (int j = 0; j < W; ++j) dw[j][e] = fmaf(grad, x[j][e], dw[j][e]);
              dw[W][e] += grad;
            }
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) v = fmaf(w[W - 1 - i][e], d[i][e], v);
            g[e] = v;
          }
          const int s = t - (W - 1), last = s - (q.len - (W - 1));  // last >= 0: the input is a row of the final state
          if (s >= t0 || (seg == 0 && p.d_state_in)) {
            if (last >= 0 && p.d_state_out) {
              float more[V];
              loadv<false>(p.d_state_out, ((long)blockIdx.z * (W - 1) + last) * p.D + c, more);
#pragma unroll
              for (int e = 0; e < V; ++e) g[e] += more[e];
            }
            if (s < 0) storev<false>(p.d_state_in, ((long)blockIdx.z * (W - 1) + s + W - 1) * p.D + c, g);
            else if (p.y_bf16) storev<true>(p.y, (q.off + s) * p.D + c, g);
            else storev<false>(p.y, (q.off + s) * p.D + c, g);
          }
        }
      }
    }
  }
  const long row = (long)blockIdx.z * p.nseg + seg;
#pragma unroll
  for (int j = 0; j <= W; ++j) storev<false>(p.partial, (row * (W + 1) + j) * p.D + c, dw[j]);
}

// dweight [D, W] and dbias [D] from the segments' rows [W + 1, D]: 16 threads each add every 16th row,
// then their sums in order.
__global__ void __launch_bounds__(256) ssm_conv_sum_kernel(ConvParams p) {
  __shared__ float s[16][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4, j = blockIdx.y;
  const long d = (long)blockIdx.x * 16 + c, rows = (long)p.seq.units * p.nseg;
  float a = 0.f;
  if (d < p.D) {
#pragma unroll 4
    for (long r = k; r < rows; r += 16) a += p.partial[(r * (p.W + 1) + j) * p.D + d];
  }
  s[k][c] = a;
  __syncthreads();
  if (k == 0 && d < p.D) {
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += s[i][c];
    if (j < p.W) p.d_weight[d * p.W + j] = t;
    else if (p.d_bias) p.d_bias[d] = t;
  }
}

template <bool BF16, int W, int V>
hipError_t go_backward(const ConvParams &p, hipStream_t s) {
  const int lanes = (p.D + V - 1) / V;
  const int block = lanes >= 256 ? 256 : (lanes + 63) / 64 * 64;
  hipLaunchKernelGGL((ssm_conv_backward_kernel<BF16, W, V>), dim3((lanes + block - 1) / block, p.nseg, p.seq.units), dim3(block), 0, s, p);
  hipLaunchKernelGGL(ssm_conv_sum_kernel, dim3((p.D + 15) / 16, W + 1), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int V>
hipError_t backward_by_width(const ConvParams &p, hipStream_t s) {
  return p.W == 2 ? go_backward<BF16, 2, V>(p, s) : p.W == 3 ? go_backward<BF16, 3, V>(p, s) : go_backward<BF16, 4, V>(p, s);
}

template <bool BF16, int W, int V>
hipError_t go(const ConvParams &p, hipStream_t s) {
  const int lanes = (p.D + V - 1) / V;
  const int block = lanes >= 256 ? 256 : (lanes + 63) / 64 * 64;
  const dim3 grid((lanes + block - 1) / block, p.nseg, p.seq.units);
  if (p.y_bf16) hipLaunchKernelGGL((ssm_conv_kernel<BF16, true, W, V>), grid, dim3(block), 0, s, p);
  else hipLaunchKernelGGL((ssm_conv_kernel<BF16, false, W, V>), grid, dim3(block), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int V>
hipError_t by_width(const ConvParams &p, hipStream_t s) {
  return p.W == 2 ? go<BF16, 2, V>(p, s) : p.W == 3 ? go<BF16, 3, V>(p, s) : go<BF16, 4, V>(p, s);
}

// Whether V channels at a time stay aligned in every row of the array.
bool fits(const void *base, long stride, int elem, int V) {
  return stride % V == 0 && reinterpret_cast<uintptr_t>(base) % (unsigned)(V * elem) == 0;
}

}  // namespace

// Tokens of one walk.
int conv_segments(int units, int T, int D, bool backward, int *seg_len) {
  int len = 64;
  while ((long)len * 65535 < T) len *= 2;
  *seg_len = len;
  return T > 0 ? (T + len - 1) / len : 1;
}

hipError_t launch_ssm_conv(const ConvParams &p, bool bf16, hipStream_t s) {
  const int elem = bf16 ? 2 : 4, yel = p.y_bf16 ? 2 : 4;
  const auto can = [&](int V) { return p.D % V == 0 && fits(p.x.base, p.x.stride, elem, V) && fits(p.y, p.D, yel, V); };
  if (bf16) return can(8) ? by_width<true, 8>(p, s) : can(2) ? by_width<true, 2>(p, s) : by_width<true, 1>(p, s);
  return can(4) ? by_width<false, 4>(p, s) : by_width<false, 1>(p, s);
}

hipError_t launch_ssm_conv_backward(const ConvParams &p, bool bf16, hipStream_t s) {
  const auto can = [&](int V) {
    return p.D % V == 0 && fits(p.x.base, p.x.stride, bf16 ? 2 : 4, V) && fits(p.dy.base, p.dy.stride, p.dy_bf16 ? 2 : 4, V);
  };
  if (bf16) return can(4) ? backward_by_width<true, 4>(p, s) : backward_by_width<true, 1>(p, s);
  return can(4) ? backward_by_width<false, 4>(p, s) : backward_by_width<false, 1>(p, s);
}

}  // namespace wkv
