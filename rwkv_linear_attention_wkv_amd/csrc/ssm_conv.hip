// The short causal convolution over the channels of a token array, W = 2 .. 4 taps:
//   pre_t[d] = bias[d] + sum_j weight[d][j] x_(t-W+1+j)[d],   y = pre or pre * sigmoid(pre)
// with the W - 1 inputs before a sequence held as its state (oldest first).  RWKV's token shift
// x + mu (x_(t-1) - x) is the form with W = 2 and taps (mu, 1 - mu).
//
// Bound by memory: one read of x and one write of y.  A lane owns V adjacent channels (one load of
// up to 16 bytes) and walks a segment of the sequence with the last W - 1 inputs in registers, so
// that an input is read once but for the W - 1 before each segment; loads run U tokens ahead, into two
// sets of registers in turn.  The first segment also owns the state: it reads it, and writes the new
// one, so that a call may update it in place.  [8, 4096, 4096] bf16, W = 4: 108 us, 4.97 TB/s, what a
// plain copy of that size reaches (116 us with one set that each round was copied into); a step of 64
// slots, D = 2048: 6.7 us, of which an empty launch is 2.9 and the bytes 0.7.
#include "ssm_tile.hpp"

namespace wkv {
namespace {

constexpr int U = 4;  // tokens of one round of loads

// The taps and bias of V adjacent channels.
template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvParams &p, long c, float (&w)[W][V], float (&bias)[V]) {
  float flat[V * W];
  loadv<false>(p.weight, c * W, flat);
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
    bias[e] = p.bias ? p.bias[c + e] : 0.f;
  }
}

// A lane's V channels from c on (none where c is D or more), of segment seg.
template <bool BF16, bool YBF16, int W, int V>
__device__ __forceinline__ void conv_walk(const ConvParams &p, int seg, long c) {
  const int lane = threadIdx.x & 63;
  float w[W][V], bias[V], prev[W - 1][V];
  if (c < p.D) load_taps(p, c, w, bias);
  const Sequence q = find_sequence(p.seq, blockIdx.y, lane);
  const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, q.len);
  if (!q.ok || (seg && t0 >= q.len)) return;
  if (c >= p.D) return;

  constexpr int EL = BF16 ? 2 : 4, YEL = YBF16 ? 2 : 4;
  constexpr bool VEC = V > 1;
  using Raw = RawRow<BF16, VEC, V>;
  const auto wx = window<EL>(p.x.base, p.x.stride, q.off + t0, t1 - t0, 0, p.D);
  const auto wy = window<YEL>(p.y, p.D, q.off + t0, t1 - t0, 0, p.D);
  const uint32_t col[1] = {(uint32_t)c * EL}, ycol[1] = {(uint32_t)c * YEL};
  const uint32_t step = (uint32_t)p.x.stride * EL, ystep = (uint32_t)p.D * YEL;
  Raw x[2][U];  // rounds in turn, so that none is copied (a copy waits for its loads)
  const auto request = [&](Raw (&to)[U], int t) {  // rows past the segment read 0, and their results are not written
#pragma unroll
    for (int u = 0; u < U; ++u) to[u].load(wx, (t + u) * step, col);
  };
  request(x[0], 0);

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

  const auto arrive = [&](Raw (&now)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) now[u].arrive();
  };
  const auto round = [&](Raw (&now)[U], int t) {
    arrive(now);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xe = now[u].get(e);
        float a = bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], prev[j][e], a);
        a = fmaf(w[W - 1][e], xe, a);
        y[e] = p.silu ? a * sigmoid_f(a) : a;
#pragma unroll
        for (int j = 0; j < W - 2; ++j) prev[j][e] = prev[j + 1][e];
        prev[W - 2][e] = xe;
      }
      store_row<YBF16, VEC, V>(wy, (t + u) * ystep, ycol, y);
    }
  };
  for (int t = 0; t < t1 - t0; t += 2 * U) {
    request(x[1], t + U);
    round(x[0], t);
    if (t + U >= t1 - t0) {
      arrive(x[1]);  // (else the compiler waits at the head of the loop, for every round)
      break;
    }
    request(x[0], t + 2 * U);
    round(x[1], t + U);
  }
}

// The blocks of one segment: whole ones of V channels a lane, then one for the D % V channels left.
struct Blocks {
  int threads, whole, all;
};

template <int V>
Blocks blocks_of(int D) {
  const int lanes = D / V, threads = lanes >= 256 ? 256 : lanes > 0 ? (lanes + 63) / 64 * 64 : 64;
  const int whole = (lanes + threads - 1) / threads;
  return {threads, whole, whole + (D % V ? 1 : 0)};
}

template <bool BF16, bool YBF16, int W, int V>
__global__ void __launch_bounds__(256) ssm_conv_kernel(ConvParams p) {
  const int blocks = gridDim.x / p.nseg, seg = blockIdx.x / blocks, block = blockIdx.x % blocks;
  const long lane = (long)block * blockDim.x + threadIdx.x, lanes = p.D / V;
  if (V > 1 && p.D % V && block == blocks - 1) conv_walk<BF16, YBF16, W, 1>(p, seg, lanes * V + threadIdx.x);
  else conv_walk<BF16, YBF16, W, V>(p, seg, lane < lanes ? lane * V : p.D);
}

template <bool BF16, int W, int V>
hipError_t go(const ConvParams &p, hipStream_t s) {
  const Blocks b = blocks_of<V>(p.D);
  const dim3 grid((unsigned)((long)b.all * p.nseg), p.seq.units);
  if (p.y_bf16) hipLaunchKernelGGL((ssm_conv_kernel<BF16, true, W, V>), grid, dim3(b.threads), 0, s, p);
  else hipLaunchKernelGGL((ssm_conv_kernel<BF16, false, W, V>), grid, dim3(b.threads), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int V>
hipError_t by_width(const ConvParams &p, hipStream_t s) {
  return p.W == 2 ? go<BF16, 2, V>(p, s) : p.W == 3 ? go<BF16, 3, V>(p, s) : go<BF16, 4, V>(p, s);
}

// Backward.  With d_t = dy_t act'(pre_t) (0 outside the sequence):
//   dx_s = sum_j weight[j] d_(s+W-1-j), plus the final state's gradient for the last W - 1 inputs (the
//   state before the first token is such an input too);  dweight[j] = sum_t d_t x_(t-W+1+j), dbias = sum_t d_t
// One read of x and dy, one write of dx: a lane walks its segment once with the last W - 1 inputs and d
// in registers, W - 1 tokens past its end.  The sums over tokens leave one row per segment, which a
// second kernel adds in order.  [4, 2047, 2048] bf16, W = 4: 25.8 us (3.9 TB/s; some 45 vector
// instructions a value stand beside its 6 bytes) and 4.0 us for the sums.
template <bool BF16, bool DYBF16, int W, int V>
__device__ __forceinline__ void conv_walk_back(const ConvParams &p, int seg, long c) {
  const Sequence q = find_sequence(p.seq, blockIdx.y, threadIdx.x & 63);
  if (c >= p.D) return;
  float dw[W + 1][V];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.f;
  const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, q.len);
  if (q.ok) {
    constexpr int EL = BF16 ? 2 : 4, DEL = DYBF16 ? 2 : 4;
    constexpr bool VEC = V > 1;
    float w[W][V], bias[V], x[W][V], d[W][V];  // x, d: tokens t - W + 1 .. t
    const int end = t1 + W - 1, rows = min(end, q.len) - t0;
    const auto wx = window<EL>(p.x.base, p.x.stride, q.off + t0, rows, 0, p.D);
    const auto wd = window<DEL>(p.dy.base, p.dy.stride, q.off + t0, rows, 0, p.D);
    const uint32_t col[1] = {(uint32_t)c * EL}, dcol[1] = {(uint32_t)c * DEL};
    const uint32_t step = (uint32_t)p.x.stride * EL, dstep = (uint32_t)p.dy.stride * DEL;
    // Only the rows of this segment: the walk's first and last steps form others, which are not written.
    const auto wg = p.y_bf16 ? window<2>(p.y, p.D, q.off + t0, t1 - t0, 0, p.D) : window<4>(p.y, p.D, q.off + t0, t1 - t0, 0, p.D);
    const uint32_t gcol[1] = {(uint32_t)c * (p.y_bf16 ? 2 : 4)}, gstep = (uint32_t)p.D * (p.y_bf16 ? 2 : 4);
    struct Round {  // two in turn, so that none is copied (a copy waits for its loads)
      RawRow<BF16, VEC, V> x[U];
      RawRow<DYBF16, VEC, V> dy[U];
      __device__ __forceinline__ void arrive() {
#pragma unroll
        for (int u = 0; u < U; ++u) { x[u].arrive(); dy[u].arrive(); }
      }
    } rounds[2];
    const auto request = [&](Round &to, int t) {  // rows past the sequence or the walk read 0
#pragma unroll
      for (int u = 0; u < U; ++u) {
        to.x[u].load(wx, (t + u) * step, col);
        to.dy[u].load(wd, (t + u) * dstep, dcol);
      }
    };
    request(rounds[0], 0);
    load_taps(p, c, w, bias);
#pragma unroll
    for (int i = 0; i < W; ++i)  // one place early: the walk shifts before it uses them
#pragma unroll
      for (int e = 0; e < V; ++e) x[i][e] = d[i][e] = 0.f;
    if (seg) {
#pragma unroll
      for (int i = 1; i < W; ++i) loadv<BF16>(p.x.base, (q.off + t0 - W + i) * p.x.stride + c, x[i]);
    } else if (p.seq.state_in) {
#pragma unroll
      for (int i = 1; i < W; ++i) loadv<false>(p.seq.state_in, ((long)q.row_in * (W - 1) + i - 1) * p.D + c, x[i]);
    }
    const auto walk = [&](Round &now, int from) {
      now.arrive();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + from + u;
        float g[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
          for (int i = 0; i < W - 1; ++i) { x[i][e] = x[i + 1][e]; d[i][e] = d[i + 1][e]; }
          x[W - 1][e] = now.x[u].get(e);
          const float grad = now.dy[u].get(e);
          float a = bias[e];
#pragma unroll
          for (int j = 0; j < W; ++j) a = fmaf(w[j][e], x[j][e], a);
          const float sg = sigmoid_f(a), through = p.silu ? grad * (sg * fmaf(a, 1.f - sg, 1.f)) : grad;
          d[W - 1][e] = t < q.len ? through : 0.f;
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < W; ++i) v = fmaf(w[W - 1 - i][e], d[i][e], v);
          g[e] = v;
        }
        if (t < t1) {  // the taps' gradients of other tokens are another segment's
#pragma unroll
          for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] = fmaf(d[W - 1][e], x[j][e], dw[j][e]);
            dw[W][e] += d[W - 1][e];
          }
        }
        const int s = t - (W - 1), last = s - (q.len - (W - 1));  // last >= 0: the input is a row of the final state
        if (last >= 0 && t < end && p.d_state_out) {
          float more[V];
          loadv<false>(p.d_state_out, ((long)blockIdx.y * (W - 1) + last) * p.D + c, more);
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] += more[e];
        }
        const uint32_t at = (uint32_t)(s - t0) * gstep;  // before the window: beyond its end
        if (p.y_bf16) store_row<true, VEC, V>(wg, at, gcol, g);
        else store_row<false, VEC, V>(wg, at, gcol, g);
        if (s < 0 && seg == 0 && t < end && p.d_state_in)
          storev<false>(p.d_state_in, ((long)blockIdx.y * (W - 1) + s + W - 1) * p.D + c, g);
      }
    };
    for (int t = 0; t < end - t0; t += 2 * U) {
      request(rounds[1], t + U);
      walk(rounds[0], t);
      if (t + U >= end - t0) {
        rounds[1].arrive();  // (else the compiler waits at the head of the loop, for every round)
        break;
      }
      request(rounds[0], t + 2 * U);
      walk(rounds[1], t + U);
    }
  }
  const long row = (long)blockIdx.y * p.nseg + seg;
#pragma unroll
  for (int j = 0; j <= W; ++j) storev<false>(p.partial, (row * (W + 1) + j) * p.D + c, dw[j]);
}

template <bool BF16, bool DYBF16, int W, int V>
__global__ void __launch_bounds__(256) ssm_conv_backward_kernel(ConvParams p) {
  const int blocks = gridDim.x / p.nseg, seg = blockIdx.x / blocks, block = blockIdx.x % blocks;
  const long lane = (long)block * blockDim.x + threadIdx.x, lanes = p.D / V;
  if (V > 1 && p.D % V && block == blocks - 1) conv_walk_back<BF16, DYBF16, W, 1>(p, seg, lanes * V + threadIdx.x);
  else conv_walk_back<BF16, DYBF16, W, V>(p, seg, lane < lanes ? lane * V : p.D);
}

// dweight [D, W] and dbias [D] from the segments' rows [W + 1, D]: 16 threads a column each add every 16th row,
// then their sums in order; 64 columns a workgroup, so that a row is read 256 bytes at a time.
__global__ void __launch_bounds__(1024) ssm_conv_sum_kernel(ConvParams p) {
  __shared__ float s[16][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6, j = blockIdx.y;
  const long d = (long)blockIdx.x * 64 + c, rows = (long)p.seq.units * p.nseg;
  float a = 0.f;
  if (d < p.D) {
#pragma unroll 8
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
  const Blocks b = blocks_of<V>(p.D);
  const dim3 grid((unsigned)((long)b.all * p.nseg), p.seq.units);
  if (p.dy_bf16) hipLaunchKernelGGL((ssm_conv_backward_kernel<BF16, true, W, V>), grid, dim3(b.threads), 0, s, p);
  else hipLaunchKernelGGL((ssm_conv_backward_kernel<BF16, false, W, V>), grid, dim3(b.threads), 0, s, p);
  hipLaunchKernelGGL(ssm_conv_sum_kernel, dim3((p.D + 63) / 64, W + 1), dim3(1024), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int V>
hipError_t backward_by_width(const ConvParams &p, hipStream_t s) {
  return p.W == 2 ? go_backward<BF16, 2, V>(p, s) : p.W == 3 ? go_backward<BF16, 3, V>(p, s) : go_backward<BF16, 4, V>(p, s);
}

}  // namespace

// Tokens of one walk: at most 64 (its W - 1 extra rows then cost 5 %), down to 16 until the walks are about a
// wave for every SIMD (backward two, as half the bytes are a wave's).  Measured at [4, 2047, 2048] bf16,
// W = 4: forward 15.2 us for 1024 waves, 17.0 for 2048; backward with its sums 35.9 us for 1024, 29.9 for
// 2048, 33.3 for 4096; 48 slots of up to 700 tokens, fp32: 19.8 us for 1300 waves, 23.3 for 650.
int conv_segments(int T, long total, int D, bool bf16, bool backward, int *seg_len) {
  const int V = bf16 && !backward ? 8 : 4;
  const long per_token = (D / V + 63) / 64;  // total counts the tokens that slots of unlike lengths have
  if (T > total) T = (int)total;  // no slot has more tokens than the call, whatever the host's bound
  int len = 64;
  while (len > 16 && per_token * total < (backward ? 1920L : 960L) * len) len /= 2;
  *seg_len = len;
  return T > 0 ? (T + len - 1) / len : 1;
}

hipError_t launch_ssm_conv(const ConvParams &p, bool bf16, hipStream_t s) {
  return bf16 ? by_width<true, 8>(p, s) : by_width<false, 4>(p, s);
}

hipError_t launch_ssm_conv_backward(const ConvParams &p, bool bf16, hipStream_t s) {
  return bf16 ? backward_by_width<true, 4>(p, s) : backward_by_width<false, 4>(p, s);
}

}  // namespace wkv
