// The selective state space scan.  Per channel d and state n, with delta = softplus(dt + dt_bias):
//   h[n] <- e^(delta A[d][n]) h[n] + delta x B[n],   y = sum_n C[n] h[n] + skip[d] x,  y *= z sigmoid(z)
// States and sums are fp32; a bf16 y is the fp32 result rounded to nearest even.
//
// Every (channel, state) has a decay of its own, so nothing here is a matrix product: a token costs
// D N exponentials (a quarter-rate instruction) and 4 D N multiplies and fused multiply-adds on the
// vector ALUs, against 8 D bytes of bf16 traffic.  With N = 16 the ALUs bound it.
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

// ------------------------------------------------------------------------------------------------
// Long sequences.  A workgroup of four waves owns 256 / LN channels and walks its segment in tiles
// of TT tokens.  Per tile, all threads first load (coalesced rows, one tile ahead) and form what a
// token and channel need once - delta, delta x - and the widened B and C rows, into LDS; then LN
// adjacent lanes walk a channel's tokens with four states each in registers; their partial sums over
// n are spread over the LN lanes by DPP halvings (LN tokens at a time), go back through LDS, and are
// finished (skip, gate, rounding) in the loading threads' layout, for row-wide stores.  Both LDS
// sides are double-buffered: one barrier per tile.
//
// Few rows: the sequence is cut into nseg segments.  The carry pass runs all but the last from a
// state of zero and leaves each one's final state and its sum of delta; as the decay over a segment
// is e^(A sum delta), the main pass folds the earlier segments' states into its own start.

template <bool BF16, bool VEC, int VW>
struct RawRow {  // VW adjacent elements as loaded
  uint32_t w[VEC && BF16 ? (VW + 1) / 2 : VW];
  __device__ __forceinline__ void load(const TokenArray &a, long row, long c, int live) {
#pragma unroll
    for (auto &x : w) x = 0;
    if constexpr (VEC) {
      if (live > 0) {
        const char *at = static_cast<const char *>(a.base) + (row * a.stride + c) * (BF16 ? 2 : 4);
        if constexpr (sizeof w == 16) {
          const uint4 v = *reinterpret_cast<const uint4 *>(at);
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (sizeof w == 8) {
          const uint2 v = *reinterpret_cast<const uint2 *>(at);
          w[0] = v.x; w[1] = v.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t *>(at);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (e < live) {
          if constexpr (BF16) w[e] = (uint32_t) static_cast<const uint16_t *>(a.base)[row * a.stride + c + e] << 16;
          else w[e] = static_cast<const uint32_t *>(a.base)[row * a.stride + c + e];
        }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (VEC && BF16) return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else return __uint_as_float(w[e]);
  }
};

template <int LN>
struct Tile {
  static constexpr int CH = 256 / LN;                 // channels of a workgroup
  static constexpr int TT = LN >= 4 ? 32 : 8 * LN;    // tokens of a tile
  static constexpr int PT = TT / LN;                  // (token, channel) pairs of a thread
  static constexpr int VW = PT < 4 ? PT : 4;          // of them adjacent channels
  static constexpr int NI = PT / VW;
  static constexpr int NP = 4 * LN;                   // states of a channel, padded
  static constexpr int NBC = (TT * 2 * NP + 255) / 256;  // B and C values that a thread loads
  static constexpr int YROW = CH + (LN > 1 ? 64 / LN : 0);  // LN token rows written at once: distinct banks
};

template <bool BF16, bool VEC, int LN, bool CARRY>
__global__ void __launch_bounds__(256) ssm_scan_tile_kernel(ScanSsmParams p) {
  using T = Tile<LN>;
  constexpr int CH = T::CH, TT = T::TT, VW = T::VW, NI = T::NI, NP = T::NP, NBC = T::NBC;
  __shared__ __align__(16) float2 s_dx[2][TT][CH];       // delta, delta x
  __shared__ __align__(16) float s_bc[2][TT][2 * NP];    // B, C
  __shared__ __align__(16) float s_y[CARRY ? 1 : 2][CARRY ? 1 : TT][T::YROW];

  const int tid = threadIdx.x, q = tid % LN, ch = tid / LN;
  const Sequence sq = find_sequence(p.seq, blockIdx.y, tid & 63);
  if (!sq.ok) return;
  const int seg = blockIdx.z, N = p.N;
  const int t_begin = seg * p.seg_len, t_end = min(t_begin + p.seg_len, sq.len);
  if (seg && t_begin >= sq.len) return;
  const int per_group = p.D / p.G, blocks = (per_group + CH - 1) / CH;
  const int g = blockIdx.x / blocks, c_base = (blockIdx.x % blocks) * CH;
  const long d0 = (long)g * per_group + c_base;      // first channel of the workgroup
  const int c_live = min(CH, per_group - c_base);    // channels it has
  const bool live = ch < c_live;
  const long d = d0 + (live ? ch : 0);
  const bool whole = (N & 3) == 0 && 4 * q < N;

  float A[4], h[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
  load_state4(p.A + d * N, q, N, whole, A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e;

  const long slot = (long)p.D * N;  // workspace: [units][nseg][D][N] states, then [units][nseg - 1][D] sums
  float *ws_h = p.workspace + (long)blockIdx.y * p.nseg * slot + d * N;
  float *ws_s = p.workspace + (long)p.seq.units * p.nseg * slot + (long)blockIdx.y * (p.nseg - 1) * p.D + d;
  if (CARRY || p.nseg == 1) {
    if (seg == 0) {
      if (p.seq.state_in) load_state4(p.seq.state_in + ((long)sq.row_in * p.D + d) * N, q, N, whole, h);
      if (CARRY && live) store_state4(ws_h, q, N, whole, h);
    }
    if (CARRY && t_end == sq.len) return;  // its state is the main pass's own
  } else {
    load_state4(ws_h + (seg ? slot : 0), q, N, whole, h);
    for (int k = 2; k <= seg; ++k) {
      float part[4];
      load_state4(ws_h + k * slot, q, N, whole, part);
      const float sum = ws_s[(long)(k - 1) * p.D];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(sum * A[i]), h[i], part[i]);
    }
  }

  // the loading layout: item i of a thread is VW adjacent channels of one token
  constexpr int ROW = CH / VW;
  const int l_c = (tid % ROW) * VW, l_t = tid / ROW;
  constexpr int L_STEP = 256 / ROW;
  const int l_live = min(VW, c_live - l_c);
  float bias[VW], skip[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    bias[e] = p.dt_bias && e < l_live ? p.dt_bias[d0 + l_c + e] : 0.f;
    skip[e] = p.skip && e < l_live ? p.skip[d0 + l_c + e] : 0.f;
  }
  using Raw = RawRow<BF16, VEC, VW>;
  Raw x[NI], dt[NI], z[NI], nx[NI], nz[NI];
  float bc[NBC];

  const auto request = [&](int t0) {  // the loads of the tile at t0
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int t = t0 + l_t + i * L_STEP;
      const int n = t < t_end ? l_live : 0;
      nx[i].load(p.x, sq.off + t, d0 + l_c, n);
      dt[i].load(p.dt, sq.off + t, d0 + l_c, n);
      if (!CARRY && p.z.base) nz[i].load(p.z, sq.off + t, d0 + l_c, n);
    }
#pragma unroll
    for (int i = 0; i < NBC; ++i) {
      const int e = tid + i * 256, n = e % NP, which = (e / NP) & 1, t = t0 + e / (2 * NP);
      bc[i] = 0.f;
      if (e < TT * 2 * NP && n < N && t < t_end && !(CARRY && which)) {
        const TokenArray &a = which ? p.Cm : p.Bm;
        bc[i] = load1<BF16>(a.base, (sq.off + t) * a.stride + (long)g * N + n);
      }
    }
  };
  const auto stage = [&](int t0, int buf) {  // delta, delta x, B and C of the requested tile
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool in = t0 + l_t + i * L_STEP < t_end;
      float2 *row = &s_dx[buf][l_t + i * L_STEP][l_c];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float raw = dt[i].get(e) + bias[e];
        // a token past the end leaves the state as it is
        const float delta = in ? (p.softplus ? softplus_f(raw) : raw) : 0.f;
        row[e] = make_float2(delta, delta * nx[i].get(e));
      }
    }
#pragma unroll
    for (int i = 0; i < NBC; ++i) {
      const int e = tid + i * 256;
      if (e < TT * 2 * NP) s_bc[buf][e / (2 * NP)][e % (2 * NP)] = bc[i];
    }
  };

  request(t_begin);
  stage(t_begin, 0);
#pragma unroll
  for (int i = 0; i < NI; ++i) { x[i] = nx[i]; z[i] = nz[i]; }
  __syncthreads();
  int buf = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += TT, buf ^= 1) {
    const bool more = t0 + TT < t_end;
    if (more) request(t0 + TT);
#pragma unroll 1
    for (int u0 = 0; u0 < TT; u0 += LN) {
      float part[LN];
#pragma unroll
      for (int u = 0; u < LN; ++u) {
        const float2 dx = s_dx[buf][u0 + u][ch];
        const float4 B = *reinterpret_cast<const float4 *>(&s_bc[buf][u0 + u][4 * q]);
        const float b[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(dx.x * A[i]), h[i], dx.y * b[i]);
        if constexpr (CARRY) {
          total += dx.x;
        } else {
          const float4 C = *reinterpret_cast<const float4 *>(&s_bc[buf][u0 + u][NP + 4 * q]);
          part[u] = fmaf(C.w, h[3], fmaf(C.z, h[2], fmaf(C.y, h[1], C.x * h[0])));
        }
      }
      if constexpr (!CARRY) s_y[buf][u0 + q][ch] = sum_spread<LN>(part, q);
    }
    if constexpr (!CARRY) {
      if (p.chunk_states && live && (t0 + TT) % kScanChunk == 0 && t0 + TT < sq.len)
        store_state4(p.chunk_states + (((long)blockIdx.y * p.n_chunks + (t0 + TT) / kScanChunk - 1) * p.D + d) * N, q, N, whole, h);
    }
    if (more) stage(t0 + TT, buf ^ 1);
    __syncthreads();
    if constexpr (!CARRY) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int t = l_t + i * L_STEP;
        float y[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          y[e] = fmaf(skip[e], x[i].get(e), s_y[buf][t][l_c + e]);
          if (p.z.base) {
            const float zv = z[i].get(e);
            y[e] *= zv * sigmoid_f(zv);
          }
        }
        if (t0 + t < t_end) {
          const long at = (sq.off + t0 + t) * p.D + d0 + l_c;
          if constexpr (VEC) {
            if (l_live > 0) {
              if (p.y_bf16) storev<true, VW>(p.y, at, y);
              else storev<false, VW>(p.y, at, y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < VW; ++e)
              if (e < l_live) store1(p.y, at + e, p.y_bf16, y[e]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) { x[i] = nx[i]; z[i] = nz[i]; }
  }

  if constexpr (CARRY) {
    if (live) {
      store_state4(ws_h + (seg + 1) * slot, q, N, whole, h);
      if (q == 0) ws_s[(long)seg * p.D] = total;
    }
  } else if (live && t_end == sq.len && p.seq.state_out && !(sq.len == 0 && p.seq.state_out == p.seq.state_in)) {
    store_state4(p.seq.state_out + ((long)sq.row_out * p.D + d) * N, q, N, whole, h);
  }
}

template <bool BF16, int LN>
hipError_t go(const ScanSsmParams &p, hipStream_t s) {
  constexpr int CH = 256 / LN, VW = Tile<LN>::VW;
  const int per_group = p.D / p.G, blocks = p.G * ((per_group + CH - 1) / CH);
  if (p.seq.T <= kScanShort) {
    hipLaunchKernelGGL((ssm_scan_short_kernel<BF16, LN>), dim3(blocks, p.seq.units), dim3(256), 0, s, p);
    return hipGetLastError();
  }
  const auto fits = [&](const TokenArray &a) {
    return !a.base || (a.stride % VW == 0 && reinterpret_cast<uintptr_t>(a.base) % (VW * (BF16 ? 2 : 4)) == 0);
  };
  const bool vec = per_group % VW == 0 && fits(p.x) && fits(p.dt) && fits(p.z);
  if (p.nseg > 1) {
    const dim3 grid(blocks, p.seq.units, p.nseg - 1);
    if (vec) hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, true, LN, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, false, LN, true>), grid, dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(blocks, p.seq.units, p.nseg);
  if (vec) hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, true, LN, false>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, false, LN, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_states(const ScanSsmParams &p, hipStream_t s) {
  switch (lanes_of(p.N)) {
    case 1: return go<BF16, 1>(p, s);
    case 2: return go<BF16, 2>(p, s);
    case 4: return go<BF16, 4>(p, s);
    case 8: return go<BF16, 8>(p, s);
    default: return go<BF16, 16>(p, s);
  }
}

}  // namespace

// Segments of a call: one where its workgroups fill the chip, else as many as fill it.
int scan_segments(int units, int T, int D, int N, int G, int *seg_len) {
  const int CH = 256 / lanes_of(N);
  const long groups = (long)units * G * ((D / G + CH - 1) / CH);
  *seg_len = T > 0 ? T : 1;
  if (T <= kScanSplit || groups >= 192 || groups == 0) return 1;
  const int want = (int)(512 / groups) < 32 ? (int)(512 / groups) : 32;
  int len = (T + want - 1) / want;
  len = (len + kScanSplit - 1) / kScanSplit * kScanSplit;
  const int n = (T + len - 1) / len;
  if (n < 3) return 1;  // the carry pass costs about three quarters of the main one
  *seg_len = len;
  return n;
}

hipError_t launch_ssm_scan(const ScanSsmParams &p, bool bf16, hipStream_t s) {
  return bf16 ? by_states<true>(p, s) : by_states<false>(p, s);
}

}  // namespace wkv
