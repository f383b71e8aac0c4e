// The selective state space scan.  Per channel d and state n, with delta = softplus(dt + dt_bias):
//   h[n] <- e^(delta A[d][n]) h[n] + delta x B[n],   y = sum_n C[n] h[n] + skip[d] x,  y *= z sigmoid(z)
// States and sums are fp32; a bf16 y is the fp32 result rounded to nearest even.
//
// Every (channel, state) has a decay of its own, so nothing here is a matrix product: a token costs
// D N exponentials (a quarter-rate instruction) and 4 D N multiplies and fused multiply-adds on the
// vector ALUs, against 8 D bytes of bf16 traffic.  With N = 16 the ALUs bound it.
#include "ssm_tile.hpp"

namespace wkv {
namespace {

// Few tokens (single-token steps): LN adjacent lanes share a channel, four states each, and walk the
// tokens one by one.  Bound by the states' way in and out, one coalesced load and store of 16 bytes a
// lane, and by the latencies in a row: so every load goes through a window, which answers what is not
// there with zeros, and none waits behind another's branch.  A token's values and the state leave
// together; the state, the longest way, is asked for last and waited for last.  A step of 64 slots,
// D = 2048, N = 16: 8.9 us, of which the bytes are 3.6, an empty launch 2.9 and finding the slots 1.4
// (9.4 us with loads in branches, each waited for where its paths join).
template <bool BF16, bool WHOLE>
struct ShortToken {
  static constexpr int EL = BF16 ? 2 : 4;
  RawRow<BF16, false, 1> x, dt, z;
  RawRow<BF16, WHOLE, 4> B, C;
  // of the token `row`, if `rows` is 1; col: of the lane's channel and states, in elements
  __device__ __forceinline__ void load(const ScanSsmParams &p, long row, int rows, long d0, int c_live, long bc, const uint32_t (&c_col)[1],
                                       const uint32_t (&n_col)[WHOLE ? 1 : 4]) {
    x.load(window<EL>(p.x.base, p.x.stride, row, rows, d0, c_live), 0, c_col);
    dt.load(window<EL>(p.dt.base, p.dt.stride, row, rows, d0, c_live), 0, c_col);
    z.load(window<EL>(p.z.base, p.z.stride, row, p.z.base ? rows : 0, d0, c_live), 0, c_col);
    B.load(window<EL>(p.Bm.base, p.Bm.stride, row, rows, bc, p.N), 0, n_col);
    C.load(window<EL>(p.Cm.base, p.Cm.stride, row, rows, bc, p.N), 0, n_col);
  }
};

// WHOLE: N divides by 4, so that a lane's four states are there or not as one.
template <bool BF16, int LN, bool WHOLE>
__global__ void __launch_bounds__(256) ssm_scan_short_kernel(ScanSsmParams p) {
  constexpr int CH = 256 / LN, EL = BF16 ? 2 : 4, NC = WHOLE ? 1 : 4;  // CH: channels of a workgroup
  const int lane = threadIdx.x & 63, q = threadIdx.x % LN, ch = threadIdx.x / LN, N = p.N;
  const int per_group = p.D / p.G, blocks = (per_group + CH - 1) / CH;
  const int g = blockIdx.x / blocks, c_base = (blockIdx.x % blocks) * CH, c_live = min(CH, per_group - c_base);
  const bool live = ch < c_live;
  const long d0 = (long)g * per_group + c_base;
  uint32_t n_col[NC], s_col[NC];  // of B and C, and of fp32 rows [D, N] from d0 on
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t out = 4 * q + i < N ? 0u : kOutside;
    n_col[i] = (4 * q + i) * EL + out;
    s_col[i] = (ch * N + 4 * q + i) * 4 + (live ? out : kOutside);
  }
  const uint32_t c_col[1] = {ch * EL + (live ? 0u : kOutside)}, f_col[1] = {ch * 4 + (live ? 0u : kOutside)};
  const long slot = (long)p.D * N;
  RawRow<false, false, 1> raw_bias, raw_skip;
  RawRow<false, WHOLE, 4> raw_A, raw_h;
  raw_A.load(window<4>(p.A, slot, 0, 1, d0 * N, c_live * N), 0, s_col);
  raw_bias.load(window<4>(p.dt_bias, p.D, 0, p.dt_bias ? 1 : 0, d0, c_live), 0, f_col);
  raw_skip.load(window<4>(p.skip, p.D, 0, p.skip ? 1 : 0, d0, c_live), 0, f_col);
  const Sequence sq = find_sequence(p.seq, blockIdx.y, lane);
  if (!sq.ok) return;
  ShortToken<BF16, WHOLE> now, next;
  now.load(p, sq.off, sq.len > 0, d0, c_live, (long)g * N, c_col, n_col);
  raw_h.load(window<4>(p.seq.state_in, slot, sq.row_in, p.seq.state_in ? 1 : 0, d0 * N, c_live * N), 0, s_col);
  float A[4], h[4];
  const float bias = raw_bias.get(0), skip = raw_skip.get(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = decay_rate(raw_A.get(i));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = raw_h.get(i);
  for (int t = 0; t < sq.len; ++t) {
    const long r = sq.off + t;
    next.load(p, r + 1, t + 1 < sq.len, d0, c_live, (long)g * N, c_col, n_col);
    const float x = now.x.get(0), raw = now.dt.get(0) + bias, delta = p.softplus ? softplus_f(raw) : raw, dx = delta * x;
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(__builtin_amdgcn_exp2f(delta * A[i]), h[i], dx * now.B.get(i));
      part = fmaf(now.C.get(i), h[i], part);
    }
    float y = fmaf(skip, x, sum_all<LN>(part));
    if (p.z.base) y *= now.z.get(0) * sigmoid_f(now.z.get(0));
    if (live && q == 0) store1(p.y, r * p.D + d0 + ch, p.y_bf16, y);
    now = next;
  }
  if (live && p.seq.state_out && !(sq.len == 0 && p.seq.state_out == p.seq.state_in))
    store_state4(p.seq.state_out + sq.row_out * slot + (d0 + ch) * N, q, N, WHOLE && 4 * q < N, h);
}

// ------------------------------------------------------------------------------------------------
// Long sequences.  A workgroup owns 256 / LN channels and walks its segment in tiles of TT tokens,
// with four waves for each of two roles and one barrier per tile:
//   - the staging waves load a tile's rows (one tile ahead), form what a token and channel need once
//     - delta, delta x - and the widened B and C rows into LDS, and finish the results of the tile
//     before (skip, gate, rounding) for row-wide stores;
//   - the scan waves walk the channels: four states of a channel per lane, LN lanes a channel.  The
//     matrix unit forms the outer product: v_mfma_f32_4x4x1 takes, per block of four lanes, four B
//     values and four delta x, so that a state costs a lane a multiply, an exponential and two
//     multiply-adds.  (fp32 throughout; y on the matrix unit as well was slower: 367 us, not 314.)
//     The partial sums over n are spread over the LN lanes, LN tokens at a time.
// [8, 4096, 2048], N = 16, bf16: 280 us.  A scan wave's token is 20 vector instructions, four of them
// exponentials of two turns (179 us in all at 2.23 GHz), a staging wave's token and channel 33 turns (61 us
// more); the vector ALUs are busy for 0.75 of the time, the bytes would take 109 us.  Without the two
// roles, one set of waves doing both in turn: 421 us.
//
// Few rows: the sequence is cut into nseg segments.  The carry pass runs all but the last from a
// state of zero and leaves each one's final state and its sum of delta; as the decay over a segment
// is e^(A sum delta), the main pass folds the earlier segments' states into its own start.

template <int LN>
struct Tile {
  static constexpr int CH = 256 / LN;                 // channels of a workgroup
  static constexpr int TT = LN >= 4 ? 32 : 8 * LN;    // tokens of a tile
  static constexpr int PT = TT / LN;                  // (token, channel) pairs of a thread
  static constexpr int VW = PT < 4 ? PT : 4;          // of them adjacent channels
  static constexpr int NI = PT / VW;
  static constexpr int NP = 4 * LN;                   // states of a channel, padded
  static constexpr int NB = (TT * NP + 255) / 256;    // B (and C) values that a thread loads
  static constexpr int YROW = CH + (LN > 1 ? 64 / LN : 0);  // LN token rows written at once: distinct banks
};

// What four tokens need of LDS.
template <int LN, bool OUT>
struct Quad {
  float2 dx[4];
  float b[4];
  float4 c[4];
  template <int CH, int NP>
  __device__ __forceinline__ void load(const float2 (*s_dx)[CH], const float (*s_b)[NP], const float (*s_c)[NP], int t, int ch, int q, int j) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      dx[u] = s_dx[t + u][ch];
      b[u] = s_b[t + u][4 * q + j];
      if constexpr (OUT) c[u] = *reinterpret_cast<const float4 *>(&s_c[t + u][4 * q]);
    }
  }
  // One token: the states' update and the lane's part of y.
  __device__ __forceinline__ float step(int u, const float (&A)[4], f32x4 &h) const {
    const f32x4 xb = __builtin_amdgcn_mfma_f32_4x4x1f32(b[u], dx[u].y, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(dx[u].x * A[i]), h[i], xb[i]);
    if constexpr (!OUT) return 0.f;
    else return fmaf(c[u].w, h[3], fmaf(c[u].z, h[2], fmaf(c[u].y, h[1], c[u].x * h[0])));
  }
};

// CARRY: the carry pass.  OUT: whether y is formed; the main pass without it only leaves the chunk states.
template <bool BF16, Rows ROWS, int LN, bool CARRY, bool OUT>
__global__ void __launch_bounds__(512, LN <= 4 ? 4 : 2) ssm_scan_tile_kernel(ScanSsmParams p) {
  using T = Tile<LN>;
  constexpr int CH = T::CH, TT = T::TT, VW = T::VW, NI = T::NI, NP = T::NP, NB = T::NB;
  __shared__ __align__(16) float2 s_dx[2][TT][CH];  // delta, delta x
  __shared__ __align__(16) float s_b[2][TT][NP];
  __shared__ __align__(16) float s_c[OUT ? 2 : 1][OUT ? TT : 1][NP];
  __shared__ __align__(16) float s_y[OUT ? 2 : 1][OUT ? TT : 1][T::YROW];

  const int tid = threadIdx.x & 255;
  const bool scanning = uniform((int)(threadIdx.x >> 8)) == 0;
  const Sequence sq = find_sequence(p.seq, slot_by_length(p.seq, blockIdx.y, tid & 63), tid & 63);
  if (!sq.ok) return;
  const int seg = blockIdx.z, N = p.N;
  const int t_begin = seg * p.seg_len, t_end = min(t_begin + p.seg_len, sq.len);
  if (seg && t_begin >= sq.len) return;
  const int per_group = p.D / p.G, blocks = (per_group + CH - 1) / CH;
  const int g = blockIdx.x / blocks, c_base = (blockIdx.x % blocks) * CH;
  const long d0 = (long)g * per_group + c_base;      // first channel of the workgroup
  const int c_live = min(CH, per_group - c_base);    // channels it has
  const int tiles = (t_end - t_begin + TT - 1) / TT;

  if (scanning) {
    const int lane = tid & 63, j = lane & 3, q = (lane >> 2) % LN;
    const int ch = (tid >> 6) * (64 / LN) + (lane >> 2) / LN * 4 + j;
    const bool live = ch < c_live;
    const long d = d0 + (live ? ch : 0);
    const bool whole = (N & 3) == 0 && 4 * q < N;
    float A[4], h0[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
    load_decay4(p.A + d * N, q, N, whole, A);

    const long slot = (long)p.D * N;  // workspace: [units][nseg][D][N] states, then [units][nseg - 1][D] sums
    float *ws_h = p.workspace + (long)blockIdx.y * p.nseg * slot + d * N;
    float *ws_s = p.workspace + (long)p.seq.units * p.nseg * slot + (long)blockIdx.y * (p.nseg - 1) * p.D + d;
    if (CARRY || p.nseg == 1) {
      if (seg == 0) {
        if (p.seq.state_in) load_state4(p.seq.state_in + ((long)sq.row_in * p.D + d) * N, q, N, whole, h0);
        if (CARRY && live) store_state4(ws_h, q, N, whole, h0);
      }
    } else {
      load_state4(ws_h + (seg ? slot : 0), q, N, whole, h0);
      for (int k = 2; k <= seg; ++k) {
        float part[4];
        load_state4(ws_h + k * slot, q, N, whole, part);
        const float sum = ws_s[(long)(k - 1) * p.D];
#pragma unroll
        for (int i = 0; i < 4; ++i) h0[i] = fmaf(__builtin_amdgcn_exp2f(sum * A[i]), h0[i], part[i]);
      }
    }
    if (CARRY && t_end == sq.len) return;  // its state is the main pass's own (the staging waves leave too)
    // the states have arrived before the loop, which then waits for LDS only
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(h0[i]), "+v"(A[i]));
    f32x4 h = {h0[0], h0[1], h0[2], h0[3]};
    if (tiles > 0) __syncthreads();
    for (int k = 0; k < tiles; ++k) {
      const int buf = k & 1, cbuf = OUT ? buf : 0;
      constexpr int S = LN > 8 ? LN : 8;  // LDS reads run four tokens ahead of the arithmetic
      Quad<LN, OUT> quad[2];
      quad[0].load(s_dx[buf], s_b[buf], s_c[cbuf], 0, ch, q, j);
#pragma unroll 1
      for (int u0 = 0; u0 < TT; u0 += S) {
        float part[LN > 4 ? LN : 4];
#pragma unroll
        for (int v = 0; v < S; v += 4) {
          const int next = u0 + v + 4;
          if (v + 4 < S || next < TT) quad[(v / 4 + 1) & 1].load(s_dx[buf], s_b[buf], s_c[cbuf], next, ch, q, j);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float y = quad[(v / 4) & 1].step(u, A, h);
            if constexpr (CARRY) total += quad[(v / 4) & 1].dx[u].x;
            if constexpr (OUT) part[(LN > 4 ? v : 0) + u] = y;
          }
          if constexpr (OUT) {
            if constexpr (LN <= 4) {
#pragma unroll
              for (int w = 0; w < 4; w += LN) {
                float some[LN];
#pragma unroll
                for (int i = 0; i < LN; ++i) some[i] = part[w + i];
                s_y[buf][u0 + v + w + q][ch] = spread4<LN>(some, q);
              }
            } else if (v + 4 == S) {
              float some[LN];
#pragma unroll
              for (int i = 0; i < LN; ++i) some[i] = part[i];
              s_y[buf][u0 + v + 4 - LN + q][ch] = spread4<LN>(some, q);
            }
          }
        }
        if constexpr (!CARRY) {
          const int t = t_begin + k * TT + u0 + S;
          if (p.chunk_states && live && t % kScanChunk == 0 && t < sq.len) {
            const float at_t[4] = {h[0], h[1], h[2], h[3]};
            store_state4(p.chunk_states + (((long)blockIdx.y * p.n_chunks + t / kScanChunk - 1) * p.D + d) * N, q, N, whole, at_t);
          }
        }
      }
      __syncthreads();
    }
    const float out[4] = {h[0], h[1], h[2], h[3]};
    if constexpr (CARRY) {
      if (live) {
        store_state4(ws_h + (seg + 1) * slot, q, N, whole, out);
        if (q == 0) ws_s[(long)seg * p.D] = total;
      }
    } else if (live && t_end == sq.len && p.seq.state_out && !(sq.len == 0 && p.seq.state_out == p.seq.state_in)) {
      store_state4(p.seq.state_out + ((long)sq.row_out * p.D + d) * N, q, N, whole, out);
    }
    return;
  }

  // Staging waves.  Item i of a thread is VW adjacent channels of one token.
  if (tiles == 0 || (CARRY && t_end == sq.len)) return;
  constexpr int ROW = CH / VW, L_STEP = 256 / ROW, EL = BF16 ? 2 : 4;
  constexpr bool VEC = ROWS != Rows::kSingle;
  int l_c = (tid % ROW) * VW;
  const int l_t = tid / ROW;
  if constexpr (ROWS == Rows::kOverlap) l_c = min(l_c, c_live - VW);
  float bias[VW], skip[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const bool in = l_c + e < c_live;
    bias[e] = p.dt_bias && in ? p.dt_bias[d0 + l_c + e] : 0.f;
    skip[e] = p.skip && in ? p.skip[d0 + l_c + e] : 0.f;
  }
  const auto columns = [&](int el, uint32_t (&col)[VEC ? 1 : VW]) {
#pragma unroll
    for (int e = 0; e < (VEC ? 1 : VW); ++e) col[e] = (l_c + e) * el + (l_c + e < c_live ? 0u : kOutside);
  };
  uint32_t col[VEC ? 1 : VW];
  columns(EL, col);
  using Raw = RawRow<BF16, VEC, VW>;
  // A tile's x and z are needed until it is finished, when the third tile after it is requested: three
  // sets, taken in turn.  (dt, B and C are staged before the next request.)
  Raw x[3][NI], z[3][NI], dt[NI];
  uint32_t bb[NB] = {}, cc[NB] = {};
  const bool gate = OUT && p.z.base;
  const int b_n = tid % NP, b_t = tid / NP;  // B and C: state and token of this thread's first value
  constexpr int B_STEP = 256 / NP;
  const bool b_in = TT * NP >= 256 || b_t < TT;
  const uint32_t b_col = b_n * EL + (b_n < N && b_in ? 0u : kOutside);

  const auto request = [&](int t0, auto of) {  // the loads of the tile at t0
    constexpr int set = decltype(of)::value;
    const long row = sq.off + t0;
    const int rows = min(TT, t_end - t0);
    const auto wx = window<EL>(p.x.base, p.x.stride, row, rows, d0, c_live);
    const auto wd = window<EL>(p.dt.base, p.dt.stride, row, rows, d0, c_live);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t t = l_t + i * L_STEP;
      x[set][i].load(wx, t * (uint32_t)p.x.stride * EL, col);
      dt[i].load(wd, t * (uint32_t)p.dt.stride * EL, col);
    }
    if (gate) {
      const auto wz = window<EL>(p.z.base, p.z.stride, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) z[set][i].load(wz, (l_t + i * L_STEP) * (uint32_t)p.z.stride * EL, col);
    }
    const auto wb = window<EL>(p.Bm.base, p.Bm.stride, row, rows, (long)g * N, N);
    const auto wc = window<EL>(p.Cm.base, p.Cm.stride, row, rows, (long)g * N, N);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t t = b_t + i * B_STEP;
      const int ob = (int)(t * (uint32_t)p.Bm.stride * EL + b_col), oc = (int)(t * (uint32_t)p.Cm.stride * EL + b_col);
      if constexpr (BF16) {
        bb[i] = __builtin_amdgcn_raw_buffer_load_b16(wb, ob, 0, 0);
        if constexpr (OUT) cc[i] = __builtin_amdgcn_raw_buffer_load_b16(wc, oc, 0, 0);
      } else {
        bb[i] = __builtin_amdgcn_raw_buffer_load_b32(wb, ob, 0, 0);
        if constexpr (OUT) cc[i] = __builtin_amdgcn_raw_buffer_load_b32(wc, oc, 0, 0);
      }
    }
  };
  const auto stage = [&](int t0, int buf, auto of) {  // delta, delta x, B and C of the requested tile
    constexpr int set = decltype(of)::value;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      dt[i].arrive(); x[set][i].arrive();
      if (gate) z[set][i].arrive();
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(bb[i]), "+v"(cc[i]));
    float delta[NI][VW];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VW; ++e) delta[i][e] = dt[i].get(e) + bias[e];
    if (p.softplus) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) delta[i][e] = softplus_f(delta[i][e]);
    }
    if (t0 + TT > t_end) {  // tokens past the end leave the state as it is
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e)
          if (t0 + l_t + i * L_STEP >= t_end) delta[i][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float2 *row = &s_dx[buf][l_t + i * L_STEP][l_c];
#pragma unroll
      for (int e = 0; e < VW; ++e) row[e] = make_float2(delta[i][e], delta[i][e] * x[set][i].get(e));
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int t = (b_t + i * B_STEP) & (TT - 1);
      if (b_in) {
        s_b[buf][t][b_n] = BF16 ? bf16_lo(bb[i]) : __uint_as_float(bb[i]);
        if constexpr (OUT) s_c[buf][t][b_n] = BF16 ? bf16_lo(cc[i]) : __uint_as_float(cc[i]);
      }
    }
  };
  const auto finish = [&](int t0, int buf, auto of) {  // the results of the tile at t0, from the sums of its scan
    constexpr int set = decltype(of)::value;
    float y[NI][VW];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < VW; ++e) y[i][e] = fmaf(skip[e], x[set][i].get(e), s_y[buf][l_t + i * L_STEP][l_c + e]);
    if (gate) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) y[i][e] *= z[set][i].get(e) * sigmoid_f(z[set][i].get(e));
    }
    const long row = sq.off + t0;
    const int rows = min(TT, t_end - t0);
    uint32_t to[VEC ? 1 : VW];
    if (p.y_bf16) {
      columns(2, to);
      const auto wy = window<2>(p.y, p.D, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) store_row<true, VEC, VW>(wy, (l_t + i * L_STEP) * (uint32_t)p.D * 2, to, y[i]);
    } else {
      columns(4, to);
      const auto wy = window<4>(p.y, p.D, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) store_row<false, VEC, VW>(wy, (l_t + i * L_STEP) * (uint32_t)p.D * 4, to, y[i]);
    }
  };

  if constexpr (ROWS == Rows::kOverlap) {  // the columns past the block's channels, which nothing else writes
    for (int e = tid; e < 2 * TT * (CH - c_live); e += 256) {
      const int row = e / (CH - c_live), c = c_live + e % (CH - c_live);
      s_dx[row & 1][row >> 1][c] = make_float2(0.f, 0.f);
    }
  }
  request(t_begin, Set<0>{});
  stage(t_begin, 0, Set<0>{});
  if (tiles > 1) request(t_begin + TT, Set<1>{});
  __syncthreads();
  const auto step = [&](int k, auto before, auto after) {  // while tile k is scanned; the sets of the tiles beside it
    const int t0 = t_begin + k * TT, other = (k + 1) & 1;
    if constexpr (OUT) {
      if (k) finish(t0 - TT, other, before);
    }
    if (k + 1 < tiles) stage(t0 + TT, other, after);
    if (k + 2 < tiles) request(t0 + 2 * TT, before);
    __syncthreads();
  };
  for (int k = 0; k < tiles; k += 3) {
    step(k, Set<2>{}, Set<1>{});
    if (k + 1 < tiles) step(k + 1, Set<0>{}, Set<2>{});
    if (k + 2 < tiles) step(k + 2, Set<1>{}, Set<0>{});
  }
  if constexpr (OUT) {
    const int k = tiles - 1;
    if (k % 3 == 0) finish(t_begin + k * TT, k & 1, Set<0>{});
    else if (k % 3 == 1) finish(t_begin + k * TT, k & 1, Set<1>{});
    else finish(t_begin + k * TT, k & 1, Set<2>{});
  }
}

template <bool BF16, int LN, bool CARRY, bool OUT>
void go_tiles(const ScanSsmParams &p, dim3 grid, Rows rows, hipStream_t s) {
  if (rows == Rows::kWhole) hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, Rows::kWhole, LN, CARRY, OUT>), grid, dim3(512), 0, s, p);
  else if (rows == Rows::kOverlap) hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, Rows::kOverlap, LN, CARRY, OUT>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((ssm_scan_tile_kernel<BF16, Rows::kSingle, LN, CARRY, OUT>), grid, dim3(512), 0, s, p);
}

template <bool BF16, int LN>
hipError_t go(const ScanSsmParams &p, hipStream_t s) {
  constexpr int CH = 256 / LN, VW = Tile<LN>::VW;
  const int per_group = p.D / p.G, blocks = p.G * ((per_group + CH - 1) / CH);
  if (p.seq.T <= kScanShort && p.y) {
    if (p.N % 4 == 0) hipLaunchKernelGGL((ssm_scan_short_kernel<BF16, LN, true>), dim3(blocks, p.seq.units), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((ssm_scan_short_kernel<BF16, LN, false>), dim3(blocks, p.seq.units), dim3(256), 0, s, p);
    return hipGetLastError();
  }
  const Rows rows = rows_of<CH, VW>(per_group);
  if (p.nseg > 1) {
    go_tiles<BF16, LN, true, false>(p, dim3(blocks, p.seq.units, p.nseg - 1), rows, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(blocks, p.seq.units, p.nseg);
  if (p.y) go_tiles<BF16, LN, false, true>(p, grid, rows, s);
  else go_tiles<BF16, LN, false, false>(p, grid, rows, s);
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

// Segments of a call, by a model of its time in tokens of one workgroup walking alone.  A compute
// unit that has k workgroups takes `shared` k times as long for a token of each (two at once overlap a
// little; measured 0.88 forward, and 1 backward, where one fills the unit); the carry pass costs the
// share `carry` of the main one, and a workgroup's start as well as a launch as much as `start` tokens.
// groups: the workgroups of one segment of all rows.  Measured around its choices: [1, 32765, 1536] 327 us
// in the 21 that it takes, 388 in 10, 420 in 16, 318 in 32; [8, 4096, 2048] 280 uncut, 342 in two; 48
// mixed slots 67 uncut, 105 in two; training [2, 777, 1030] 116, 199 with its backward pass uncut.
int best_segments(long groups, int T, int step, double shared, double carry, int start, int *seg_len) {
  *seg_len = T > 0 ? T : 1;
  if (T <= kScanSplit || groups < 1) return 1;
  const auto walk = [&](long g, int len) {
    const long k = (g + 255) / 256;
    return k <= 1 ? double(len + start) : shared * k * len + (k + 1) / 2 * start;  // two start at once
  };
  int best = 1;
  double least = walk(groups, T);
  for (int want = 2; want <= 32; ++want) {
    int len = (T + want - 1) / want;
    len = (len + step - 1) / step * step;
    const int n = (T + len - 1) / len;
    if (n < 2) continue;
    const double t = walk(groups * n, len) + carry * walk(groups * (n - 1), len) + start;
    if (t < 0.95 * least) {
      least = t;
      best = n;
      *seg_len = len;
    }
  }
  return best;
}

// total / T stands for the full-length rows of a call whose slots differ.
int scan_segments(int units, int T, long total, int D, int N, int G, int *seg_len) {
  const int CH = 256 / lanes_of(N);
  if (T > total) T = (int)total;  // no slot has more tokens than the call, whatever the host's bound
  const long full = T > 0 && total / T + 1 < units ? total / T + 1 : units;
  return best_segments(full * G * ((D / G + CH - 1) / CH), T, 32, 0.88, 0.7, 64, seg_len);
}

hipError_t launch_ssm_scan(const ScanSsmParams &p, bool bf16, hipStream_t s) {
  return bf16 ? by_states<true>(p, s) : by_states<false>(p, s);
}

}  // namespace wkv
