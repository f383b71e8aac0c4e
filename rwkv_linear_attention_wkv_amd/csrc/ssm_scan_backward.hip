// Backward pass of the selective scan.  With c_t = dy_t z_t sigmoid(z_t) (the gradient of the ungated
// output) and G the gradient of the state, walked from the last token to the first:
//   G <- G + C_t c_t                                     (G starts as the final state's gradient)
//   dB_t = sum_d G delta x,  dC_t = sum_d h_t c_t         (over the channels of a group)
//   dx_t = delta sum_n G B + skip c_t
//   G <- a_t G,  a_t = e^(delta A);   q = G h_(t-1)
//   d delta = x sum_n G_before B + sum_n A q,   dA = sum_t delta q,   ddt = d delta softplus'
//   dz_t = dy_t y_t silu'(z_t),  y_t = sum_n C h_t + skip x_t;   d skip = sum c x
// The states h are needed in reverse order.  The forward pass leaves them every 16 tokens; a tile of
// 16 tokens is walked forward from there with its states and decays kept in registers, then back.
//
// As in the forward kernel, four staging waves prepare a tile and finish the one before it, and four
// scan waves hold four states of a channel per lane and get their outer products (delta x B, and C c)
// from the matrix unit.  Sums over n spread over the LN lanes of a channel; sums over channels take
// 16 steps for the eight values of a token (halvings by lane swaps), the rest in LDS and, over blocks
// of channels, in a second kernel: every sum has one order.  About 67 vector instructions and 4
// exponentials a token for 4 states of 16 channels: the ALUs bound it, as they do the forward pass.
// [8, 2048, 2048], N = 16, bf16: 413 to 445 us, as the clock allows, with the ALUs busy for 0.79 of it; the
// sums that are left 13 us.  Reading the next tokens from LDS four ahead was slower (499 us, not 479 at
// that stage), so was a higher priority for the staging waves (10 %).
#include "ssm_tile.hpp"

namespace wkv {
namespace {

constexpr int TT = kScanChunk;  // tokens of a tile

template <int LN>
struct BTile {
  static constexpr int CH = 256 / LN;
  static constexpr int PT = TT / LN;                 // (token, channel) pairs of a thread
  static constexpr int VW = PT < 4 ? PT : 4;
  static constexpr int NI = PT / VW;
  static constexpr int NP = 4 * LN;
  static constexpr int NB = (TT * NP + 255) / 256;
  static constexpr int YROW = CH + 64 / LN;
};

// Sums of v[0 .. 7] (dB of four states, dC of four) over the channels of a wave: the lanes that
// differ from this one in the bits above the LN lanes of a channel (each swap or rotation joins two
// lanes and halves the values) and in the two lowest bits.  Returns the values left in r and the
// place of the first among the eight; lanes may hold copies of the same value.
template <int LN>
__device__ __forceinline__ void sum_channels(const float (&v)[8], int lane, float (&r)[LN == 16 ? 2 : 1], int &place) {
  constexpr int B = LN == 2 ? 3 : LN == 4 ? 2 : LN == 8 ? 1 : 0;  // lane bits above a channel's lanes
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = v[i];
  place = 0;
  int n = 8;
#pragma unroll
  for (int s = 0; s < B; ++s) {
    const int half = n / 2;
    if (s < 2) {
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const uint32_t a = __float_as_uint(w[i]), b = __float_as_uint(w[i + half]);
        const auto x = s == 0 ? __builtin_amdgcn_permlane32_swap(a, b, false, false) : __builtin_amdgcn_permlane16_swap(a, b, false, false);
        w[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
      }
      place += (lane >> (5 - s) & 1) * half;
    } else {
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float lo = w[i] + dpp<0x128>(w[i]), hi = w[i + half] + dpp<0x128>(w[i + half]);
        w[i] = lane & 8 ? hi : lo;
      }
      place += (lane >> 3 & 1) * half;
    }
    n = half;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int half = n / 2;
    if (half) {
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float lo = w[i] + (s ? dpp<kXor2>(w[i]) : dpp<kXor1>(w[i]));
        const float hi = w[i + half] + (s ? dpp<kXor2>(w[i + half]) : dpp<kXor1>(w[i + half]));
        w[i] = lane >> s & 1 ? hi : lo;
      }
      place += (lane >> s & 1) * half;
      n = half;
    } else {
      w[0] += s ? dpp<kXor2>(w[0]) : dpp<kXor1>(w[0]);
    }
  }
#pragma unroll
  for (int i = 0; i < (LN == 16 ? 2 : 1); ++i) r[i] = w[i];
}

// CARRY: only the gradient of the state at the start of each segment but the first, from a gradient
// of zero at its end, and the segment's sum of delta.
template <bool BF16, Rows ROWS, int LN, bool CARRY>
__global__ void __launch_bounds__(512, 2) ssm_scan_backward_kernel(ScanBackwardParams p) {
  using T = BTile<LN>;
  constexpr int CH = T::CH, VW = T::VW, NI = T::NI, NP = T::NP, NB = T::NB;
  __shared__ __align__(16) float2 s_dx[2][TT][CH];  // delta, delta x
  __shared__ __align__(16) float s_dc[2][TT][CH];   // c
  __shared__ __align__(16) float s_b[2][CARRY ? 1 : TT][NP];
  __shared__ __align__(16) float s_c[2][TT][NP];
  __shared__ __align__(16) float s_out[CARRY ? 1 : 2][3][CARRY ? 1 : TT][T::YROW];  // sums over n: C h, G B, A q
  __shared__ __align__(16) float s_bc[CARRY ? 1 : 2][4][CARRY ? 1 : TT][2 * NP];    // sums over a wave's channels

  const ScanSsmParams &f = p.f;
  const int tid = threadIdx.x & 255;
  const bool scanning = uniform((int)(threadIdx.x >> 8)) == 0;
  const int unit = blockIdx.y, N = f.N, D = f.D;
  const int seg = CARRY ? blockIdx.z + 1 : blockIdx.z;
  const int t_begin = seg * p.seg_len, t_end = min(t_begin + p.seg_len, f.seq.T);
  const int per_group = D / f.G, blocks = (per_group + CH - 1) / CH;
  const int g = blockIdx.x / blocks, block = blockIdx.x % blocks, c_base = block * CH;
  const long d0 = (long)g * per_group + c_base;
  const int c_live = min(CH, per_group - c_base);
  const int tiles = (t_end - t_begin + TT - 1) / TT;  // at least one
  float *shares = p.part + ((long)unit * p.nseg + seg) * D * (N + 2);  // of dA, then d_skip and d_bias
  const Sequence sq = find_sequence(f.seq, unit, tid & 63);
  if (!sq.ok) {  // a rejected row has no share in the parameters' gradients
    if (!CARRY) {
      for (long i = threadIdx.x; i < (long)c_live * N; i += 512) shares[d0 * N + i] = 0.f;
      for (int i = threadIdx.x; i < c_live; i += 512) shares[(long)D * N + d0 + i] = shares[(long)D * N + D + d0 + i] = 0.f;
    }
    return;
  }

  if (scanning) {
    const int lane = tid & 63, wave = tid >> 6, j = lane & 3, q = (lane >> 2) % LN;
    const int ch = wave * (64 / LN) + (lane >> 2) / LN * 4 + j;
    const bool live = ch < c_live;
    const long d = d0 + (live ? ch : 0);
    const bool whole = (N & 3) == 0 && 4 * q < N;
    float A[4], g0[4] = {0.f, 0.f, 0.f, 0.f};
    load_decay4(f.A + d * N, q, N, whole, A);
    const long slot = (long)D * N;
    float *carry = p.carry + (long)unit * p.nseg * slot + d * N;
    float *sums = p.carry + (long)f.seq.units * p.nseg * slot + (long)unit * p.nseg * D + d;
    if constexpr (!CARRY) {
      if (p.d_state_out) load_state4(p.d_state_out + ((long)unit * D + d) * N, q, N, whole, g0);
      for (int k = p.nseg - 1; k > seg; --k) {
        float from[4];
        load_state4(carry + k * slot, q, N, whole, from);
        const float sum = sums[(long)k * D];
#pragma unroll
        for (int i = 0; i < 4; ++i) g0[i] = fmaf(__builtin_amdgcn_exp2f(sum * A[i]), g0[i], from[i]);
      }
    }
    // The state at the start of the tile at t0, without a branch: where paths join, the compiler would
    // copy what is loaded and wait for it at once, here for a whole load a tile (498 us instead of 445 at
    // [8, 2048, 2048], N = 16).
    uint32_t value[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) value[i] = (ch * N + 4 * q + i) * 4 + (live && 4 * q + i < N ? 0u : kOutside);
    const auto state_at = [&](int t0, float (&h)[4]) {
      const float *from = t0 ? f.chunk_states : f.seq.state_in;
      const long row = t0 ? (long)unit * f.n_chunks + t0 / TT - 1 : sq.row_in;
      const auto w = window<4>(from, slot, from ? row : 0, from ? 1 : 0, d0 * N, c_live * N);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(w, value[i], 0, 0));
    };
    float h0[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
    f32x4 G = {g0[0], g0[1], g0[2], g0[3]};
    if constexpr (!CARRY) state_at(t_begin + (tiles - 1) * TT, h0);
    __syncthreads();
    for (int k = 0; k < tiles; ++k) {
      const int buf = k & 1, t0 = t_begin + (tiles - 1 - k) * TT;
      if constexpr (CARRY) {
#pragma unroll 4
        for (int u = TT - 1; u >= 0; --u) {
          const float delta = s_dx[buf][u][ch].x;
          G = __builtin_amdgcn_mfma_f32_4x4x1f32(s_c[buf][u][4 * q + j], s_dc[buf][u][ch], G, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) G[i] *= __builtin_amdgcn_exp2f(delta * A[i]);
          total += delta;
        }
      } else {
        float a[TT][4], h[TT][4], sum[LN];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(h0[i]));
#pragma unroll
        for (int u = 0; u < TT; ++u) {
          const float2 dx = s_dx[buf][u][ch];
          const float4 C = *reinterpret_cast<const float4 *>(&s_c[buf][u][4 * q]);
          const f32x4 xb = __builtin_amdgcn_mfma_f32_4x4x1f32(s_b[buf][u][4 * q + j], dx.y, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[u][i] = __builtin_amdgcn_exp2f(dx.x * A[i]);
            h[u][i] = fmaf(a[u][i], u ? h[u - 1][i] : h0[i], xb[i]);
          }
          sum[u % LN] = fmaf(C.w, h[u][3], fmaf(C.z, h[u][2], fmaf(C.y, h[u][1], C.x * h[u][0])));
          if (u % LN == LN - 1) s_out[buf][0][u - (LN - 1) + q][ch] = spread4<LN>(sum, q);
        }
        float next[4];  // the state of the tile that comes next: on its way during this one
        state_at(max(t0 - TT, 0), next);  // (after the last tile, not used)
        float gb[LN], ga[LN];
#pragma unroll
        for (int u = TT - 1; u >= 0; --u) {
          const float2 dx = s_dx[buf][u][ch];
          const float c = s_dc[buf][u][ch];
          const float4 B = *reinterpret_cast<const float4 *>(&s_b[buf][u][4 * q]);
          G = __builtin_amdgcn_mfma_f32_4x4x1f32(s_c[buf][u][4 * q + j], c, G, 0, 0, 0);
          gb[u % LN] = fmaf(B.w, G[3], fmaf(B.z, G[2], fmaf(B.y, G[1], B.x * G[0])));
          float v[8], s = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = G[i] * dx.y;
            v[4 + i] = h[u][i] * c;
            G[i] *= a[u][i];
            const float w = G[i] * (u ? h[u - 1][i] : h0[i]);
            s = i ? fmaf(A[i], w, s) : A[i] * w;
            dA[i] = fmaf(dx.x, w, dA[i]);
          }
          ga[u % LN] = s;
          if (u % LN == 0) {
            s_out[buf][1][u + q][ch] = spread4<LN>(gb, q);
            s_out[buf][2][u + q][ch] = spread4<LN>(ga, q);
          }
          float r[LN == 16 ? 2 : 1];
          int place;
          sum_channels<LN>(v, lane, r, place);
#pragma unroll
          for (int i = 0; i < (LN == 16 ? 2 : 1); ++i) s_bc[buf][wave][u][((place + i) >> 2) * NP + 4 * q + ((place + i) & 3)] = r[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) h0[i] = next[i];
      }
      __syncthreads();
    }
    const float out[4] = {G[0], G[1], G[2], G[3]};
    if (CARRY) {
      if (live) {
        store_state4(carry + seg * slot, q, N, whole, out);
        if (q == 0) sums[(long)seg * D] = total;
      }
    } else if (live) {
      if (seg == 0 && p.d_state_in) store_state4(p.d_state_in + ((long)unit * D + d) * N, q, N, whole, out);
      store_state4(shares + d * N, q, N, whole, dA);
    }
    if constexpr (!CARRY) __syncthreads();  // the staging waves' last sums
    return;
  }

  constexpr int ROW = CH / VW, L_STEP = 256 / ROW, EL = BF16 ? 2 : 4;
  constexpr bool VEC = ROWS != Rows::kSingle;
  int l_c = (tid % ROW) * VW;
  const int l_t = tid / ROW;
  if constexpr (ROWS == Rows::kOverlap) l_c = min(l_c, c_live - VW);
  float bias[VW], skip[VW], d_skip[VW] = {}, d_bias[VW] = {};
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const bool in = l_c + e < c_live;
    bias[e] = f.dt_bias && in ? f.dt_bias[d0 + l_c + e] : 0.f;
    skip[e] = f.skip && in ? f.skip[d0 + l_c + e] : 0.f;
  }
  const auto columns = [&](int el, uint32_t (&col)[VEC ? 1 : VW]) {
#pragma unroll
    for (int e = 0; e < (VEC ? 1 : VW); ++e) col[e] = (l_c + e) * el + (l_c + e < c_live ? 0u : kOutside);
  };
  uint32_t col[VEC ? 1 : VW];
  columns(EL, col);
  using Raw = RawRow<BF16, VEC, VW>;
  using Dy = RawRow<false, VEC, VW>;  // dy as fp32, or bf16 in the first words
  struct Item { Raw x, dt, z; Dy dy; };
  Item want[NI];  // as loaded, of the tile requested
  // What the gradients of a (token, channel) need beside the sums.  A tile's are overwritten by those of
  // the second tile after it, staged after it is finished: two sets, by the tile's parity.
  struct Kept { float x[VW], delta[VW], slope[VW], c[VW], gate[VW]; };
  Kept kept[2][NI];
  uint32_t bb[NB] = {}, cc[NB] = {};
  const bool gate = f.z.base;
  const int b_n = tid % NP, b_t = tid / NP;
  constexpr int B_STEP = 256 / NP;
  const bool b_in = TT * NP >= 256 || b_t < TT;
  const uint32_t b_col = b_n * EL + (b_n < N && b_in ? 0u : kOutside);

  const auto dy_of = [&](const Item &it, int e) {
    if (!p.dy_bf16) return it.dy.get(e);
    if constexpr (VEC) return e & 1 ? bf16_hi(it.dy.w[e / 2]) : bf16_lo(it.dy.w[e / 2]);
    else return bf16_lo(it.dy.w[e]);
  };
  const auto request = [&](int t0) {
    const long row = sq.off + t0;
    const int rows = min(TT, t_end - t0);
    const auto wx = window<EL>(f.x.base, f.x.stride, row, rows, d0, c_live);
    const auto wd = window<EL>(f.dt.base, f.dt.stride, row, rows, d0, c_live);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t t = l_t + i * L_STEP;
      want[i].x.load(wx, t * (uint32_t)f.x.stride * EL, col);
      want[i].dt.load(wd, t * (uint32_t)f.dt.stride * EL, col);
    }
    if (gate) {
      const auto wz = window<EL>(f.z.base, f.z.stride, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) want[i].z.load(wz, (l_t + i * L_STEP) * (uint32_t)f.z.stride * EL, col);
    }
    uint32_t to[VEC ? 1 : VW];
    if (p.dy_bf16) {
      columns(2, to);
      const auto wy = window<2>(p.dy.base, p.dy.stride, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        RawRow<true, VEC, VW> v;
        v.load(wy, (l_t + i * L_STEP) * (uint32_t)p.dy.stride * 2, to);
#pragma unroll
        for (int e = 0; e < (int)(sizeof v.w / 4); ++e) want[i].dy.w[e] = v.w[e];
      }
    } else {
      columns(4, to);
      const auto wy = window<4>(p.dy.base, p.dy.stride, row, rows, d0, c_live);
#pragma unroll
      for (int i = 0; i < NI; ++i) want[i].dy.load(wy, (l_t + i * L_STEP) * (uint32_t)p.dy.stride * 4, to);
    }
    const auto wb = window<EL>(f.Bm.base, f.Bm.stride, row, rows, (long)g * N, N);
    const auto wc = window<EL>(f.Cm.base, f.Cm.stride, row, rows, (long)g * N, N);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t t = b_t + i * B_STEP;
      const int ob = (int)(t * (uint32_t)f.Bm.stride * EL + b_col), oc = (int)(t * (uint32_t)f.Cm.stride * EL + b_col);
      if constexpr (BF16) {
        if constexpr (!CARRY) bb[i] = __builtin_amdgcn_raw_buffer_load_b16(wb, ob, 0, 0);
        cc[i] = __builtin_amdgcn_raw_buffer_load_b16(wc, oc, 0, 0);
      } else {
        if constexpr (!CARRY) bb[i] = __builtin_amdgcn_raw_buffer_load_b32(wb, ob, 0, 0);
        cc[i] = __builtin_amdgcn_raw_buffer_load_b32(wc, oc, 0, 0);
      }
    }
  };
  const auto stage = [&](int t0, auto parity) {
    constexpr int buf = decltype(parity)::value;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      want[i].x.arrive(); want[i].dt.arrive(); want[i].dy.arrive();
      if (gate) want[i].z.arrive();
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(bb[i]), "+v"(cc[i]));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      Kept &k = kept[buf][i];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        k.x[e] = want[i].x.get(e);
        k.delta[e] = want[i].dt.get(e) + bias[e];
        k.slope[e] = 1.f;
        k.c[e] = dy_of(want[i], e);
        k.gate[e] = 0.f;
      }
      if (f.softplus) {
#pragma unroll
        for (int e = 0; e < VW; ++e) k.delta[e] = softplus_f(k.delta[e], k.slope[e]);
      }
      if (gate) {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const float z = want[i].z.get(e), sg = sigmoid_f(z), dy = k.c[e], u = z * sg;
          k.c[e] = dy * u;
          k.gate[e] = dy * (sg + u * (1.f - sg));
        }
      }
      const int t = l_t + i * L_STEP;
      if (t0 + TT > t_end && t0 + t >= t_end) {  // a token past the end leaves states and gradients as they are
#pragma unroll
        for (int e = 0; e < VW; ++e) k.delta[e] = k.slope[e] = 0.f;
      }
      float2 *dx = &s_dx[buf][t][l_c];
      float *dc = &s_dc[buf][t][l_c];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        dx[e] = make_float2(k.delta[e], k.delta[e] * k.x[e]);
        dc[e] = k.c[e];
        if constexpr (!CARRY) d_skip[e] = fmaf(k.c[e], k.x[e], d_skip[e]);
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int t = (b_t + i * B_STEP) & (TT - 1);
      if (b_in) {
        if constexpr (!CARRY) s_b[buf][t][b_n] = BF16 ? bf16_lo(bb[i]) : __uint_as_float(bb[i]);
        s_c[buf][t][b_n] = BF16 ? bf16_lo(cc[i]) : __uint_as_float(cc[i]);
      }
    }
  };
  const auto write = [&](void *to, int i, int t0, const float (&v)[VW]) {
    const long row = sq.off + t0;
    const int rows = min(TT, t_end - t0);
    uint32_t at[VEC ? 1 : VW];
    if (p.grad_bf16) {
      columns(2, at);
      store_row<true, VEC, VW>(window<2>(to, D, row, rows, d0, c_live), (l_t + i * L_STEP) * (uint32_t)D * 2, at, v);
    } else {
      columns(4, at);
      store_row<false, VEC, VW>(window<4>(to, D, row, rows, d0, c_live), (l_t + i * L_STEP) * (uint32_t)D * 4, at, v);
    }
  };
  const auto finish = [&](int t0, auto parity) {  // the gradients of the tile at t0
    constexpr int buf = decltype(parity)::value;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int t = l_t + i * L_STEP;
      const Kept &k = kept[buf][i];
      float gx[VW], gt[VW], gz[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float gb = s_out[buf][1][t][l_c + e];
        gz[e] = k.gate[e] * fmaf(skip[e], k.x[e], s_out[buf][0][t][l_c + e]);
        gx[e] = fmaf(k.delta[e], gb, skip[e] * k.c[e]);
        gt[e] = k.slope[e] * fmaf(k.x[e], gb, s_out[buf][2][t][l_c + e] * 0.6931471805599453f);
        d_bias[e] += gt[e];
      }
      write(p.dx, i, t0, gx);
      write(p.ddt, i, t0, gt);
      if (gate) write(p.dz, i, t0, gz);
    }
    // dB and dC of the tile's tokens: this block's sums
    constexpr int COLS = 2 * NP, PER = TT * COLS / 256, STEP = 256 / COLS;
    const int n = tid % COLS, t = tid / COLS;
    if (n % NP < N) {
      float *to = p.part_bc + (((long)block * f.seq.total_tokens + sq.off + t0 + t) * f.G + g) * 2 * N + (n < NP ? n : n - NP + N);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const auto &v = s_bc[buf];
        const int u = t + i * STEP;
        if (t0 + u < t_end) to[(long)i * STEP * f.G * 2 * N] = (v[0][u][n] + v[1][u][n]) + (v[2][u][n] + v[3][u][n]);
      }
    }
  };

  if constexpr (ROWS == Rows::kOverlap) {  // the columns past the block's channels, which nothing writes, have no share in sums
    for (int e = tid; e < 2 * TT * (CH - c_live); e += 256) {
      const int row = e / (CH - c_live), c = c_live + e % (CH - c_live);
      s_dx[row & 1][row >> 1][c] = make_float2(0.f, 0.f);
      s_dc[row & 1][row >> 1][c] = 0.f;
    }
  }
  const int last = t_begin + (tiles - 1) * TT;
  request(last);
  stage(last, Set<0>{});
  if (tiles > 1) request(last - TT);
  __syncthreads();
  const auto step = [&](int k, auto other) {  // while tile k is walked; other: the parity of the tiles beside it
    const int t0 = last - k * TT;
    if constexpr (!CARRY) {
      if (k) finish(t0 + TT, other);
    }
    if (k + 1 < tiles) {
      stage(t0 - TT, other);
      if (k + 2 < tiles) request(t0 - 2 * TT);
    }
    __syncthreads();
  };
  for (int k = 0; k < tiles; k += 2) {
    step(k, Set<1>{});
    if (k + 1 < tiles) step(k + 1, Set<0>{});
  }
  if constexpr (!CARRY) {
    if (tiles & 1) finish(t_begin, Set<0>{});
    else finish(t_begin, Set<1>{});
    // the threads that share channels add their sums in the order of their tokens (the scan waves are done with s_dx)
    float2 (*sum)[CH] = s_dx[0];
#pragma unroll
    for (int e = 0; e < VW; ++e) sum[l_t][l_c + e] = make_float2(d_skip[e], d_bias[e]);
    __syncthreads();
    if (tid < c_live) {
      float a = 0.f, b = 0.f;
      for (int i = 0; i < L_STEP; ++i) {
        a += sum[i][tid].x;
        b += sum[i][tid].y;
      }
      shares[(long)D * N + d0 + tid] = a;
      shares[(long)D * N + D + d0 + tid] = b;
    }
  }
}

// The sums that are left, in one launch.  The first `bc_groups` workgroups add the channel blocks' dB
// and dC in their order.  The others add the rows' and segments' shares of dA, d_skip and d_bias, 64
// columns each (a row is read 256 bytes at a time): each of 16 threads of a column every 16th row,
// then the 16 sums in order.
__global__ void __launch_bounds__(1024) ssm_backward_sum_kernel(ScanBackwardParams p, int blocks, unsigned bc_groups) {
  const ScanSsmParams &f = p.f;
  if (blockIdx.x < bc_groups) {
    const long GN = (long)f.G * f.N, total = f.seq.total_tokens * 2 * GN;
    const long at = (long)blockIdx.x * 1024 + threadIdx.x;
    if (at >= total) return;
    const int n = (int)(at % (2 * f.N));
    const long row = at / (2 * GN), g = at / (2 * f.N) % f.G;
    if (f.seq.state_map) {  // rows without a state have no gradients
      const int s = f.seq.state_map[row / f.seq.T];
      if (s < 0 || s >= f.seq.n_state) return;
    }
    float sum = 0.f;
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) sum += p.part_bc[b * total + at];
    const long to = row * GN + g * f.N;
    if (n < f.N) store1(p.dB, to + n, p.grad_bf16, sum);
    else store1(p.dC, to + n - f.N, p.grad_bf16, sum);
    return;
  }
  __shared__ float s[16][64];
  const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
  const long DN = (long)f.D * f.N, cols = DN + 2L * f.D, rows = (long)f.seq.units * p.nseg;
  const long col = (long)(blockIdx.x - bc_groups) * 64 + c;
  float a = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (long r = k; r < rows; r += 16) a += p.part[r * cols + col];
  }
  s[k][c] = a;
  __syncthreads();
  if (k == 0 && col < cols) {
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += s[i][c];
    if (col < DN) p.dA[col] = t;
    else if (col < DN + f.D) { if (p.d_skip) p.d_skip[col - DN] = t; }
    else if (p.d_bias) p.d_bias[col - DN - f.D] = t;
  }
}

template <bool BF16, Rows ROWS, int LN>
void go_rows(const ScanBackwardParams &p, int blocks, hipStream_t s) {
  if (p.nseg > 1)
    hipLaunchKernelGGL((ssm_scan_backward_kernel<BF16, ROWS, LN, true>), dim3(blocks, p.f.seq.units, p.nseg - 1), dim3(512), 0, s, p);
  hipLaunchKernelGGL((ssm_scan_backward_kernel<BF16, ROWS, LN, false>), dim3(blocks, p.f.seq.units, p.nseg), dim3(512), 0, s, p);
}

template <bool BF16, int LN>
hipError_t go(const ScanBackwardParams &p, hipStream_t s) {
  constexpr int CH = 256 / LN, VW = BTile<LN>::VW;
  const int per_group = p.f.D / p.f.G, nb = (per_group + CH - 1) / CH, blocks = p.f.G * nb;
  const Rows rows = rows_of<CH, VW>(per_group);
  if constexpr (VW > 1) {
    if (rows == Rows::kWhole) go_rows<BF16, Rows::kWhole, LN>(p, blocks, s);
    else if (rows == Rows::kOverlap) go_rows<BF16, Rows::kOverlap, LN>(p, blocks, s);
  }
  if (rows == Rows::kSingle) go_rows<BF16, Rows::kSingle, LN>(p, blocks, s);
  const long values = p.f.seq.total_tokens * 2 * p.f.G * p.f.N, cols = (long)p.f.D * (p.f.N + 2);
  const unsigned bc_groups = (unsigned)((values + 1023) / 1024);
  hipLaunchKernelGGL(ssm_backward_sum_kernel, dim3(bc_groups + (unsigned)((cols + 63) / 64)), dim3(1024), 0, s, p, nb, bc_groups);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_states(const ScanBackwardParams &p, hipStream_t s) {
  switch (lanes_of(p.f.N)) {
    case 1:
    case 2: return go<BF16, 2>(p, s);
    case 4: return go<BF16, 4>(p, s);
    case 8: return go<BF16, 8>(p, s);
    default: return go<BF16, 16>(p, s);
  }
}

}  // namespace

int backward_blocks(int D, int N, int G) {
  const int CH = 256 / (lanes_of(N) < 2 ? 2 : lanes_of(N));
  return (D / G + CH - 1) / CH;
}

int backward_segments(int units, int T, int D, int N, int G, int *seg_len) {
  return best_segments((long)units * G * backward_blocks(D, N, G), T, TT, 1.0, 0.3, 30, seg_len);
}

hipError_t launch_ssm_scan_backward(const ScanBackwardParams &p, bool bf16, hipStream_t s) {
  return bf16 ? by_states<true>(p, s) : by_states<false>(p, s);
}

}  // namespace wkv
