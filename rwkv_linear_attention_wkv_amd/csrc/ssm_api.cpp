// C ABI of the state space operators: argument validation and launch.  Every
// host-checkable problem is reported before any HIP call.
#include "wkv_ssm.h"

#include <limits>
#include <type_traits>
#include <utility>

#include "api_common.hpp"
#include "ssm.hpp"

using namespace wkv::api;

namespace {

constexpr int kMaxChannels = wkv::kMaxStride;
constexpr int kMaxStates = 64;
constexpr int kMaxTokens = 1 << 30;  // of one sequence

// Sequences and states of a dense call; `state_row` floats per state row.
wkv_status dense_seq(const char *fn, int B, int T, const float *state_in, const int32_t *state_map, int n_state,
                     float *state_out, int32_t *dev_status, wkv::SeqParams *out) {
  REQUIRE(B >= 1 && T >= 0, "%s: need B >= 1 and T >= 0 (got B=%d T=%d)", fn, B, T);
  REQUIRE(B <= kMaxGridY, "%s: B=%d exceeds %d", fn, B, kMaxGridY);
  REQUIRE(T <= kMaxTokens, "%s: T=%d exceeds %d", fn, T, kMaxTokens);
  if (state_in) {
    REQUIRE(aligned(state_in, 16), "%s: state_in must be 16-byte aligned", fn);
    REQUIRE(n_state >= 1, "%s: n_state must be >= 1 when state_in is given (got %d)", fn, n_state);
    if (!state_map)
      REQUIRE(n_state == 1 || n_state == B, "%s: without state_map, n_state must be 1 or B (got %d, B=%d)", fn,
              n_state, B);
    else
      REQUIRE(aligned(state_map, 4), "%s: state_map must be 4-byte aligned", fn);
  } else {
    REQUIRE(!state_map, "%s: state_map given without state_in", fn);
  }
  if (state_out) {
    REQUIRE(aligned(state_out, 16), "%s: state_out must be 16-byte aligned", fn);
    if (state_out == state_in)
      REQUIRE(!state_map && n_state == B, "%s: in-place state needs state_map == NULL and n_state == B", fn);
  }
  REQUIRE(!dev_status || aligned(dev_status, 4), "%s: dev_status must be 4-byte aligned", fn);
  *out = wkv::SeqParams{B, T, nullptr, (long)B * T, state_in, state_map, n_state, state_out, dev_status};
  return WKV_OK;
}

wkv_status varlen_seq(const char *fn, int num_slots, const int32_t *lengths, int max_len, int total_tokens,
                      const float *state_in, float *state_out, const int32_t *state_map, int n_state,
                      int32_t *dev_status, wkv::SeqParams *out) {
  REQUIRE(num_slots >= 0 && max_len >= 0 && total_tokens >= 0,
          "%s: need num_slots >= 0, max_len >= 0, total_tokens >= 0", fn);
  REQUIRE(max_len <= kMaxTokens, "%s: max_len=%d exceeds %d", fn, max_len, kMaxTokens);
  REQUIRE(num_slots <= kMaxGridY, "%s: num_slots=%d exceeds %d", fn, num_slots, kMaxGridY);
  if (num_slots > 0) {
    REQUIRE(lengths && aligned(lengths, 4), "%s: lengths must be a non-NULL, 4-byte aligned device array", fn);
    REQUIRE(state_in && state_out, "%s: state_in and state_out must be non-NULL", fn);
    REQUIRE(aligned(state_in, 16) && aligned(state_out, 16), "%s: states must be 16-byte aligned", fn);
    REQUIRE(n_state >= 1, "%s: n_state must be >= 1", fn);
    if (!state_map)
      REQUIRE(n_state >= num_slots, "%s: without state_map, n_state (%d) must be >= num_slots (%d)", fn, n_state,
              num_slots);
    else
      REQUIRE(aligned(state_map, 4), "%s: state_map must be 4-byte aligned", fn);
    REQUIRE(!dev_status || aligned(dev_status, 4), "%s: dev_status must be 4-byte aligned", fn);
  }
  *out = wkv::SeqParams{num_slots, max_len, lengths, total_tokens, state_in, state_map, n_state, state_out, dev_status};
  return WKV_OK;
}

// One token array of the call: present, aligned to its element, rows at least `width` apart.
wkv_status token_array(const char *fn, const char *name, const void *base, int64_t stride, long width,
                       wkv_dtype dtype) {
  REQUIRE(base, "%s: %s must be non-NULL", fn, name);
  REQUIRE(aligned(base, dtype == WKV_BF16 ? 2 : 4), "%s: %s must be aligned to its element", fn, name);
  REQUIRE(stride >= width && stride <= wkv::kMaxStride, "%s: %s has row stride %lld for rows of %ld", fn, name,
          (long long)stride, width);
  return WKV_OK;
}

#define CHECK(call)                   \
  do {                                \
    const wkv_status st_ = (call);    \
    if (st_ != WKV_OK) return st_;    \
  } while (0)

wkv_status conv_checks(const char *fn, int D, int W, wkv_dtype in_dtype, const float *weight, const float *bias,
                       wkv_activation act) {
  REQUIRE(D >= 1 && D <= kMaxChannels, "%s: need 1 <= D <= %d (got %d)", fn, kMaxChannels, D);
  if (W < 2 || W > 4) return fail(WKV_ERR_UNSUPPORTED, "%s: W=%d is not supported (2, 3 or 4)", fn, W);
  if (!dtype_ok(in_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown input dtype %d", fn, in_dtype);
  if (act != WKV_ACT_NONE && act != WKV_ACT_SILU) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, act);
  REQUIRE(weight && aligned(weight, 4) && aligned(bias, 4), "%s: weight must be given; weight and bias 4-byte aligned", fn);
  return WKV_OK;
}

wkv_status conv(const char *fn, const wkv::SeqParams &seq, int D, int W, const void *x, int64_t x_stride,
                wkv_dtype in_dtype, const float *weight, const float *bias, wkv_activation act, void *y,
                wkv_dtype out_dtype, void *stream) {
  CHECK(conv_checks(fn, D, W, in_dtype, weight, bias, act));
  if (!dtype_ok(out_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown output dtype %d", fn, out_dtype);
  if (seq.units == 0) return ok();
  if (seq.total_tokens > 0) {
    CHECK(token_array(fn, "x", x, x_stride, D, in_dtype));
    REQUIRE(y && aligned(y, 16), "%s: y must be non-NULL and 16-byte aligned", fn);
    REQUIRE(y != x, "%s: y may not overlap x", fn);
  } else if (!seq.lengths && !seq.state_out) {
    return ok();
  }
  wkv::ConvParams p{};
  p.seq = seq;
  p.D = D; p.W = W;
  p.x = {x, (long)x_stride};
  p.weight = weight; p.bias = bias;
  p.silu = act == WKV_ACT_SILU;
  p.y = y; p.y_bf16 = out_dtype == WKV_BF16;
  p.nseg = wkv::conv_segments(seq.T, seq.total_tokens, D, in_dtype == WKV_BF16, false, &p.seg_len);
  return launched(wkv::launch_ssm_conv(p, in_dtype == WKV_BF16, static_cast<hipStream_t>(stream)), fn);
}

size_t scan_workspace(int units, int nseg, int D, int N) {
  return nseg > 1 ? sizeof(float) * (size_t)units * ((size_t)nseg * D * N + (size_t)(nseg - 1) * D) : 0;
}

int chunks_of(int T) { return T > 0 ? (T + wkv::kScanChunk - 1) / wkv::kScanChunk - 1 : 0; }

// The backward pass's workspace, in floats from its start; each part starts at a multiple of four.
struct BackwardSpace {
  size_t carry, part, part_bc, chunks, total;
  int nseg, seg_len;
};

BackwardSpace backward_space(int B, int T, int D, int N, int G, bool with_chunks) {
  BackwardSpace w{};
  size_t at = 0;
  const auto take = [&at](size_t floats) {
    const size_t here = at;
    at += (floats + 3) / 4 * 4;
    return here;
  };
  w.nseg = wkv::backward_segments(B, T, D, N, G, &w.seg_len);
  const size_t row = (size_t)D * N, parts = (size_t)B * w.nseg;
  size_t carry = w.nseg > 1 ? parts * (row + D) : 0;
  if (!with_chunks) {  // the forward pass's segments use the same part before it
    int len;
    const size_t fwd = scan_workspace(B, wkv::scan_segments(B, T, (long)B * T, D, N, G, &len), D, N) / sizeof(float);
    if (fwd > carry) carry = fwd;
  }
  w.carry = take(carry);
  w.part = take(parts * (row + 2 * D));
  w.part_bc = take((size_t)wkv::backward_blocks(D, N, G) * B * T * G * 2 * N);
  w.chunks = take(with_chunks ? 0 : (size_t)B * chunks_of(T) * row);
  w.total = at;
  return w;
}

// Checks shared by the scan's calls, and their parameters.
wkv_status scan_params(const char *fn, const wkv::SeqParams &seq, int D, int N, int G, const void *x,
                       int64_t x_stride, const void *dt, int64_t dt_stride, const float *A, const void *Bm,
                       int64_t b_stride, const void *Cm, int64_t c_stride, wkv_dtype in_dtype, const float *skip,
                       const void *z, int64_t z_stride, const float *dt_bias, int dt_softplus,
                       wkv::ScanSsmParams *p) {
  REQUIRE(D >= 1 && D <= kMaxChannels, "%s: need 1 <= D <= %d (got %d)", fn, kMaxChannels, D);
  if (N < 1 || N > kMaxStates)
    return fail(WKV_ERR_UNSUPPORTED, "%s: N=%d states per channel are not supported (1 .. %d)", fn, N, kMaxStates);
  REQUIRE(G >= 1 && D % G == 0, "%s: D=%d channels do not divide into G=%d groups", fn, D, G);
  if (!dtype_ok(in_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown input dtype %d", fn, in_dtype);
  REQUIRE(A && aligned(A, 16), "%s: A must be non-NULL and 16-byte aligned", fn);
  REQUIRE(aligned(skip, 4) && aligned(dt_bias, 4), "%s: skip and dt_bias must be 4-byte aligned", fn);
  if (seq.total_tokens > 0) {
    CHECK(token_array(fn, "x", x, x_stride, D, in_dtype));
    CHECK(token_array(fn, "dt", dt, dt_stride, D, in_dtype));
    CHECK(token_array(fn, "B", Bm, b_stride, (long)G * N, in_dtype));
    CHECK(token_array(fn, "C", Cm, c_stride, (long)G * N, in_dtype));
    if (z) CHECK(token_array(fn, "z", z, z_stride, D, in_dtype));
  }
  *p = wkv::ScanSsmParams{};
  p->seq = seq;
  p->D = D; p->N = N; p->G = G;
  p->x = {x, (long)x_stride}; p->dt = {dt, (long)dt_stride}; p->z = {z, (long)z_stride};
  p->Bm = {Bm, (long)b_stride}; p->Cm = {Cm, (long)c_stride};
  p->A = A; p->skip = skip; p->dt_bias = dt_bias;
  p->softplus = dt_softplus != 0;
  return WKV_OK;
}

wkv_status scan(const char *fn, wkv::ScanSsmParams &p, wkv_dtype in_dtype, void *y, wkv_dtype out_dtype,
                void *workspace, size_t workspace_bytes, void *stream) {
  if (!dtype_ok(out_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown output dtype %d", fn, out_dtype);
  if (p.seq.units == 0) return ok();
  if (p.seq.total_tokens > 0) {
    REQUIRE(y && aligned(y, 16), "%s: y must be non-NULL and 16-byte aligned", fn);
    REQUIRE(y != p.x.base && y != p.dt.base && y != p.z.base, "%s: y may not overlap an input", fn);
  } else if (!p.seq.lengths && !p.seq.state_out) {
    return ok();
  }
  p.y = y; p.y_bf16 = out_dtype == WKV_BF16;
  p.nseg = wkv::scan_segments(p.seq.units, p.seq.T, p.seq.total_tokens, p.D, p.N, p.G, &p.seg_len);
  if (p.nseg > 1) {
    const size_t need = scan_workspace(p.seq.units, p.nseg, p.D, p.N);
    if (workspace) {
      REQUIRE(aligned(workspace, 16) && workspace_bytes >= need,
              "%s: the workspace must be 16-byte aligned and hold %zu bytes (got %zu)", fn, need, workspace_bytes);
      p.workspace = static_cast<float *>(workspace);
    } else {
      p.nseg = 1; p.seg_len = p.seq.T;  // every sequence in one piece
    }
  }
  return launched(wkv::launch_ssm_scan(p, in_dtype == WKV_BF16, static_cast<hipStream_t>(stream)), fn);
}

wkv_status store(const char *fn, const void *data, const float *scale, int n_store, wkv_store_format format,
                 const float *states, int n_state, int64_t row, const int32_t *store_rows,
                 const int32_t *state_rows, int count, int32_t *dev_status, wkv::StoreParams *p) {
  REQUIRE(count >= 0 && n_store >= 0 && n_state >= 0 && row >= 1 && row <= (int64_t)1 << 40,
          "%s: need count, n_store, n_state >= 0 and row >= 1", fn);
  if (format != WKV_STORE_INT8 && format != WKV_STORE_E4M3)
    return fail(WKV_ERR_UNSUPPORTED, "%s: unknown store format %d", fn, format);
  REQUIRE(count <= kMaxGridY, "%s: count=%d exceeds %d", fn, count, kMaxGridY);
  if (count > 0) {
    REQUIRE(data && scale && states, "%s: data, scale and states must be non-NULL", fn);
    REQUIRE(aligned(data, 16) && aligned(scale, 4) && aligned(states, 16),
            "%s: data and states must be 16-byte aligned, scale 4-byte aligned", fn);
    REQUIRE(store_rows || count <= n_store, "%s: without store_rows, count (%d) must be <= n_store (%d)", fn, count, n_store);
    REQUIRE(state_rows || count <= n_state, "%s: without state_rows, count (%d) must be <= n_state (%d)", fn, count, n_state);
    REQUIRE(aligned(store_rows, 4) && aligned(state_rows, 4) && aligned(dev_status, 4),
            "%s: store_rows, state_rows and dev_status must be 4-byte aligned", fn);
  }
  *p = wkv::StoreParams{const_cast<void *>(data), const_cast<float *>(scale), const_cast<float *>(states), store_rows,
                        state_rows, n_store, n_state, count, (long)row, format == WKV_STORE_E4M3, dev_status};
  return WKV_OK;
}

// A parameter from its word; `fits` is cleared where the word is out of its range.
template <class T>
T from_word(int64_t w, bool &fits) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(w));
  } else {
    if (sizeof(T) < sizeof w && (w < std::numeric_limits<T>::min() || w > std::numeric_limits<T>::max())) fits = false;
    return static_cast<T>(w);
  }
}

template <class... A, size_t... I>
wkv_status call_words(const char *fn, wkv_status (*f)(A...), const int64_t *w, int count, std::index_sequence<I...>) {
  REQUIRE(count == (int)sizeof...(A), "%s: takes %d arguments (got %d)", fn, (int)sizeof...(A), count);
  bool fits = true;
  const auto call = [&](A... a) { return fits ? f(a...) : fail(WKV_ERR_INVALID_ARG, "%s: an argument is out of its range", fn); };
  return call(from_word<A>(w[I], fits)...);
}

template <class... A>
wkv_status call_words(const char *fn, wkv_status (*f)(A...), const int64_t *w, int count) {
  return call_words(fn, f, w, count, std::make_index_sequence<sizeof...(A)>{});
}

}  // namespace

extern "C" {

wkv_status wkv_ssm_conv_forward(int B, int T, int D, int W, const void *x, int64_t x_stride, wkv_dtype in_dtype,
                                const float *weight, const float *bias, wkv_activation act, void *y,
                                wkv_dtype out_dtype, const float *state_in, const int32_t *state_map, int n_state,
                                float *state_out, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_ssm_conv_forward";
  wkv::SeqParams seq;
  CHECK(dense_seq(fn, B, T, state_in, state_map, n_state, state_out, dev_status, &seq));
  return conv(fn, seq, D, W, x, x_stride, in_dtype, weight, bias, act, y, out_dtype, stream);
}

wkv_status wkv_ssm_conv_forward_varlen(int num_slots, int D, int W, const int32_t *lengths, int max_len,
                                       int total_tokens, const void *x, int64_t x_stride, wkv_dtype in_dtype,
                                       const float *weight, const float *bias, wkv_activation act, void *y,
                                       wkv_dtype out_dtype, const float *state_in, float *state_out,
                                       const int32_t *state_map, int n_state, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_ssm_conv_forward_varlen";
  wkv::SeqParams seq;
  CHECK(varlen_seq(fn, num_slots, lengths, max_len, total_tokens, state_in, state_out, state_map, n_state, dev_status, &seq));
  return conv(fn, seq, D, W, x, x_stride, in_dtype, weight, bias, act, y, out_dtype, stream);
}

size_t wkv_ssm_conv_backward_workspace(int B, int T, int D, int W) {
  if (B < 1 || T < 1 || D < 1 || W < 2 || W > 4) return 0;
  int len;
  return sizeof(float) * (size_t)B * wkv::conv_segments(T, (long)B * T, D, true, true, &len) * (W + 1) * D;
}

wkv_status wkv_ssm_conv_backward(int B, int T, int D, int W, const void *x, int64_t x_stride, wkv_dtype in_dtype,
                                 const float *weight, const float *bias, wkv_activation act, const void *dy,
                                 int64_t dy_stride, wkv_dtype dy_dtype, const float *state_in,
                                 const int32_t *state_map, int n_state, const float *d_state_out, void *dx,
                                 wkv_dtype grad_dtype, float *d_weight, float *d_bias, float *d_state_in,
                                 void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_ssm_conv_backward";
  REQUIRE(T >= 1, "%s: need T >= 1 (got %d)", fn, T);
  wkv::ConvParams p{};
  CHECK(dense_seq(fn, B, T, state_in, state_map, n_state, nullptr, dev_status, &p.seq));
  CHECK(conv_checks(fn, D, W, in_dtype, weight, bias, act));
  if (!dtype_ok(dy_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown dtype of dy %d", fn, dy_dtype);
  if (!dtype_ok(grad_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown gradient dtype %d", fn, grad_dtype);
  CHECK(token_array(fn, "x", x, x_stride, D, in_dtype));
  CHECK(token_array(fn, "dy", dy, dy_stride, D, dy_dtype));
  REQUIRE(dx && d_weight, "%s: dx and d_weight must be non-NULL", fn);
  REQUIRE(aligned(dx, 16) && aligned(d_weight, 4) && aligned(d_bias, 4) && aligned(d_state_in, 16) && aligned(d_state_out, 16),
          "%s: dx and the states' gradients must be 16-byte aligned, d_weight and d_bias 4-byte aligned", fn);
  REQUIRE(dx != x && dx != dy, "%s: dx may not overlap an input", fn);
  const size_t need = wkv_ssm_conv_backward_workspace(B, T, D, W);
  REQUIRE(workspace && aligned(workspace, 16) && workspace_bytes >= need,
          "%s: the workspace must be 16-byte aligned and hold %zu bytes (got %zu)", fn, need, workspace_bytes);
  p.D = D; p.W = W;
  p.x = {x, (long)x_stride};
  p.weight = weight; p.bias = bias;
  p.silu = act == WKV_ACT_SILU;
  p.y = dx; p.y_bf16 = grad_dtype == WKV_BF16;
  p.dy = {dy, (long)dy_stride}; p.dy_bf16 = dy_dtype == WKV_BF16;
  p.d_state_out = d_state_out; p.d_state_in = d_state_in;
  p.partial = static_cast<float *>(workspace);
  p.d_weight = d_weight; p.d_bias = d_bias;
  p.nseg = wkv::conv_segments(T, (long)B * T, D, in_dtype == WKV_BF16, true, &p.seg_len);
  return launched(wkv::launch_ssm_conv_backward(p, in_dtype == WKV_BF16, static_cast<hipStream_t>(stream)), fn);
}

size_t wkv_ssm_scan_workspace(int rows, int T, int64_t total_tokens, int D, int N, int G) {
  if (rows < 1 || T < 1 || total_tokens < 0 || D < 1 || N < 1 || N > kMaxStates || G < 1 || D % G) return 0;
  int len;
  return scan_workspace(rows, wkv::scan_segments(rows, T, (long)total_tokens, D, N, G, &len), D, N);
}

wkv_status wkv_ssm_scan_forward(int B, int T, int D, int N, int G, const void *x, int64_t x_stride, const void *dt,
                                int64_t dt_stride, const float *A, const void *Bm, int64_t b_stride, const void *Cm,
                                int64_t c_stride, wkv_dtype in_dtype, const float *skip, const void *z,
                                int64_t z_stride, const float *dt_bias, int dt_softplus, void *y,
                                wkv_dtype out_dtype, const float *state_in, const int32_t *state_map, int n_state,
                                float *state_out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                void *stream) {
  const char *fn = "wkv_ssm_scan_forward";
  wkv::SeqParams seq;
  CHECK(dense_seq(fn, B, T, state_in, state_map, n_state, state_out, dev_status, &seq));
  wkv::ScanSsmParams p;
  CHECK(scan_params(fn, seq, D, N, G, x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, in_dtype, skip, z,
                    z_stride, dt_bias, dt_softplus, &p));
  return scan(fn, p, in_dtype, y, out_dtype, workspace, workspace_bytes, stream);
}

wkv_status wkv_ssm_scan_forward_train(int B, int T, int D, int N, int G, const void *x, int64_t x_stride,
                                      const void *dt, int64_t dt_stride, const float *A, const void *Bm,
                                      int64_t b_stride, const void *Cm, int64_t c_stride, wkv_dtype in_dtype,
                                      const float *skip, const void *z, int64_t z_stride, const float *dt_bias,
                                      int dt_softplus, void *y, wkv_dtype out_dtype, const float *state_in,
                                      const int32_t *state_map, int n_state, float *state_out, float *chunk_states,
                                      void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_ssm_scan_forward_train";
  wkv::SeqParams seq;
  CHECK(dense_seq(fn, B, T, state_in, state_map, n_state, state_out, dev_status, &seq));
  wkv::ScanSsmParams p;
  CHECK(scan_params(fn, seq, D, N, G, x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, in_dtype, skip, z,
                    z_stride, dt_bias, dt_softplus, &p));
  p.n_chunks = chunks_of(T);
  if (p.n_chunks > 0) {
    REQUIRE(chunk_states && aligned(chunk_states, 16),
            "%s: chunk_states must be a non-NULL, 16-byte aligned device array (T > %d)", fn, wkv::kScanChunk);
    p.chunk_states = chunk_states;
  }
  return scan(fn, p, in_dtype, y, out_dtype, workspace, workspace_bytes, stream);
}

size_t wkv_ssm_scan_backward_workspace(int B, int T, int D, int N, int G, int with_chunk_states) {
  if (B < 1 || T < 1 || D < 1 || N < 1 || N > kMaxStates || G < 1 || D % G) return 0;
  return sizeof(float) * backward_space(B, T, D, N, G, with_chunk_states != 0).total;
}

wkv_status wkv_ssm_scan_backward(int B, int T, int D, int N, int G, const void *x, int64_t x_stride, const void *dt,
                                 int64_t dt_stride, const float *A, const void *Bm, int64_t b_stride,
                                 const void *Cm, int64_t c_stride, wkv_dtype in_dtype, const float *skip,
                                 const void *z, int64_t z_stride, const float *dt_bias, int dt_softplus,
                                 const void *dy, int64_t dy_stride, wkv_dtype dy_dtype, const float *state_in,
                                 const int32_t *state_map, int n_state, const float *chunk_states,
                                 const float *d_state_out, void *dx, void *ddt, void *dB, void *dC, void *dz,
                                 wkv_dtype grad_dtype, float *dA, float *d_skip, float *d_dt_bias,
                                 float *d_state_in, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                 void *stream) {
  const char *fn = "wkv_ssm_scan_backward";
  REQUIRE(T >= 1, "%s: need T >= 1 (got %d)", fn, T);
  wkv::SeqParams seq;
  CHECK(dense_seq(fn, B, T, state_in, state_map, n_state, nullptr, dev_status, &seq));
  wkv::ScanBackwardParams p{};
  CHECK(scan_params(fn, seq, D, N, G, x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, in_dtype, skip, z,
                    z_stride, dt_bias, dt_softplus, &p.f));
  if (!dtype_ok(dy_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown dtype of dy %d", fn, dy_dtype);
  if (!dtype_ok(grad_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown gradient dtype %d", fn, grad_dtype);
  CHECK(token_array(fn, "dy", dy, dy_stride, D, dy_dtype));
  REQUIRE(dx && ddt && dB && dC && dA && (dz != nullptr) == (z != nullptr),
          "%s: dx, ddt, dB, dC and dA must be non-NULL, and dz given exactly when z is", fn);
  REQUIRE(aligned(dx, 16) && aligned(ddt, 16) && aligned(dB, 16) && aligned(dC, 16) && aligned(dz, 16) &&
              aligned(dA, 16) && aligned(d_skip, 4) && aligned(d_dt_bias, 4) && aligned(d_state_in, 16) &&
              aligned(d_state_out, 16) && aligned(chunk_states, 16),
          "%s: gradients and states must be 16-byte aligned", fn);
  const void *ins[] = {x, dt, z, Bm, Cm, dy}, *outs[] = {dx, ddt, dz, dB, dC};
  for (const void *o : outs)
    for (const void *i : ins) REQUIRE(!o || o != i, "%s: a gradient may not overlap an input", fn);
  const BackwardSpace w = backward_space(B, T, D, N, G, chunk_states || chunks_of(T) == 0);
  REQUIRE(workspace && aligned(workspace, 16) && workspace_bytes >= w.total * sizeof(float),
          "%s: the workspace must be 16-byte aligned and hold %zu bytes (got %zu)", fn, w.total * sizeof(float),
          workspace_bytes);
  float *ws = static_cast<float *>(workspace);
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  const bool bf16 = in_dtype == WKV_BF16;
  p.f.n_chunks = chunks_of(T);
  p.f.chunk_states = const_cast<float *>(chunk_states);
  if (!chunk_states && p.f.n_chunks > 0) {
    p.f.chunk_states = ws + w.chunks;
    wkv::ScanSsmParams states = p.f;  // the forward pass without its output
    states.nseg = wkv::scan_segments(B, T, (long)B * T, D, N, G, &states.seg_len);
    states.workspace = ws + w.carry;
    const hipError_t e = wkv::launch_ssm_scan(states, bf16, hs);
    if (e != hipSuccess) return launched(e, fn);
  }
  p.dy = {dy, (long)dy_stride};
  p.dy_bf16 = dy_dtype == WKV_BF16;
  p.d_state_out = d_state_out;
  p.dx = dx; p.ddt = ddt; p.dz = dz; p.dB = dB; p.dC = dC;
  p.grad_bf16 = grad_dtype == WKV_BF16;
  p.dA = dA; p.d_skip = d_skip; p.d_bias = d_dt_bias; p.d_state_in = d_state_in;
  p.seg_len = w.seg_len; p.nseg = w.nseg;
  p.carry = ws + w.carry; p.part = ws + w.part; p.part_bc = ws + w.part_bc;
  return launched(wkv::launch_ssm_scan_backward(p, bf16, hs), fn);
}

wkv_status wkv_ssm_scan_forward_varlen(int num_slots, int D, int N, int G, const int32_t *lengths, int max_len,
                                       int total_tokens, const void *x, int64_t x_stride, const void *dt,
                                       int64_t dt_stride, const float *A, const void *Bm, int64_t b_stride,
                                       const void *Cm, int64_t c_stride, wkv_dtype in_dtype, const float *skip,
                                       const void *z, int64_t z_stride, const float *dt_bias, int dt_softplus,
                                       void *y, wkv_dtype out_dtype, const float *state_in, float *state_out,
                                       const int32_t *state_map, int n_state, void *workspace,
                                       size_t workspace_bytes, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_ssm_scan_forward_varlen";
  wkv::SeqParams seq;
  CHECK(varlen_seq(fn, num_slots, lengths, max_len, total_tokens, state_in, state_out, state_map, n_state, dev_status, &seq));
  wkv::ScanSsmParams p;
  CHECK(scan_params(fn, seq, D, N, G, x, x_stride, dt, dt_stride, A, Bm, b_stride, Cm, c_stride, in_dtype, skip, z,
                    z_stride, dt_bias, dt_softplus, &p));
  return scan(fn, p, in_dtype, y, out_dtype, workspace, workspace_bytes, stream);
}

wkv_status wkv_state_store_write(void *data, float *scale, int n_store, wkv_store_format format,
                                 const float *states, int n_state, int64_t row, const int32_t *store_rows,
                                 const int32_t *state_rows, int count, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_state_store_write";
  wkv::StoreParams p;
  CHECK(store(fn, data, scale, n_store, format, states, n_state, row, store_rows, state_rows, count, dev_status, &p));
  if (count == 0) return ok();
  return launched(wkv::launch_store_write(p, static_cast<hipStream_t>(stream)), fn);
}

wkv_status wkv_state_store_read(const void *data, const float *scale, int n_store, wkv_store_format format,
                                float *states, int n_state, int64_t row, const int32_t *store_rows,
                                const int32_t *state_rows, int count, int32_t *dev_status, void *stream) {
  const char *fn = "wkv_state_store_read";
  wkv::StoreParams p;
  CHECK(store(fn, data, scale, n_store, format, states, n_state, row, store_rows, state_rows, count, dev_status, &p));
  if (count == 0) return ok();
  return launched(wkv::launch_store_read(p, static_cast<hipStream_t>(stream)), fn);
}

wkv_status wkv_ssm_call(wkv_ssm_op op, const int64_t *args, int count) {
  const char *fn = "wkv_ssm_call";
  REQUIRE(args, "%s: args must be non-NULL", fn);
  switch (op) {
    case WKV_OP_CONV_FORWARD: return call_words(fn, wkv_ssm_conv_forward, args, count);
    case WKV_OP_CONV_FORWARD_VARLEN: return call_words(fn, wkv_ssm_conv_forward_varlen, args, count);
    case WKV_OP_CONV_BACKWARD: return call_words(fn, wkv_ssm_conv_backward, args, count);
    case WKV_OP_SCAN_FORWARD: return call_words(fn, wkv_ssm_scan_forward, args, count);
    case WKV_OP_SCAN_FORWARD_TRAIN: return call_words(fn, wkv_ssm_scan_forward_train, args, count);
    case WKV_OP_SCAN_FORWARD_VARLEN: return call_words(fn, wkv_ssm_scan_forward_varlen, args, count);
    case WKV_OP_SCAN_BACKWARD: return call_words(fn, wkv_ssm_scan_backward, args, count);
    case WKV_OP_STORE_WRITE: return call_words(fn, wkv_state_store_write, args, count);
    case WKV_OP_STORE_READ: return call_words(fn, wkv_state_store_read, args, count);
    default: return fail(WKV_ERR_INVALID_ARG, "%s: unknown op %d", fn, op);
  }
}

}  // extern "C"
