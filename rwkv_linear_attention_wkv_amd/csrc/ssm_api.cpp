// C ABI of the state space operators: argument validation and launch.  Every
// host-checkable problem is reported before any HIP call.
#include "wkv_ssm.h"

#include "api_common.hpp"
#include "ssm.hpp"

using namespace wkv::api;

namespace {

constexpr int kMaxChannels = 1 << 24;
constexpr int kMaxStates = 64;

// Sequences and states of a dense call; `state_row` floats per state row.
wkv_status dense_seq(const char *fn, int B, int T, const float *state_in, const int32_t *state_map, int n_state,
                     float *state_out, int32_t *dev_status, wkv::SeqParams *out) {
  REQUIRE(B >= 1 && T >= 0, "%s: need B >= 1 and T >= 0 (got B=%d T=%d)", fn, B, T);
  REQUIRE(B <= kMaxGridY, "%s: B=%d exceeds %d", fn, B, kMaxGridY);
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

wkv_status conv(const char *fn, const wkv::SeqParams &seq, int D, int W, const void *x, int64_t x_stride,
                wkv_dtype in_dtype, const float *weight, const float *bias, wkv_activation act, void *y,
                wkv_dtype out_dtype, void *stream) {
  REQUIRE(D >= 1 && D <= kMaxChannels, "%s: need 1 <= D <= %d (got %d)", fn, kMaxChannels, D);
  if (W < 2 || W > 4) return fail(WKV_ERR_UNSUPPORTED, "%s: W=%d is not supported (2, 3 or 4)", fn, W);
  if (!dtype_ok(in_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown input dtype %d", fn, in_dtype);
  if (!dtype_ok(out_dtype)) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown output dtype %d", fn, out_dtype);
  if (act != WKV_ACT_NONE && act != WKV_ACT_SILU) return fail(WKV_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, act);
  if (seq.units == 0) return ok();
  REQUIRE(weight && aligned(weight, 4) && aligned(bias, 4), "%s: weight must be given; weight and bias 4-byte aligned", fn);
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
  p.nseg = wkv::conv_segments(seq.units, seq.T, D, false, &p.seg_len);
  return launched(wkv::launch_ssm_conv(p, in_dtype == WKV_BF16, static_cast<hipStream_t>(stream)), fn);
}

size_t scan_workspace(int units, int nseg, int D, int N) {
  return nseg > 1 ? sizeof(float) * (size_t)units * ((size_t)nseg * D * N + (size_t)(nseg - 1) * D) : 0;
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
  p.nseg = wkv::scan_segments(p.seq.units, p.seq.T, p.D, p.N, p.G, &p.seg_len);
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

size_t wkv_ssm_scan_workspace(int rows, int T, int D, int N, int G) {
  if (rows < 1 || T < 1 || D < 1 || N < 1 || N > kMaxStates || G < 1 || D % G) return 0;
  int len;
  return scan_workspace(rows, wkv::scan_segments(rows, T, D, N, G, &len), D, N);
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

}  // extern "C"
