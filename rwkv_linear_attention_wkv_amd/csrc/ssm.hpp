// Host-side launchers of the state space kernels (internal to libwkv.so).
// Arguments have been validated by the C ABI layer before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wkv {

// The sequences of a call and their state rows.  Dense: unit b holds tokens
// [b*T, b*T + T), reads state row state_map[b] (or b, or the one shared row) and writes row b.
// Varlen (lengths given): unit s holds lengths[s] packed tokens and reads and writes row
// state_map[s] (or s).
struct SeqParams {
  int units;
  int T;  // tokens of every row; varlen: the host's bound on every length
  const int32_t *lengths;
  long total_tokens;
  const float *state_in;
  const int32_t *state_map;
  int n_state;
  float *state_out;
  int32_t *dev_status;
};

constexpr long kMaxStride = 1 << 22;  // elements between token rows

// A token array: element (token t of the call, column c) at base[t * stride + c].
struct TokenArray {
  const void *base;
  long stride;
};

struct ConvParams {
  SeqParams seq;
  int D, W;
  TokenArray x;
  const float *weight, *bias;  // [D, W], [D] or null
  bool silu;
  void *y;  // [tokens, D], bf16 when y_bf16 (backward: dx)
  bool y_bf16;
  // backward
  TokenArray dy;
  bool dy_bf16;
  const float *d_state_out;  // gradient of the final state, or null
  float *d_state_in;         // or null
  float *partial;            // [units * nseg, W + 1, D] sums of one segment: dweight taps, dbias
  float *d_weight, *d_bias;
  int seg_len, nseg;  // tokens of one workgroup's walk
};

hipError_t launch_ssm_conv(const ConvParams &p, bool bf16, hipStream_t s);
hipError_t launch_ssm_conv_backward(const ConvParams &p, bool bf16, hipStream_t s);
int conv_segments(int T, long total, int D, bool bf16, bool backward, int *seg_len);

struct ScanSsmParams {
  SeqParams seq;
  int D, N, G;
  TokenArray x, dt, z, Bm, Cm;  // z.base may be null
  const float *A, *skip, *dt_bias;
  bool softplus;
  void *y;
  bool y_bf16;
  // null, or [units, n_chunks, D, N]: the state at the start of each 16-token chunk but the first;
  // with y null these are all that is computed
  float *chunk_states;
  int n_chunks;
  int seg_len, nseg;  // tokens of a segment; with nseg > 1 the workspace holds the segments' states
  float *workspace;   // [units][nseg][D][N] states, [units][nseg - 1][D] sums of delta
};

constexpr int kScanChunk = 16;  // tokens between saved states
constexpr int kScanShort = 8;   // calls of at most this many tokens a sequence take the kernel without tiles
constexpr int kScanSplit = 64;  // no sequence of at most this many tokens is split

// Lanes that share a channel, four states each.
inline int lanes_of(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

int best_segments(long groups, int T, int step, double shared, double carry, int start, int *seg_len);
int scan_segments(int units, int T, long total, int D, int N, int G, int *seg_len);
hipError_t launch_ssm_scan(const ScanSsmParams &p, bool bf16, hipStream_t s);

// The scan's backward pass, dense rows.
struct ScanBackwardParams {
  ScanSsmParams f;  // the forward call: its sequences (state_out unused), arrays and chunk states
  TokenArray dy;
  bool dy_bf16;
  const float *d_state_out;  // [B, D, N] gradient of the final state, or null
  void *dx, *ddt, *dz, *dB, *dC;  // contiguous, bf16 when grad_bf16
  bool grad_bf16;
  float *dA, *d_skip, *d_bias, *d_state_in;
  int seg_len, nseg;
  // workspace
  float *carry;     // [B][nseg][D][N] states' gradients at the start of a segment from one of zero at
                    // its end, then [B][nseg][D] sums of delta
  float *part;      // [B * nseg][D * N + 2 * D]: a segment's shares of dA, d_skip and d_bias
  float *part_bc;   // [blocks of a group][B * T][G][2 N]: dB, dC of one block of channels
};

int backward_segments(int units, int T, int D, int N, int G, int *seg_len);
int backward_blocks(int D, int N, int G);  // blocks of channels of a group
hipError_t launch_ssm_scan_backward(const ScanBackwardParams &p, bool bf16, hipStream_t s);

// The 8-bit state store: rows of `row` values in groups of 64 with one scale each.
struct StoreParams {
  void *data;    // [n_store, row] codes
  float *scale;  // [n_store, ceil(row / 64)]
  float *states; // [n_state, row]
  const int32_t *store_rows, *state_rows;  // [count] or null (identity)
  int n_store, n_state, count;
  long row;
  bool e4m3;
  int32_t *dev_status;
};

hipError_t launch_store_write(const StoreParams &p, hipStream_t s);
hipError_t launch_store_read(const StoreParams &p, hipStream_t s);

}  // namespace wkv
