// Launch arguments of the transformer block's operators (layer norm, packed
// causal attention), shared by their host entry points and kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

// Sets the calling thread's error message and returns `code` (api.hip).
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);
void clear_error();

// Launches a kernel that takes one argument struct; the error is this
// launch's own (hipGetLastError would also report an earlier call's).
template <class A>
hipError_t launch_kernel(void (*kernel)(A), int64_t grid, int block, A args, hipStream_t stream) {
  void* p[] = {&args};
  return hipLaunchKernel((const void*)kernel, dim3((unsigned)grid), dim3((unsigned)block), p, 0, stream);
}

// ------------------------------------------------------------- layer norm --
struct NormArgs {
  const void* x;
  const void* dy;       // backward only
  const void* weight;   // null: ones
  const void* bias;     // forward only; null: zeros
  void* out;            // y, or dx (null: not wanted)
  float* mean;          // written by the forward pass, read by the backward
  float* rstd;
  float* part;          // backward: per-block column sums, [blocks][2][cols]; null: not wanted
  int64_t rows;
  int64_t ld_x, ld_dy, ld_out;
  int32_t cols;
  int32_t blocks;       // backward: grid, and rows of `part`
  float eps;
};

struct NormSumArgs {
  const float* part;
  float* dweight;       // either may be null
  float* dbias;
  int32_t cols;
  int32_t blocks;
};

int norm_backward_blocks(int64_t rows, int64_t cols);
hipError_t launch_norm_forward(const NormArgs& a, bool x_bf16, bool p_bf16, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, bool x_bf16, bool p_bf16, hipStream_t stream);
hipError_t launch_norm_sum(const NormSumArgs& a, hipStream_t stream);

// -------------------------------------------------------------- attention --
// One (tokens, heads, head_dim) operand: strides in elements, head_dim
// contiguous.
struct HeadView {
  void* data;
  int64_t token;
  int64_t head;
};

struct AttnArgs {
  HeadView q, k, v, o;
  HeadView dout, dq, dk, dv;  // backward only
  float* lse;                 // (q_heads, tokens)
  float* delta;               // backward workspace: (q_heads, tokens), delta; bf16: -delta
  float* lse2;                // and again, lse / log 2; bf16: -lse / scale
  float* part;                // backward: partial dK, dV, [split][token][kv head][2][dim]; null without splits
  const int32_t* cu;          // (seqs + 1) token offsets of the packed sequences
  int64_t tokens;
  int32_t seqs;
  int32_t q_heads, kv_heads, group;
  int32_t splits;             // backward: parts a group's query heads are split into
  int32_t dim;
  float scale;
  uint32_t zero_tail;         // bit i: output i's rows behind the last sequence are set to zero
};

enum { kZeroOut = 1, kZeroLse = 2 };               // AttnArgs::zero_tail, forward
enum { kZeroDq = 1, kZeroDk = 2, kZeroDv = 4 };    // and backward

// Threads of the largest launch: one for the query rows.  (Twice as many a
// block where blocks are few do not count.)
int64_t attention_threads(int64_t tokens, int seqs, int q_heads, int dim, bool bf16);
int attention_splits(int64_t tokens, int seqs, int q_heads, int kv_heads);
hipError_t launch_attention_forward(const AttnArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_attention_backward(const AttnArgs& a, bool bf16, hipStream_t stream);

}  // namespace muon
