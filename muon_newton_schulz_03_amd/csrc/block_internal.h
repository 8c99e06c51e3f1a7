// Launch arguments of the transformer block's operators (embedding, layer
// norm, query/key norm with rotation, packed causal attention), shared by
// their host entry points and kernels.
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

constexpr int kMaxDim = 128;  // of a head

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


// ---------------------------------------------------- query and key norms --
// One side, queries or keys.
struct QkSide {
  HeadView x, out;     // out: y, or dx
  HeadView dy;         // backward only
  const void* weight;  // null: ones
  int32_t heads;
  int32_t zero_tail;   // set out's rows behind the last sequence to zero
};

struct QkArgs {
  QkSide side[2];
  const int32_t* cu;       // null: no sequences, every token counts
  const void* positions;   // null: offset within the sequence (without sequences, the token's number)
  float* part;             // backward: weight gradients of each block, [blocks][2][dim]; null: not wanted
  int64_t tokens;
  int32_t seqs;
  int32_t dim;
  int32_t rotated;         // elements of a head that turn, the first ones
  int32_t p_bf16;
  int32_t pos64;
  int32_t blocks;
  int32_t apart;           // 1: even blocks take the queries, odd ones the keys
  int32_t wide, wide_log;  // heads of a token that a wave takes at once, a power of two
  int32_t pair_lanes;      // log2 of the lanes that compute a token's angles
  float eps;
  uint64_t turns[kMaxDim / 2];  // a pair's turn per position, as a fraction of 2^64
};

struct QkSumArgs {
  const float* part;
  float* dweight[2];  // either may be null
  int32_t blocks;
  int32_t dim;
};

constexpr int kQkBlocks = 1024;  // at most: four waves a SIMD
enum { kPairHalves = 0, kPairNeighbours = 1 };
// Fills in the launch's layout: blocks, wide, pair_lanes.
void plan_qk(QkArgs& a, bool bf16, int pairs);
hipError_t launch_qk(const QkArgs& a, bool bf16, int pairs, bool backward, hipStream_t stream);
hipError_t launch_qk_sum(const QkSumArgs& a, hipStream_t stream);

// -------------------------------------------------------------- embedding --
struct EmbedArgs {
  const void* ids;
  const void* table;
  void* out;
  int64_t tokens, vocab, ld_table, ld_out;
  int32_t cols;
  int32_t id64;
  int32_t rows;    // tokens of a block
  uint32_t magic;  // 2^32 / vectors of a row, rounded up (rows > 1)
  float scale;
};
hipError_t launch_embed_forward(const EmbedArgs& a, bool table_bf16, bool out_bf16, hipStream_t stream);

struct EmbedEntry {
  uint32_t id;  // vocab: an id outside the table
  uint32_t token;
};
struct EmbedGradArgs {
  const void* ids;
  const void* dout;
  void* dtable;
  int64_t tokens, vocab, ld_dout, ld_dtable;
  int32_t cols;
  int32_t id64;
  int32_t accumulate;
  float scale;
  // workspace
  EmbedEntry* sorted;       // the tokens by id
  EmbedEntry* entry[2];     // between passes: after even ones, after odd ones
  uint32_t* hist;           // [blocks][1 << digit]
  float* part;              // [chunks][2][cols]
  // layout
  int32_t table_size;       // bytes of the table's elements
  int32_t blocks, segment;  // blocks of a pass, and tokens of each
  int32_t digit, passes;    // bits of a digit
  int32_t pass;             // this launch's
  int32_t lanes;            // that sum a row's vectors
  int32_t chunk;            // sorted tokens that a block sums
  int32_t direct;           // one launch does it all; segment: rows of a block
  int32_t stream;           // dout is larger than what the caches keep
};
constexpr int kEmbedEach = 8;         // sorted tokens that a row's lanes sum
constexpr int kFewEach = 4;           // the same while blocks are few
constexpr int kDirect = 512;          // tokens that the one launch takes
constexpr int kDirectRows = 1024;     // of a block
constexpr int kMaxDigit = 9;
constexpr int64_t kOneBlock = 8192;    // tokens that one block sorts
// Fills in the layout from tokens, vocab and cols.
void plan_embed(EmbedGradArgs& a, bool table_bf16, bool out_bf16);
hipError_t launch_embed_backward(const EmbedGradArgs& a, bool table_bf16, bool out_bf16, hipStream_t stream);

}  // namespace muon
