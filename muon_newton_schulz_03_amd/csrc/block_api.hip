// Host side of the transformer block's operators: argument checks, workspace
// layout and launches of layer norm and packed causal attention.  See
// include/muon.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/muon.h"
#include "block_internal.h"
#include "muon_internal.h"

using namespace muon;

namespace {

constexpr int64_t kMaxCols = 1 << 20;
constexpr int64_t kMaxRows = (int64_t)1 << 40;
constexpr int64_t kMaxStride = (int64_t)1 << 31;
constexpr double kMaxElements = 0x1p56;  // byte offsets fit 64 bits
constexpr int64_t kMaxTokenStride = 1 << 24;  // a 64-row tile stays within 32-bit byte offsets
constexpr int64_t kMaxTokens = 0x7FFFFF00;
constexpr int64_t kMaxThreads = 0xFFFFFFFF;  // of one launch
constexpr int kMaxSeqs = 1 << 24;
constexpr int kMaxHeads = 1 << 16;
constexpr int kMaxDim = 128;
constexpr float kMinScale = 0x1p-60f;  // lse / scale stays finite
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool misaligned(const void* p, size_t n) { return (uintptr_t)p % n != 0; }
int elem_size(int dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

// ---------------------------------------------------------------- overlap --
// The bytes of an operand: n x m pieces of `width` bytes, `step` and `inner`
// bytes apart.  A step of 0 repeats a piece.
struct Area {
  int64_t at, n, step, m, inner, width;
};
Area flat(const void* p, size_t bytes) { return Area{(int64_t)(uintptr_t)p, 1, 0, 1, 0, p ? (int64_t)bytes : 0}; }
Area area(const void* p, int64_t n, int64_t step, int64_t m, int64_t inner, int64_t width) {
  if (n == 1 || step == 0) n = 1, step = 0;
  if (m == 1 || inner == 0) m = 1, inner = 0;
  return Area{(int64_t)(uintptr_t)p, n, step, m, inner, p && n ? width : 0};
}
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Whether two operands share a byte.  Exact for operands whose steps agree
// (slices of one buffer; one piece agrees with everything) or whose pieces of
// a row are few; others count as sharing where their extents meet.
bool meet(const Area& a, const Area& b) {
  if (!a.width || !b.width) return false;
  const int64_t ea = (a.m - 1) * a.inner + a.width, eb = (b.m - 1) * b.inner + b.width;  // a row's extent
  const int64_t apart = b.at - a.at;
  if (apart >= (a.n - 1) * a.step + ea || -apart >= (b.n - 1) * b.step + eb) return false;
  const int64_t step = a.step ? a.step : b.step, inner = a.inner ? a.inner : b.inner;
  if (a.step && b.step && a.step != b.step) return true;
  if (step) {  // columns of one buffer: b's rows start r bytes into a's, or between them
    const int64_t r = apart - floor_div(apart, step) * step;
    if (r >= ea && step - r >= eb) return false;
  }
  // a piece of b lies x + di step behind one of a, di from -(a.n - 1) to b.n - 1
  auto hit = [&](int64_t x) {
    if (!step) return x < a.width && -x < b.width;
    const int64_t lo = floor_div(-b.width - x, step) + 1, hi = -floor_div(x - a.width, step) - 1;
    return (lo > -(a.n - 1) ? lo : -(a.n - 1)) <= (hi < b.n - 1 ? hi : b.n - 1);
  };
  if (!a.inner || !b.inner || a.inner == b.inner) {
    for (int64_t j = -(a.m - 1); j < b.m; ++j)
      if (hit(apart + j * inner)) return true;
    return false;
  }
  if (a.m * b.m > 1 << 14) return true;
  for (int64_t i = 0; i < a.m; ++i)
    for (int64_t j = 0; j < b.m; ++j)
      if (hit(apart + j * b.inner - i * a.inner)) return true;
  return false;
}

struct Operand {
  const char* name;
  Area area;
};
// The first `written` operands share no byte with any other.
int check_apart(const char* what, const Operand* ops, int written, int n) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (meet(ops[i].area, ops[j].area))
        return fail(MUON_E_INVAL, "%s: %s overlaps %s (or lies between its rows with other strides)", what, ops[i].name,
                    ops[j].name);
  return MUON_OK;
}

// ------------------------------------------------------------- layer norm --
int check_norm(const muon_layernorm_desc* d) {
  if (!d) return fail(MUON_E_INVAL, "layer norm descriptor is NULL");
  if (d->rows < 0 || d->rows > kMaxRows)
    return fail(MUON_E_INVAL, "layer norm: rows=%lld outside [0, 2^40]", (long long)d->rows);
  if (d->cols <= 0 || d->cols > kMaxCols)
    return fail(MUON_E_INVAL, "layer norm: cols=%lld outside [1, 2^20]", (long long)d->cols);
  const int64_t lds[] = {d->ld_x, d->ld_y, d->ld_dy, d->ld_dx};
  const char* names[] = {"ld_x", "ld_y", "ld_dy", "ld_dx"};
  for (int i = 0; i < 4; ++i)
    if (lds[i] != 0 && (lds[i] < d->cols || lds[i] > kMaxStride))
      return fail(MUON_E_INVAL, "layer norm: %s=%lld is below cols=%lld or above 2^31", names[i], (long long)lds[i],
                  (long long)d->cols);
  if (d->x_dtype != MUON_DTYPE_F32 && d->x_dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "layer norm: x_dtype %d unsupported", d->x_dtype);
  if (d->p_dtype != MUON_DTYPE_F32 && d->p_dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "layer norm: p_dtype %d unsupported", d->p_dtype);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps))
    return fail(MUON_E_INVAL, "layer norm: eps must be finite and not negative");
  if (d->reserved != 0) return fail(MUON_E_INVAL, "layer norm: reserved field must be 0");
  for (int i = 0; i < 4; ++i)
    if ((double)d->rows * (double)(lds[i] ? lds[i] : d->cols) > kMaxElements)
      return fail(MUON_E_INVAL, "layer norm: rows=%lld of %s exceed any memory", (long long)d->rows, names[i]);
  return MUON_OK;
}

size_t norm_workspace(const muon_layernorm_desc* d) {
  return align_up((size_t)norm_backward_blocks(d->rows, d->cols) * 2 * (size_t)d->cols * sizeof(float));
}

int64_t ld_of(int64_t ld, int64_t cols) { return ld ? ld : cols; }
Area rows_area(const muon_layernorm_desc* d, const void* p, int64_t ld) {
  const int es = elem_size(d->x_dtype);
  return area(p, d->rows, ld_of(ld, d->cols) * es, 1, 0, d->cols * es);
}

// -------------------------------------------------------------- attention --
int check_attention(const muon_attention_desc* d) {
  if (!d) return fail(MUON_E_INVAL, "attention descriptor is NULL");
  if (d->tokens < 0 || d->tokens > kMaxTokens)
    return fail(MUON_E_INVAL, "attention: tokens=%lld outside [0, %lld]", (long long)d->tokens, (long long)kMaxTokens);
  if (d->seqs < 0 || d->seqs > kMaxSeqs)
    return fail(MUON_E_INVAL, "attention: seqs=%d outside [0, %d]", d->seqs, kMaxSeqs);
  if (d->q_heads <= 0 || d->kv_heads <= 0 || d->q_heads > kMaxHeads || d->q_heads % d->kv_heads)
    return fail(MUON_E_INVAL, "attention: q_heads=%d must be a positive multiple of kv_heads=%d, at most %d", d->q_heads,
                d->kv_heads, kMaxHeads);
  if (d->head_dim <= 0 || d->head_dim > kMaxDim || d->head_dim % 8)
    return fail(MUON_E_UNSUPPORTED, "attention: head_dim=%d must be a multiple of 8, at most %d", d->head_dim, kMaxDim);
  if (d->dtype != MUON_DTYPE_F32 && d->dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "attention: dtype %d unsupported", d->dtype);
  if (!(d->scale >= kMinScale && d->scale <= 1.f / kMinScale))
    return fail(MUON_E_INVAL, "attention: scale %g outside [2^-60, 2^60]", d->scale);
  if (d->reserved != 0) return fail(MUON_E_INVAL, "attention: reserved field must be 0");
  if (attention_threads(d->tokens, d->seqs, d->q_heads, d->head_dim, d->dtype == MUON_DTYPE_BF16) > kMaxThreads)
    return fail(MUON_E_UNSUPPORTED, "attention: %lld tokens, %d sequences and %d heads exceed one launch's grid",
                (long long)d->tokens, d->seqs, d->q_heads);
  return MUON_OK;
}

int check_heads(const muon_attention_desc* d, const muon_heads* v, const char* name, int heads, bool written,
                HeadView* out) {
  if (!v || !v->data) return fail(MUON_E_INVAL, "attention: %s is NULL", name);
  const int es = elem_size(d->dtype);
  // a stride that no address uses does not matter
  const int64_t token = d->tokens > 1 ? v->token_stride : 0, head = heads > 1 ? v->head_stride : 0;
  if (token < 0 || head < 0 || token > kMaxTokenStride || head > kMaxStride)
    return fail(MUON_E_INVAL, "attention: %s: strides %lld, %lld outside [0, 2^24] and [0, 2^31]", name,
                (long long)token, (long long)head);
  if (misaligned(v->data, 16) || token * es % 16 || head * es % 16)
    return fail(MUON_E_UNSUPPORTED, "attention: %s must start, and step from token to token and head to head, at "
                "multiples of 16 bytes", name);
  if (written) {
    const int64_t dim = d->head_dim;
    const bool by_token = (d->tokens <= 1 || token >= (heads - 1) * head + dim) && (heads <= 1 || head >= dim);
    const bool by_head = (heads <= 1 || head >= (d->tokens - 1) * token + dim) && (d->tokens <= 1 || token >= dim);
    if (!by_token && !by_head)
      return fail(MUON_E_INVAL, "attention: rows of the output %s overlap (strides %lld, %lld)", name, (long long)token,
                  (long long)head);
  }
  *out = HeadView{v->data, token, head};
  return MUON_OK;
}

size_t attention_part_bytes(const muon_attention_desc* d, int splits) {
  return splits > 1 ? (size_t)splits * d->tokens * d->kv_heads * 2 * d->head_dim * sizeof(float) : 0;
}
int splits_of(const muon_attention_desc* d) {
  return attention_splits(d->tokens, d->seqs, d->q_heads, d->kv_heads);
}
size_t lse_bytes(const muon_attention_desc* d) { return (size_t)d->q_heads * d->tokens * sizeof(float); }
size_t attention_row_bytes(const muon_attention_desc* d) {  // one fp32 per query row
  return align_up(lse_bytes(d));
}
size_t attention_workspace(const muon_attention_desc* d) {
  return 2 * attention_row_bytes(d) + align_up(attention_part_bytes(d, splits_of(d))) +
         kAlign;  // never 0, which means an error
}

Area heads_area(const muon_attention_desc* d, const HeadView& v, int heads) {
  const int es = elem_size(d->dtype);
  return area(v.data, d->tokens, v.token * es, heads, v.head * es, d->head_dim * es);
}

AttnArgs common_args(const muon_attention_desc* d, const int32_t* cu, uint32_t flags) {
  AttnArgs a{};
  a.cu = cu;
  a.tokens = d->tokens;
  a.seqs = d->seqs;
  a.q_heads = d->q_heads;
  a.kv_heads = d->kv_heads;
  a.group = d->q_heads / d->kv_heads;
  a.splits = 1;
  a.dim = d->head_dim;
  a.scale = d->scale;
  a.zero_tail = flags;
  return a;
}

}  // namespace

extern "C" {

int muon_layernorm_forward(const muon_layernorm_desc* d, const void* x, const void* weight, const void* bias, void* y,
                           float* mean, float* rstd, void* hip_stream) {
  clear_error();
  if (int rc = check_norm(d)) return rc;
  if (d->rows == 0) return MUON_OK;
  if (!x || !y || !mean || !rstd) return fail(MUON_E_INVAL, "layer norm: x, y, mean or rstd is NULL");
  const int es = elem_size(d->x_dtype), ps = elem_size(d->p_dtype);
  if (misaligned(x, es) || misaligned(y, es) || misaligned(weight, ps) || misaligned(bias, ps) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return fail(MUON_E_INVAL, "layer norm: pointer not aligned to its element size");
  const Operand ops[] = {{"y", rows_area(d, y, d->ld_y)},     {"mean", flat(mean, d->rows * 4)},
                         {"rstd", flat(rstd, d->rows * 4)},   {"x", rows_area(d, x, d->ld_x)},
                         {"weight", flat(weight, d->cols * ps)}, {"bias", flat(bias, d->cols * ps)}};
  if (int rc = check_apart("layer norm", ops, 3, 6)) return rc;
  NormArgs a{};
  a.x = x, a.weight = weight, a.bias = bias, a.out = y, a.mean = mean, a.rstd = rstd;
  a.rows = d->rows, a.cols = (int32_t)d->cols, a.eps = d->eps;
  a.ld_x = ld_of(d->ld_x, d->cols), a.ld_out = ld_of(d->ld_y, d->cols);
  const hipError_t e = launch_norm_forward(a, d->x_dtype == MUON_DTYPE_BF16, d->p_dtype == MUON_DTYPE_BF16,
                                           (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "layer norm forward launch");
}

size_t muon_layernorm_workspace_size(const muon_layernorm_desc* d) {
  clear_error();
  if (check_norm(d)) return 0;
  return norm_workspace(d) + kAlign;
}

int muon_layernorm_backward(const muon_layernorm_desc* d, const void* dy, const void* x, const void* weight,
                            const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                            void* workspace, size_t ws_bytes, void* hip_stream) {
  clear_error();
  if (int rc = check_norm(d)) return rc;
  if (d->rows > 0 && !dx && !dweight && !dbias)
    return fail(MUON_E_INVAL, "layer norm: dx, dweight and dbias are all NULL");
  const int es = elem_size(d->x_dtype), ps = elem_size(d->p_dtype);
  if (d->rows > 0 && (!dy || !x || !mean || !rstd))
    return fail(MUON_E_INVAL, "layer norm: dy, x, mean or rstd is NULL");
  if (misaligned(x, es) || misaligned(dy, es) || misaligned(dx, es) || misaligned(weight, ps) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(dweight, 4) || misaligned(dbias, 4))
    return fail(MUON_E_INVAL, "layer norm: pointer not aligned to its element size");
  const bool sums = dweight || dbias;
  if (sums) {
    if (!workspace) return fail(MUON_E_WORKSPACE, "layer norm: workspace is NULL");
    if (misaligned(workspace, kAlign)) return fail(MUON_E_WORKSPACE, "layer norm: workspace is not 256-byte aligned");
    if (ws_bytes < norm_workspace(d))
      return fail(MUON_E_WORKSPACE, "layer norm: workspace has %zu bytes, the call needs %zu", ws_bytes,
                  norm_workspace(d));
  }
  const Operand ops[] = {{"dx", rows_area(d, dx, d->ld_dx)},
                         {"dweight", flat(dweight, d->cols * 4)},
                         {"dbias", flat(dbias, d->cols * 4)},
                         {"workspace", flat(sums ? workspace : nullptr, norm_workspace(d))},
                         {"dy", rows_area(d, dy, d->ld_dy)},
                         {"x", rows_area(d, x, d->ld_x)},
                         {"mean", flat(mean, d->rows * 4)},
                         {"rstd", flat(rstd, d->rows * 4)},
                         {"weight", flat(weight, d->cols * ps)}};
  if (int rc = check_apart("layer norm", ops, 4, 9)) return rc;
  NormArgs a{};
  a.x = x, a.dy = dy, a.weight = weight, a.out = dx;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.part = sums ? (float*)workspace : nullptr;
  a.rows = d->rows, a.cols = (int32_t)d->cols, a.eps = d->eps;
  a.ld_x = ld_of(d->ld_x, d->cols), a.ld_dy = ld_of(d->ld_dy, d->cols), a.ld_out = ld_of(d->ld_dx, d->cols);
  a.blocks = norm_backward_blocks(d->rows, d->cols);
  hipError_t e = hipSuccess;
  if (d->rows > 0)
    e = launch_norm_backward(a, d->x_dtype == MUON_DTYPE_BF16, d->p_dtype == MUON_DTYPE_BF16,
                             (hipStream_t)hip_stream);
  if (e == hipSuccess && sums)
    e = launch_norm_sum(NormSumArgs{a.part, dweight, dbias, a.cols, d->rows > 0 ? a.blocks : 0},
                        (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "layer norm backward launch");
}

int muon_attention_forward(const muon_attention_desc* d, const int32_t* cu_seqlens, const muon_heads* q,
                           const muon_heads* k, const muon_heads* v, const muon_heads* out, float* lse, uint32_t flags,
                           void* hip_stream) {
  clear_error();
  if (int rc = check_attention(d)) return rc;
  if (flags & ~(uint32_t)(MUON_ATTENTION_ZERO_OUT | MUON_ATTENTION_ZERO_LSE))
    return fail(MUON_E_INVAL, "attention: unknown flags 0x%x", flags);
  if (d->tokens == 0) return MUON_OK;
  if (!cu_seqlens || misaligned(cu_seqlens, 4)) return fail(MUON_E_INVAL, "attention: cu_seqlens is NULL or misaligned");
  if (!lse || misaligned(lse, 4)) return fail(MUON_E_INVAL, "attention: lse is NULL or misaligned");
  AttnArgs a = common_args(d, cu_seqlens, flags);
  int rc = check_heads(d, q, "q", d->q_heads, false, &a.q);
  if (!rc) rc = check_heads(d, k, "k", d->kv_heads, false, &a.k);
  if (!rc) rc = check_heads(d, v, "v", d->kv_heads, false, &a.v);
  if (!rc) rc = check_heads(d, out, "out", d->q_heads, true, &a.o);
  if (rc) return rc;
  const Operand ops[] = {{"out", heads_area(d, a.o, d->q_heads)}, {"lse", flat(lse, lse_bytes(d))},
                         {"q", heads_area(d, a.q, d->q_heads)},   {"k", heads_area(d, a.k, d->kv_heads)},
                         {"v", heads_area(d, a.v, d->kv_heads)},
                         {"cu_seqlens", flat(cu_seqlens, ((size_t)d->seqs + 1) * 4)}};
  if ((rc = check_apart("attention", ops, 2, 6))) return rc;
  a.lse = lse;
  const hipError_t e = launch_attention_forward(a, d->dtype == MUON_DTYPE_BF16, (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "attention forward launch");
}

size_t muon_attention_workspace_size(const muon_attention_desc* d) {
  clear_error();
  if (check_attention(d)) return 0;
  return attention_workspace(d);
}

int muon_attention_backward(const muon_attention_desc* d, const int32_t* cu_seqlens, const muon_heads* dout,
                            const muon_heads* q, const muon_heads* k, const muon_heads* v, const muon_heads* out,
                            const float* lse, const muon_heads* dq, const muon_heads* dk, const muon_heads* dv,
                            uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream) {
  clear_error();
  if (int rc = check_attention(d)) return rc;
  if (flags & ~(uint32_t)(MUON_ATTENTION_ZERO_DQ | MUON_ATTENTION_ZERO_DK | MUON_ATTENTION_ZERO_DV))
    return fail(MUON_E_INVAL, "attention: unknown flags 0x%x", flags);
  if (d->tokens == 0) return MUON_OK;
  if (!cu_seqlens || misaligned(cu_seqlens, 4)) return fail(MUON_E_INVAL, "attention: cu_seqlens is NULL or misaligned");
  if (!lse || misaligned(lse, 4)) return fail(MUON_E_INVAL, "attention: lse is NULL or misaligned");
  AttnArgs a = common_args(d, cu_seqlens, flags);
  int rc = check_heads(d, dout, "dout", d->q_heads, false, &a.dout);
  if (!rc) rc = check_heads(d, q, "q", d->q_heads, false, &a.q);
  if (!rc) rc = check_heads(d, k, "k", d->kv_heads, false, &a.k);
  if (!rc) rc = check_heads(d, v, "v", d->kv_heads, false, &a.v);
  if (!rc) rc = check_heads(d, out, "out", d->q_heads, false, &a.o);
  if (!rc) rc = check_heads(d, dq, "dq", d->q_heads, true, &a.dq);
  if (!rc) rc = check_heads(d, dk, "dk", d->kv_heads, true, &a.dk);
  if (!rc) rc = check_heads(d, dv, "dv", d->kv_heads, true, &a.dv);
  if (rc) return rc;
  if (!workspace) return fail(MUON_E_WORKSPACE, "attention: workspace is NULL");
  if (misaligned(workspace, kAlign)) return fail(MUON_E_WORKSPACE, "attention: workspace is not 256-byte aligned");
  if (ws_bytes < attention_workspace(d))
    return fail(MUON_E_WORKSPACE, "attention: workspace has %zu bytes, the call needs %zu", ws_bytes,
                attention_workspace(d));
  const Operand ops[] = {{"dq", heads_area(d, a.dq, d->q_heads)},    {"dk", heads_area(d, a.dk, d->kv_heads)},
                         {"dv", heads_area(d, a.dv, d->kv_heads)},
                         {"workspace", flat(workspace, attention_workspace(d))},
                         {"dout", heads_area(d, a.dout, d->q_heads)}, {"q", heads_area(d, a.q, d->q_heads)},
                         {"k", heads_area(d, a.k, d->kv_heads)},     {"v", heads_area(d, a.v, d->kv_heads)},
                         {"out", heads_area(d, a.o, d->q_heads)},    {"lse", flat(lse, lse_bytes(d))},
                         {"cu_seqlens", flat(cu_seqlens, ((size_t)d->seqs + 1) * 4)}};
  if ((rc = check_apart("attention", ops, 4, 11))) return rc;
  a.lse = const_cast<float*>(lse);
  a.splits = splits_of(d);
  a.delta = (float*)workspace;
  a.lse2 = (float*)((char*)workspace + attention_row_bytes(d));
  a.part = a.splits > 1 ? (float*)((char*)workspace + 2 * attention_row_bytes(d)) : nullptr;
  const hipError_t e = launch_attention_backward(a, d->dtype == MUON_DTYPE_BF16, (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "attention backward launch");
}

}  // extern "C"
