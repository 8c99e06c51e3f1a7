// Host side of the transformer block's operators: argument checks, workspace
// layout and launches of the embedding, layer norm, query/key norm with
// rotation and packed causal attention.  See
// include/muon.h for the contract of every entry point.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

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
constexpr int64_t kMaxIds = 1 << 30;
constexpr double kMaxFrequency = 64.;  // radians a position
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

// One (tokens, heads, head_dim) operand of the operator `what`.
struct HeadShape {
  const char* what;
  int64_t tokens;
  int dim, dtype;
};
int check_heads(const HeadShape& d, const muon_heads* v, const char* name, int heads, bool written, HeadView* out) {
  if (!v || !v->data) return fail(MUON_E_INVAL, "%s: %s is NULL", d.what, name);
  const int es = elem_size(d.dtype);
  // a stride that no address uses does not matter
  const int64_t token = d.tokens > 1 ? v->token_stride : 0, head = heads > 1 ? v->head_stride : 0;
  if (token < 0 || head < 0 || token > kMaxTokenStride || head > kMaxStride)
    return fail(MUON_E_INVAL, "%s: %s: strides %lld, %lld outside [0, 2^24] and [0, 2^31]", d.what, name,
                (long long)token, (long long)head);
  if (misaligned(v->data, 16) || token * es % 16 || head * es % 16)
    return fail(MUON_E_UNSUPPORTED, "%s: %s must start, and step from token to token and head to head, at "
                "multiples of 16 bytes", d.what, name);
  if (written) {
    const int64_t dim = d.dim;
    const bool by_token = (d.tokens <= 1 || token >= (heads - 1) * head + dim) && (heads <= 1 || head >= dim);
    const bool by_head = (heads <= 1 || head >= (d.tokens - 1) * token + dim) && (d.tokens <= 1 || token >= dim);
    if (!by_token && !by_head)
      return fail(MUON_E_INVAL, "%s: rows of the output %s overlap (strides %lld, %lld)", d.what, name,
                  (long long)token, (long long)head);
  }
  *out = HeadView{v->data, token, head};
  return MUON_OK;
}
Area heads_area(const HeadShape& d, const HeadView& v, int heads) {
  const int es = elem_size(d.dtype);
  return area(v.data, d.tokens, v.token * es, heads, v.head * es, d.dim * es);
}
HeadShape shape_of(const muon_attention_desc* d) { return HeadShape{"attention", d->tokens, d->head_dim, d->dtype}; }

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

// ---------------------------------------------------- query and key norms --
int check_qk(const muon_qk_norm_desc* d, const muon_rotation* r) {
  if (!d) return fail(MUON_E_INVAL, "query/key norm descriptor is NULL");
  if (d->tokens < 0 || d->tokens > kMaxTokens)
    return fail(MUON_E_INVAL, "query/key norm: tokens=%lld outside [0, %lld]", (long long)d->tokens,
                (long long)kMaxTokens);
  if (d->seqs < 0 || d->seqs > kMaxSeqs)
    return fail(MUON_E_INVAL, "query/key norm: seqs=%d outside [0, %d]", d->seqs, kMaxSeqs);
  if (d->q_heads <= 0 || d->k_heads <= 0 || d->q_heads > kMaxHeads || d->k_heads > kMaxHeads)
    return fail(MUON_E_INVAL, "query/key norm: q_heads=%d or k_heads=%d outside [1, %d]", d->q_heads, d->k_heads,
                kMaxHeads);
  if (d->head_dim <= 0 || d->head_dim > kMaxDim || d->head_dim % 8)
    return fail(MUON_E_UNSUPPORTED, "query/key norm: head_dim=%d must be a multiple of 8, at most %d", d->head_dim,
                kMaxDim);
  if (d->dtype != MUON_DTYPE_F32 && d->dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "query/key norm: dtype %d unsupported", d->dtype);
  if (d->p_dtype != MUON_DTYPE_F32 && d->p_dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "query/key norm: p_dtype %d unsupported", d->p_dtype);
  if (d->position_dtype != MUON_INDEX_I32 && d->position_dtype != MUON_INDEX_I64)
    return fail(MUON_E_UNSUPPORTED, "query/key norm: position_dtype %d unsupported", d->position_dtype);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps))
    return fail(MUON_E_INVAL, "query/key norm: eps must be finite and not negative");
  if (d->reserved != 0) return fail(MUON_E_INVAL, "query/key norm: reserved field must be 0");
  if (!r) return MUON_OK;
  if (r->dim < 0 || r->dim > d->head_dim || r->dim % 8)
    return fail(MUON_E_UNSUPPORTED, "query/key norm: a rotation of %d elements must be a multiple of 8, at most "
                "head_dim=%d", r->dim, d->head_dim);
  if (r->pairs != MUON_PAIRS_HALVES && r->pairs != MUON_PAIRS_NEIGHBOURS)
    return fail(MUON_E_INVAL, "query/key norm: pairs %d unknown", r->pairs);
  if (r->dim > 0 && !r->frequencies) return fail(MUON_E_INVAL, "query/key norm: frequencies is NULL");
  for (int i = 0; i < r->dim / 2; ++i)
    if (!(std::fabs(r->frequencies[i]) <= kMaxFrequency))
      return fail(MUON_E_INVAL, "query/key norm: frequency %g of pair %d outside [-%g, %g]", r->frequencies[i], i,
                  kMaxFrequency, kMaxFrequency);
  return MUON_OK;
}

// A frequency in radians (at most 64) as the fraction of a turn, in units of
// 2^-64, modulo whole turns, which no position sees.  In integers: the mantissa
// times 2 / pi in units of 2^-64, shifted to its place and rounded.  (32 of
// them took 9 us in long doubles, this way 0.5.)
uint64_t turn_of(double frequency) {
  constexpr uint64_t kTwoOverPi = 0xA2F9836E4E44152Aull;
  uint64_t bits;
  std::memcpy(&bits, &frequency, sizeof bits);
  // frequency / 2 pi 2^64 = mantissa 2^(exponent - 1075) (2 / pi) 2^64 / 4
  const int shift = 1077 - (int)(bits >> 52 & 0x7FF);  // at least 48
  if (shift > 118) return 0;
  const uint64_t mantissa = (bits & 0xFFFFFFFFFFFFFull) | 1ull << 52;
  const unsigned __int128 product = (unsigned __int128)mantissa * kTwoOverPi;
  const uint64_t turn = (uint64_t)((product + ((unsigned __int128)1 << (shift - 1))) >> shift);
  return bits >> 63 ? 0 - turn : turn;
}

size_t qk_workspace(const muon_qk_norm_desc* d) { return align_up((size_t)kQkBlocks * 2 * d->head_dim * sizeof(float)); }

// What both calls share: the views, the rotation and the split over blocks.
int qk_args(const muon_qk_norm_desc* d, const muon_rotation* r, const int32_t* cu, const void* positions,
            uint32_t flags, const muon_heads* q, const muon_heads* k, const muon_heads* oq, const muon_heads* ok,
            const char* nq, const char* nk, const void* q_weight, const void* k_weight, QkArgs* a) {
  if (flags & ~(uint32_t)(MUON_QK_ZERO_Q | MUON_QK_ZERO_K))
    return fail(MUON_E_INVAL, "query/key norm: unknown flags 0x%x", flags);
  if (misaligned(cu, 4)) return fail(MUON_E_INVAL, "query/key norm: cu_seqlens is misaligned");
  if (misaligned(positions, d->position_dtype == MUON_INDEX_I64 ? 8 : 4))
    return fail(MUON_E_INVAL, "query/key norm: positions are misaligned");
  const int ps = elem_size(d->p_dtype);
  if (misaligned(q_weight, ps) || misaligned(k_weight, ps))
    return fail(MUON_E_INVAL, "query/key norm: a weight is not aligned to its element size");
  const HeadShape shape{"query/key norm", d->tokens, d->head_dim, d->dtype};
  int rc = check_heads(shape, q, "q", d->q_heads, false, &a->side[0].x);
  if (!rc) rc = check_heads(shape, k, "k", d->k_heads, false, &a->side[1].x);
  if (!rc) rc = check_heads(shape, oq, nq, d->q_heads, true, &a->side[0].out);
  if (!rc) rc = check_heads(shape, ok, nk, d->k_heads, true, &a->side[1].out);
  if (rc) return rc;
  a->side[0].weight = q_weight, a->side[1].weight = k_weight;
  a->side[0].heads = d->q_heads, a->side[1].heads = d->k_heads;
  a->side[0].zero_tail = (flags & MUON_QK_ZERO_Q) != 0, a->side[1].zero_tail = (flags & MUON_QK_ZERO_K) != 0;
  a->cu = cu, a->positions = positions;
  a->tokens = d->tokens, a->seqs = d->seqs, a->dim = d->head_dim;
  a->rotated = r ? r->dim : 0;
  a->p_bf16 = d->p_dtype == MUON_DTYPE_BF16, a->pos64 = d->position_dtype == MUON_INDEX_I64;
  a->eps = d->eps;
  for (int i = 0; i < a->rotated / 2; ++i) a->turns[i] = turn_of(r->frequencies[i]);
  return MUON_OK;
}

// -------------------------------------------------------------- embedding --
int check_embedding(const muon_embedding_desc* d) {
  if (!d) return fail(MUON_E_INVAL, "embedding descriptor is NULL");
  if (d->tokens < 0 || d->tokens > kMaxIds)
    return fail(MUON_E_INVAL, "embedding: tokens=%lld outside [0, 2^30]", (long long)d->tokens);
  if (d->vocab <= 0 || d->vocab >= kMaxIds)
    return fail(MUON_E_INVAL, "embedding: vocab=%lld outside [1, 2^30)", (long long)d->vocab);
  if (d->cols <= 0 || d->cols > kMaxCols)
    return fail(MUON_E_INVAL, "embedding: cols=%lld outside [1, 2^20]", (long long)d->cols);
  const int64_t lds[] = {d->ld_table, d->ld_out};
  const char* names[] = {"ld_table", "ld_out"};
  for (int i = 0; i < 2; ++i)
    if (lds[i] != 0 && (lds[i] < d->cols || lds[i] > kMaxStride))
      return fail(MUON_E_INVAL, "embedding: %s=%lld is below cols=%lld or above 2^31", names[i], (long long)lds[i],
                  (long long)d->cols);
  if (d->table_dtype != MUON_DTYPE_F32 && d->table_dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "embedding: table_dtype %d unsupported", d->table_dtype);
  if (d->out_dtype != MUON_DTYPE_F32 && d->out_dtype != MUON_DTYPE_BF16)
    return fail(MUON_E_UNSUPPORTED, "embedding: out_dtype %d unsupported", d->out_dtype);
  if (d->id_dtype != MUON_INDEX_I32 && d->id_dtype != MUON_INDEX_I64)
    return fail(MUON_E_UNSUPPORTED, "embedding: id_dtype %d unsupported", d->id_dtype);
  if (!std::isfinite(d->scale)) return fail(MUON_E_INVAL, "embedding: scale must be finite");
  if (d->reserved != 0) return fail(MUON_E_INVAL, "embedding: reserved field must be 0");
  return MUON_OK;
}
int id_size(const muon_embedding_desc* d) { return d->id_dtype == MUON_INDEX_I64 ? 8 : 4; }
Area table_area(const muon_embedding_desc* d, const void* p) {
  const int es = elem_size(d->table_dtype);
  return area(p, d->vocab, ld_of(d->ld_table, d->cols) * es, 1, 0, d->cols * es);
}
Area out_area(const muon_embedding_desc* d, const void* p) {
  const int es = elem_size(d->out_dtype);
  return area(p, d->tokens, ld_of(d->ld_out, d->cols) * es, 1, 0, d->cols * es);
}

// The backward call's workspace: the sorted list, what sorting it takes, and two
// partial rows for each chunk.
EmbedGradArgs embed_layout(const muon_embedding_desc* d, void* workspace, size_t* bytes) {
  EmbedGradArgs a{};
  a.tokens = d->tokens, a.vocab = d->vocab, a.cols = (int32_t)d->cols;
  plan_embed(a, d->table_dtype == MUON_DTYPE_BF16, d->out_dtype == MUON_DTYPE_BF16);
  char* p = (char*)workspace;
  size_t at = 0;
  auto take = [&](size_t n) {
    char* q = p ? p + at : nullptr;
    at += align_up(n);
    return q;
  };
  *bytes = kAlign;  // never 0, which means an error
  if (a.direct) return a;
  const size_t list = (size_t)d->tokens * sizeof(EmbedEntry);
  a.sorted = (EmbedEntry*)take(list);
  if (d->tokens > kOneBlock) {
    for (int i = 0; i < 2; ++i)
      if (a.passes > i + 1) a.entry[i] = (EmbedEntry*)take(list);
    a.hist = (uint32_t*)take(((size_t)a.blocks << a.digit) * sizeof(uint32_t));
  }
  const size_t chunks = ((size_t)d->tokens + a.chunk - 1) / a.chunk;
  a.part = (float*)take(chunks * 2 * (size_t)d->cols * sizeof(float));
  *bytes += at;
  return a;
}

}  // namespace

extern "C" {

int muon_embedding_forward(const muon_embedding_desc* d, const void* ids, const void* table, void* out,
                           void* hip_stream) {
  clear_error();
  if (int rc = check_embedding(d)) return rc;
  if (d->tokens == 0) return MUON_OK;
  if (!ids || !table || !out) return fail(MUON_E_INVAL, "embedding: ids, table or out is NULL");
  if (misaligned(ids, id_size(d)) || misaligned(table, elem_size(d->table_dtype)) ||
      misaligned(out, elem_size(d->out_dtype)))
    return fail(MUON_E_INVAL, "embedding: pointer not aligned to its element size");
  const Operand ops[] = {{"out", out_area(d, out)}, {"table", table_area(d, table)},
                         {"ids", flat(ids, (size_t)d->tokens * id_size(d))}};
  if (int rc = check_apart("embedding", ops, 1, 3)) return rc;
  EmbedArgs a{};
  a.ids = ids, a.table = table, a.out = out;
  a.tokens = d->tokens, a.vocab = d->vocab, a.cols = (int32_t)d->cols;
  a.ld_table = ld_of(d->ld_table, d->cols), a.ld_out = ld_of(d->ld_out, d->cols);
  a.id64 = d->id_dtype == MUON_INDEX_I64, a.scale = d->scale;
  const hipError_t e = launch_embed_forward(a, d->table_dtype == MUON_DTYPE_BF16, d->out_dtype == MUON_DTYPE_BF16,
                                            (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "embedding forward launch");
}

size_t muon_embedding_workspace_size(const muon_embedding_desc* d) {
  clear_error();
  if (check_embedding(d)) return 0;
  size_t bytes;
  embed_layout(d, nullptr, &bytes);
  return bytes;
}

int muon_embedding_backward(const muon_embedding_desc* d, const void* ids, const void* dout, void* dtable,
                            uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream) {
  clear_error();
  if (int rc = check_embedding(d)) return rc;
  if (flags & ~(uint32_t)MUON_EMBEDDING_ACCUMULATE) return fail(MUON_E_INVAL, "embedding: unknown flags 0x%x", flags);
  if (d->tokens == 0 && flags) return MUON_OK;
  if (!dtable || (d->tokens > 0 && (!ids || !dout)))
    return fail(MUON_E_INVAL, "embedding: ids, dout or dtable is NULL");
  if (misaligned(ids, id_size(d)) || misaligned(dtable, elem_size(d->table_dtype)) ||
      misaligned(dout, elem_size(d->out_dtype)))
    return fail(MUON_E_INVAL, "embedding: pointer not aligned to its element size");
  if (!workspace) return fail(MUON_E_WORKSPACE, "embedding: workspace is NULL");
  if (misaligned(workspace, kAlign)) return fail(MUON_E_WORKSPACE, "embedding: workspace is not 256-byte aligned");
  size_t need;
  EmbedGradArgs a = embed_layout(d, workspace, &need);
  if (ws_bytes < need)
    return fail(MUON_E_WORKSPACE, "embedding: workspace has %zu bytes, the call needs %zu", ws_bytes, need);
  const Operand ops[] = {{"dtable", table_area(d, dtable)},
                         {"workspace", flat(workspace, need)},
                         {"dout", out_area(d, dout)},
                         {"ids", flat(ids, (size_t)d->tokens * id_size(d))}};
  if (int rc = check_apart("embedding", ops, 2, 4)) return rc;
  a.ids = ids, a.dout = dout, a.dtable = dtable;
  a.ld_dout = ld_of(d->ld_out, d->cols), a.ld_dtable = ld_of(d->ld_table, d->cols);
  a.id64 = d->id_dtype == MUON_INDEX_I64, a.scale = d->scale;
  a.accumulate = (flags & MUON_EMBEDDING_ACCUMULATE) != 0;
  const hipError_t e = launch_embed_backward(a, d->table_dtype == MUON_DTYPE_BF16, d->out_dtype == MUON_DTYPE_BF16,
                                             (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "embedding backward launch");
}

int muon_qk_norm_forward(const muon_qk_norm_desc* d, const muon_rotation* rotation, const int32_t* cu_seqlens,
                         const void* positions, const muon_heads* q, const muon_heads* k, const void* q_weight,
                         const void* k_weight, const muon_heads* q_out, const muon_heads* k_out, uint32_t flags,
                         void* hip_stream) {
  clear_error();
  if (int rc = check_qk(d, rotation)) return rc;
  if (d->tokens == 0) return MUON_OK;
  QkArgs a{};
  if (int rc = qk_args(d, rotation, cu_seqlens, positions, flags, q, k, q_out, k_out, "q_out", "k_out", q_weight,
                       k_weight, &a))
    return rc;
  const HeadShape shape{"query/key norm", d->tokens, d->head_dim, d->dtype};
  const size_t params = (size_t)d->head_dim * elem_size(d->p_dtype);
  const Operand ops[] = {{"q_out", heads_area(shape, a.side[0].out, d->q_heads)},
                         {"k_out", heads_area(shape, a.side[1].out, d->k_heads)},
                         {"q", heads_area(shape, a.side[0].x, d->q_heads)},
                         {"k", heads_area(shape, a.side[1].x, d->k_heads)},
                         {"q_weight", flat(q_weight, params)},
                         {"k_weight", flat(k_weight, params)},
                         {"cu_seqlens", flat(cu_seqlens, ((size_t)d->seqs + 1) * 4)},
                         {"positions", flat(positions, (size_t)d->tokens * (a.pos64 ? 8 : 4))}};
  if (int rc = check_apart("query/key norm", ops, 2, 8)) return rc;
  const bool bf16 = d->dtype == MUON_DTYPE_BF16;
  const int pairs = rotation ? rotation->pairs : kPairHalves;
  plan_qk(a, bf16, pairs);
  const hipError_t e = launch_qk(a, bf16, pairs, false, (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "query/key norm forward launch");
}

size_t muon_qk_norm_workspace_size(const muon_qk_norm_desc* d) {
  clear_error();
  if (check_qk(d, nullptr)) return 0;
  return qk_workspace(d) + kAlign;
}

int muon_qk_norm_backward(const muon_qk_norm_desc* d, const muon_rotation* rotation, const int32_t* cu_seqlens,
                          const void* positions, const muon_heads* dq_out, const muon_heads* dk_out,
                          const muon_heads* q, const muon_heads* k, const void* q_weight, const void* k_weight,
                          const muon_heads* dq, const muon_heads* dk, float* dq_weight, float* dk_weight,
                          uint32_t flags, void* workspace, size_t ws_bytes, void* hip_stream) {
  clear_error();
  if (int rc = check_qk(d, rotation)) return rc;
  const bool sums = dq_weight || dk_weight;
  if (misaligned(dq_weight, 4) || misaligned(dk_weight, 4))
    return fail(MUON_E_INVAL, "query/key norm: a weight gradient is not aligned to its element size");
  if (sums) {
    if (!workspace) return fail(MUON_E_WORKSPACE, "query/key norm: workspace is NULL");
    if (misaligned(workspace, kAlign))
      return fail(MUON_E_WORKSPACE, "query/key norm: workspace is not 256-byte aligned");
    if (ws_bytes < qk_workspace(d))
      return fail(MUON_E_WORKSPACE, "query/key norm: workspace has %zu bytes, the call needs %zu", ws_bytes,
                  qk_workspace(d));
  }
  const HeadShape shape{"query/key norm", d->tokens, d->head_dim, d->dtype};
  const size_t params = (size_t)d->head_dim * elem_size(d->p_dtype), grads = (size_t)d->head_dim * 4;
  QkArgs a{};
  if (d->tokens > 0) {
    int rc = qk_args(d, rotation, cu_seqlens, positions, flags, q, k, dq, dk, "dq", "dk", q_weight, k_weight, &a);
    if (!rc) rc = check_heads(shape, dq_out, "dq_out", d->q_heads, false, &a.side[0].dy);
    if (!rc) rc = check_heads(shape, dk_out, "dk_out", d->k_heads, false, &a.side[1].dy);
    if (rc) return rc;
  }
  const Operand ops[] = {{"dq", heads_area(shape, a.side[0].out, d->q_heads)},
                         {"dk", heads_area(shape, a.side[1].out, d->k_heads)},
                         {"dq_weight", flat(dq_weight, grads)},
                         {"dk_weight", flat(dk_weight, grads)},
                         {"workspace", flat(sums ? workspace : nullptr, qk_workspace(d))},
                         {"dq_out", heads_area(shape, a.side[0].dy, d->q_heads)},
                         {"dk_out", heads_area(shape, a.side[1].dy, d->k_heads)},
                         {"q", heads_area(shape, a.side[0].x, d->q_heads)},
                         {"k", heads_area(shape, a.side[1].x, d->k_heads)},
                         {"q_weight", flat(q_weight, params)},
                         {"k_weight", flat(k_weight, params)},
                         {"cu_seqlens", flat(cu_seqlens, ((size_t)d->seqs + 1) * 4)},
                         {"positions", flat(positions, (size_t)d->tokens * (a.pos64 ? 8 : 4))}};
  if (int rc = check_apart("query/key norm", ops, 5, 13)) return rc;
  a.part = sums ? (float*)workspace : nullptr;
  const bool bf16 = d->dtype == MUON_DTYPE_BF16;
  const int pairs = rotation ? rotation->pairs : kPairHalves;
  plan_qk(a, bf16, pairs);
  hipError_t e = hipSuccess;
  if (d->tokens > 0) e = launch_qk(a, bf16, pairs, true, (hipStream_t)hip_stream);
  if (e == hipSuccess && sums)
    e = launch_qk_sum(QkSumArgs{a.part, {dq_weight, dk_weight}, d->tokens > 0 ? a.blocks : 0, d->head_dim},
                      (hipStream_t)hip_stream);
  return e == hipSuccess ? MUON_OK : hip_fail(e, "query/key norm backward launch");
}

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
  const HeadShape shape = shape_of(d);
  AttnArgs a = common_args(d, cu_seqlens, flags);
  int rc = check_heads(shape, q, "q", d->q_heads, false, &a.q);
  if (!rc) rc = check_heads(shape, k, "k", d->kv_heads, false, &a.k);
  if (!rc) rc = check_heads(shape, v, "v", d->kv_heads, false, &a.v);
  if (!rc) rc = check_heads(shape, out, "out", d->q_heads, true, &a.o);
  if (rc) return rc;
  const Operand ops[] = {{"out", heads_area(shape, a.o, d->q_heads)}, {"lse", flat(lse, lse_bytes(d))},
                         {"q", heads_area(shape, a.q, d->q_heads)},   {"k", heads_area(shape, a.k, d->kv_heads)},
                         {"v", heads_area(shape, a.v, d->kv_heads)},
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
  const HeadShape shape = shape_of(d);
  AttnArgs a = common_args(d, cu_seqlens, flags);
  int rc = check_heads(shape, dout, "dout", d->q_heads, false, &a.dout);
  if (!rc) rc = check_heads(shape, q, "q", d->q_heads, false, &a.q);
  if (!rc) rc = check_heads(shape, k, "k", d->kv_heads, false, &a.k);
  if (!rc) rc = check_heads(shape, v, "v", d->kv_heads, false, &a.v);
  if (!rc) rc = check_heads(shape, out, "out", d->q_heads, false, &a.o);
  if (!rc) rc = check_heads(shape, dq, "dq", d->q_heads, true, &a.dq);
  if (!rc) rc = check_heads(shape, dk, "dk", d->kv_heads, true, &a.dk);
  if (!rc) rc = check_heads(shape, dv, "dv", d->kv_heads, true, &a.dv);
  if (rc) return rc;
  if (!workspace) return fail(MUON_E_WORKSPACE, "attention: workspace is NULL");
  if (misaligned(workspace, kAlign)) return fail(MUON_E_WORKSPACE, "attention: workspace is not 256-byte aligned");
  if (ws_bytes < attention_workspace(d))
    return fail(MUON_E_WORKSPACE, "attention: workspace has %zu bytes, the call needs %zu", ws_bytes,
                attention_workspace(d));
  const Operand ops[] = {{"dq", heads_area(shape, a.dq, d->q_heads)},    {"dk", heads_area(shape, a.dk, d->kv_heads)},
                         {"dv", heads_area(shape, a.dv, d->kv_heads)},
                         {"workspace", flat(workspace, attention_workspace(d))},
                         {"dout", heads_area(shape, a.dout, d->q_heads)}, {"q", heads_area(shape, a.q, d->q_heads)},
                         {"k", heads_area(shape, a.k, d->kv_heads)},     {"v", heads_area(shape, a.v, d->kv_heads)},
                         {"out", heads_area(shape, a.o, d->q_heads)},    {"lse", flat(lse, lse_bytes(d))},
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
