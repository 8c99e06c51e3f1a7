// gfx950 (CDNA4) causal attention over packed sequences with grouped heads,
// forward and backward.
//
// Per sequence and query head h (key/value head h / group), with
// s_ij = scale q_i . k_j for j <= i:
//   lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j
//   dk_j = scale sum_{h in group, i >= j} ds_ij q_i,  dv_j = sum_{h in group, i >= j} p_ij do_i
//
// Design.
//   * A block owns 128 rows of the side that is kept (queries for the output
//     and dQ, keys for dK and dV), 32 a wave, as columns of 32x32 MFMA blocks:
//     scores come out transposed, so a lane holds 16 scores of ONE row, row
//     statistics are a lane's own (two lanes share a row), and the same
//     registers, packed to bf16, are the right operand of the next product.
//   * The other side streams through LDS in tiles, copied there directly;
//     row-wise fragments are 16-byte reads and column-wise ones transposing
//     reads, both without bank conflicts (SQ_LDS_BANK_CONFLICT is 0).
//   * dQ has a kernel of its own and repeats the two score products (7
//     products instead of 5): adding dQ from the other kernel would need
//     atomics, whose order changes results.
//   * Registers decide: one wave alone on a SIMD issues a vector operation
//     every 3 ns, two or more every 1.2 ns, so the kernels are shaped to have
//     two to four waves a SIMD; in fp32, dK/dV at heads above 64 and dQ at 128
//     have one.  Hand-pipelined versions with one wave, or a tile of scores
//     ahead, were slower or no faster (bf16 dK/dV at heads of 128: 757 us
//     against 507 now).
//   * What bounds the long bf16 runs: matrix and vector operations of the
//     waves on a SIMD overlap in part; the MFMA units are busy 45 to 52% of
//     the time (a library GEMM: 69%).  Rates on 8192 tokens, 16 query and 4
//     key/value heads of 128: forward 978, dQ 1051, dK/dV 1085 TFLOP/s of their
//     own products (library GEMM of 8192^3: 1410).
#include "block_internal.h"
#include "device_common.h"

namespace muon {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;  // see the forward kernel's running maximum

// ------------------------------------------------------------ element types --
// A fragment is one lane's share of 16 contraction steps of a 32x32 product:
// 8 elements, contraction indices 8 (lane / 32) .. +7 for operands read along
// their rows.  bf16: one v_mfma_f32_32x32x16_bf16; fp32: eight
// v_mfma_f32_32x32x2_f32, whose step e pairs element e of both lane halves.
template <class T>
struct Elem;

template <>
struct Elem<__bf16> {
  typedef u32x4 Frag;
  static constexpr int kFragChunks = 1;
  __device__ static __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  __device__ static __forceinline__ Frag pack(const float* v) { return pack8_bf16(v); }
  __device__ static __forceinline__ void unpack(Frag f, float* v) { unpack8_bf16(f, v); }
};

struct F32Frag {
  f32x4 lo, hi;
};
template <>
struct Elem<float> {
  typedef F32Frag Frag;
  static constexpr int kFragChunks = 2;
  __device__ static __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.lo[e], b.lo[e], c, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.hi[e], b.hi[e], c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ Frag pack(const float* v) {
    return Frag{f32x4{v[0], v[1], v[2], v[3]}, f32x4{v[4], v[5], v[6], v[7]}};
  }
  __device__ static __forceinline__ void unpack(Frag f, float* v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f.lo[e], v[4 + e] = f.hi[e];
  }
};

// --------------------------------------------------------------- LDS tiles --
// A tile is `rows` rows of DP elements without padding; 16-byte chunk c of
// row r sits at chunk c ^ swz(r).  The swizzles make both kinds of fragment
// read conflict-free (16-byte reads of one chunk of 16 rows; transposing
// reads of 4 rows x 64 bytes): swz has period 16 in r, takes a row's share of
// the 256 bytes served per clock into account, and moves 4 consecutive rows
// to different 64-byte quarters.
template <int ROW_BYTES>
__device__ __forceinline__ int swz(int r) {
  if (ROW_BYTES % 256 == 0) return ((r & 3) << 2) | ((r >> 2) & 3);
  if (ROW_BYTES % 128 == 0) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  return (r >> 2) & 3;
}

template <class T, int DP>
struct Tiles {
  typedef typename Elem<T>::Frag Frag;
  static constexpr int kRow = DP * (int)sizeof(T);  // bytes
  static constexpr int kCpr = kRow / 16;            // chunks a row

  // Row-wise fragment: 16-step s of row `row`, lane half h.
  __device__ static __forceinline__ Frag row_frag(const char* tile, int row, int s, int h) {
    if constexpr (sizeof(T) == 2) {
      return *(const u32x4*)(tile + row * kRow + (((2 * s + h) ^ swz<kRow>(row)) << 4));
    } else {
      const int c = 4 * s + 2 * h;
      return Frag{*(const f32x4*)(tile + row * kRow + ((c ^ swz<kRow>(row)) << 4)),
                  *(const f32x4*)(tile + row * kRow + (((c + 1) ^ swz<kRow>(row)) << 4))};
    }
  }
  // Column-wise fragment: element (lane & 31) of 32-column group t over the
  // 16 rows base .. base + 15, in the order in which an accumulator holds
  // them: rows 4 h .. 4 h + 3, then 8 + 4 h .. 8 + 4 h + 3.  bf16: two
  // transposing reads (each 16 lanes fetch 4 rows x 16 columns, and lane r
  // of them gets column r's 4 values).
  __device__ static __forceinline__ Frag col_frag(const char* tile, int base, int t, int lane) {
    if constexpr (sizeof(T) == 2) {
      const int g = lane >> 4, r = lane & 15;
      const int row = 4 * (g >> 1) + (r >> 2), c = 4 * t + 2 * (g & 1) + ((r & 3) >> 1);
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* lds_v4;
      const char* p0 = tile + (base + row) * kRow + ((c ^ swz<kRow>(row)) << 4) + ((r & 1) << 3);
      const char* p1 = tile + (base + row + 8) * kRow + ((c ^ swz<kRow>(row + 8)) << 4) + ((r & 1) << 3);
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(void*)p0));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(void*)p1));
      return u32x4{a.x, a.y, b.x, b.y};
    } else {
      const int h = lane >> 5, d = 32 * t + (lane & 31);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 8 * (e >> 2) + 4 * h + (e & 3);
        v[e] = *(const float*)(tile + (base + row) * kRow + (((d >> 2) ^ swz<kRow>(row)) << 4) + ((d & 3) << 2));
      }
      return Elem<float>::pack(v);
    }
  }
};

// Copies tiles of ROWS rows of one head from global memory straight to LDS.
// Each wave instruction writes 64 x 16 contiguous bytes of the tile, and the
// swizzle is applied by choosing which chunk each lane fetches.  The buffer
// resource covers the tile's rows inside the sequence, past which loads return
// zeros; a chunk past the head dimension gets an offset beyond every resource.
//
// The instruction is written in assembly because the compiler, which sees a
// builtin's LDS write, waits for it before every later LDS read of either
// buffer.  It has no register outputs; wait_tiles() waits for it.  (m0, which
// holds the LDS address, is reserved: the compiler keeps nothing in it.)
constexpr uint32_t kOob = 0x80000000u;
__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes) {  // uniform arguments
  const uint64_t p = (uint64_t)base;
  auto word = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); };
  return u32x4{word((uint32_t)p), word((uint32_t)(p >> 32) & 0xFFFFu), word(bytes), 0x00020000u};
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)p);
}
__device__ __forceinline__ void dma_b128(u32x4 rs, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(off), "s"(rs) : "memory");
}
__device__ __forceinline__ void dma_b32(u32x4 rs, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(off), "s"(rs) : "memory");
}
// Waits for this wave's copies, then for the block's other waves: the tiles
// copied since the last call can be read, and those read before it written.
__device__ __forceinline__ void wait_tiles() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The same with the wave's last N copies still in flight.
template <int N>
__device__ __forceinline__ void wait_but() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Copies ROWS rows at a time of two operands (K and V, or Q and dO) into a
// pair of adjacent tiles.  The first half of a group's WR waves copies the
// first operand, the other half the second, kN instructions each, so a wave
// keeps one pointer and one resource, and waits can count instructions.
template <class T, int DP, int ROWS, int WR>
struct PairCopier {
  static constexpr int kTile = ROWS * DP * (int)sizeof(T), kN = 2 * kTile / 1024 / WR, kHalf = WR / 2;
  static_assert(kN * WR * 1024 == 2 * kTile, "whole instructions per wave");
  const char* at;           // the next row of this wave's operand
  int64_t step;             // bytes from row to row
  int left;                 // rows from there to the sequence's end
  uint32_t row_bytes;
  uint32_t off[kN];
  __device__ __forceinline__ void init(const HeadView& x, const HeadView& y, int dim, int w, int lane) {
    constexpr int cpr = Tiles<T, DP>::kCpr, kRow = Tiles<T, DP>::kRow;
    step = (w < kHalf ? x.token : y.token) * (int64_t)sizeof(T);
    row_bytes = dim * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int idx = (w % kHalf * kN + i) * 64 + lane, row = idx / cpr, c = (idx % cpr) ^ swz<kRow>(row);
      off[i] = (uint32_t)c * 16 < row_bytes ? (uint32_t)(row * step) + 16u * c : kOob;
    }
  }
  __device__ __forceinline__ void seek(const HeadView& x, int xhead, const HeadView& y, int yhead, int64_t token,
                                       int rows, int w) {
    const HeadView& v = w < kHalf ? x : y;
    at = (const char*)((const T*)v.data + token * v.token + (w < kHalf ? xhead : yhead) * v.head);
    left = rows;
  }
  // `pair`: the two tiles.  Moves on by NG tiles; past the last row, tiles of zeros.
  template <int NG>
  __device__ __forceinline__ void copy(char* pair, int w, int lane) {
    const uint32_t lds = lds_offset(pair + w * kN * 1024);
    if (left >= ROWS) {
      const u32x4 rs = buffer_of(at, (uint32_t)((ROWS - 1) * step) + row_bytes);
#pragma unroll
      for (int i = 0; i < kN; ++i) dma_b128(rs, lds + 1024 * i, off[i]);
    } else {  // rows may overlap (a step of 0 repeats one), so the resource's end alone does not tell them apart
      const u32x4 rs = buffer_of(at, left > 0 ? (uint32_t)((left - 1) * step) + row_bytes : 0u);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        dma_b128(rs, lds + 1024 * i,
                 ((w % kHalf * kN + i) * 64 + lane) / Tiles<T, DP>::kCpr < left ? off[i] : kOob);
    }
    at += NG * ROWS * step;
    left -= NG * ROWS;
  }
};

// Row-wise fragments of one row straight from global memory (the operand that
// stays in registers); zeros where the row is not valid or past `dim`.
template <class T, int DP>
__device__ __forceinline__ void load_frags(typename Elem<T>::Frag (&f)[DP / 16], const T* row, bool valid, int dim,
                                           int h) {
  constexpr int epc = 16 / (int)sizeof(T);
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    u32x4 w[Elem<T>::kFragChunks];
#pragma unroll
    for (int e = 0; e < Elem<T>::kFragChunks; ++e) {
      const int at = 16 * s + 8 * h + e * epc;
      w[e] = u32x4{0, 0, 0, 0};
      if (valid && at < dim) w[e] = *gv<u32x4>(row + at);
    }
    f[s] = __builtin_bit_cast(typename Elem<T>::Frag, w);
  }
}

// The lane's columns of an accumulator tile set, acc[t][i] = element
// d = 32 t + 8 (i / 4) + 4 h + i % 4 of its row, times `f`, as elements.
template <class T, int DP>
__device__ __forceinline__ void store_row(T* row, const f32x16 (&acc)[DP / 32], float f, int dim, int h) {
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * t + 8 * g + 4 * h;
      if (d >= dim) continue;
      const float a = acc[t][4 * g] * f, b = acc[t][4 * g + 1] * f, c = acc[t][4 * g + 2] * f,
                  e = acc[t][4 * g + 3] * f;
      if constexpr (sizeof(T) == 2)
        *gv<u32x2>(row + d) = pack4_bf16(a, b, c, e);
      else
        *gv<f32x4>(row + d) = f32x4{a, b, c, e};
    }
}

// ---------------------------------------------- what a mask hides, no one sees --
// A masked pair has weight 0, but 0 times a NaN or an infinity is NaN, and a
// matrix instruction multiplies every pair of its block.  So every pass ends
// with a test of the accumulators (0 x each, summed: a few dozen operations a
// wave), and where one is not finite the thread block makes its pass again,
// carefully: products that are masked as a whole are skipped, and in those on
// the diagonal the streamed side's values that are not finite are taken as 0,
// and added afterwards to the rows that see them.  The careful pass is code of
// its own, behind the first: one loop with both ways in it cost 50 to 130
// registers.  Times with the test and without, forward and backward: 8192
// tokens of 12 heads of 64 131 / 417 and 133 / 421 us, 16/4 heads of 128
// 280 / 914 and 276 / 911; nothing but NaN takes three times as long.
template <class T>
__device__ __forceinline__ typename Elem<T>::Frag finite_part(typename Elem<T>::Frag f, bool diag) {
  float v[8];
  Elem<T>::unpack(f, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (__builtin_isfinite(v[e]) | !diag) ? v[e] : 0.f;
  return Elem<T>::pack(v);
}
template <int DT>
__device__ __forceinline__ float not_finite(const f32x16 (&acc)[DT]) {  // 0 or NaN
  float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i % 4] = __builtin_fmaf(acc[t][i], 0.f, x[i % 4]);
  return (x[0] + x[1]) + (x[2] + x[3]);
}
// Whether any wave of the block holds a NaN; `flags`: a word a wave, used once.
template <int WAVES>
__device__ __forceinline__ bool any_nan(float x, int* flags, int wave) {
  flags[wave] = __any(x != x);
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) any |= flags[i];
  return __builtin_amdgcn_readfirstlane(any) != 0;
}
// Adds to the lane's columns of an accumulator tile set (laid out as in
// store_row) `f` times what finite_part() took from `rows` rows, the lane's
// being those from `lo` to `hi`.
template <class T, int DP>
__device__ __forceinline__ void add_not_finite(f32x16 (&acc)[DP / 32], const T* row, int64_t step, int rows, int lo,
                                               int hi, float f, int dim, int h) {
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * t + 8 * g + 4 * h;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int r = 0; r < rows; ++r) {
        if (r < lo || r > hi || d >= dim) continue;
        float v[4];
        if constexpr (sizeof(T) == 2) {
          unpack4_bf16(*gv<u32x2>(row + r * step + d), v);
        } else {
          const f32x4 y = *gv<f32x4>(row + r * step + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = y[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += __builtin_isfinite(v[e]) ? 0.f : f * v[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][4 * g + e] += x[e];
    }
}
// Waves a SIMD that the first pass's registers leave room for.  As launch
// bounds they make the careful pass spill where it would take more.
template <class T, int DP, int NG>
constexpr int kForwardWaves = sizeof(T) == 4 ? (DP == 32 ? 4 : 2)
                              : DP == 32     ? 5
                              : DP == 64     ? 4
                              : DP == 96     ? (NG == 1 ? 3 : 2)
                                             : 2;
template <class T, int DP, int NG>
constexpr int kDqWaves = sizeof(T) == 4 ? (DP == 32    ? 3
                                           : DP == 128 ? 1
                                                       : 2)
                         : DP == 32     ? 4
                         : DP == 64     ? (NG == 1 ? 3 : 2)
                                        : 2;
template <int DP>
constexpr int kDkvWaves = DP == 32 ? 4 : DP == 64 ? 3 : 2;

// Adds the other groups of waves' accumulators to the first's, in order,
// through LDS (kJoin bytes); true in the others, whose work is done.
template <int DT, int WR, int NG>
constexpr int kJoin = (NG - 1) * WR * 16 * DT * 64 * 4;
template <int WR, int NG, int DT>
__device__ __forceinline__ bool join_groups(f32x16 (&acc)[DT], float* lds, int grp, int w, int lane) {
  float* sum = lds + w * 16 * DT * 64 + lane;
  wait_tiles();  // nothing is copied to or read from the tiles any more
  if (grp) {
    float* to = sum + (grp - 1) * WR * 16 * DT * 64;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) to[(16 * t + i) * 64] = acc[t][i];
  }
  __syncthreads();
  if (grp) return true;
#pragma unroll
  for (int g = 0; g < NG - 1; ++g)
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][i] += sum[(g * WR * 16 * DT + 16 * t + i) * 64];
  return false;
}

// Largest of / sum over the two lanes l, l ^ 32 that share a column.
__device__ __forceinline__ float halves_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// -------------------------------------------------------- sequences, tiles --
// Sequence i's tiles of `bm` rows take the slots from cu[i] / bm + i on: that
// many are always free before the next sequence's first slot, so a block
// finds its sequence by a search in cu alone, with no table built beforehand.
// The rows behind the last sequence are "sequence" seqs.
struct SeqTile {
  int start, len;  // the sequence's first token and its length
  int row0;        // first row of this tile, within the sequence
  bool tail;       // rows behind the last sequence
};
__device__ __forceinline__ int token_at(const AttnArgs& a, int i) {
  const int n = (int)a.tokens;
  return i > a.seqs ? n : min(max(a.cu[i], 0), n);
}
__device__ __forceinline__ SeqTile find_tile(const AttnArgs& a, int slot, int bm, int lane) {
  int lo = 0, hi = a.seqs + 1;  // the last i in [lo, hi) whose first slot is at or below `slot`
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const int i = lo + lane * step;
    const bool below = i < hi && token_at(a, i) / bm + i <= slot;
    const int n = __popcll(__ballot(below));
    lo += (n > 0 ? n - 1 : 0) * step;
    hi = min(hi, lo + step);
  }
  SeqTile t;
  t.tail = lo == a.seqs;
  t.start = token_at(a, lo);
  t.len = max(token_at(a, lo + 1) - t.start, 0);
  const int tile = slot - (t.start / bm + lo);
  t.row0 = tile < 0 || tile >= (t.len + bm - 1) / bm ? t.len : tile * bm;
  return t;
}
inline int64_t slots_of(int64_t tokens, int seqs, int bm) { return tokens / bm + seqs + 1; }

// The tile of a block in order of decreasing work, for up to kRankSeqs
// sequences: tile `t` of a sequence looks at t + 1 tiles of keys, so the tiles
// of equal work w are one of each sequence of at least w tiles, and
// N(w) = sum over sequences of max(0, tiles - w + 1) tiles have work w or
// more.  Every wave keeps the sequences' tile counts in its lanes, finds the
// largest w with N(w) > rank, and in that level the sequence.  (Backward, the
// keys of tile t are looked at by tiles - t tiles of queries.)
constexpr int kRankSeqs = 256;
// Sum and maximum (of values that are not negative) over the wave in six
// data-parallel steps: within rows of 16 lanes, then across them; lane 63
// ends with the result.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_sum(int x) {
  x += dpp<0x111, 0xf>(x);
  x += dpp<0x112, 0xf>(x);
  x += dpp<0x114, 0xf>(x);
  x += dpp<0x118, 0xf>(x);
  x += dpp<0x142, 0xa>(x);
  x += dpp<0x143, 0xc>(x);
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ int wave_max(int x) {
  x = max(x, dpp<0x111, 0xf>(x));
  x = max(x, dpp<0x112, 0xf>(x));
  x = max(x, dpp<0x114, 0xf>(x));
  x = max(x, dpp<0x118, 0xf>(x));
  x = max(x, dpp<0x142, 0xa>(x));
  x = max(x, dpp<0x143, 0xc>(x));
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ SeqTile ranked_tile(const AttnArgs& a, int rank, int bm, int lane, bool keys) {
  constexpr int kC = kRankSeqs / 64;
  int from[kC], to[kC], nt[kC], most = 0, all = 0, end = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    from[c] = to[c] = nt[c] = 0;
    if (c == 0 || a.seqs > 64 * c) {
      const int i = min(64 * c + lane, a.seqs);
      from[c] = token_at(a, i);
      to[c] = token_at(a, min(i + 1, a.seqs));
      end = __builtin_amdgcn_readlane(to[c], 63);  // the last sequence's, in the last chunk
      nt[c] = (max(to[c] - from[c], 0) + bm - 1) / bm;
      most = max(most, nt[c]);
      all += nt[c];
    }
  }
  SeqTile t;
  all = wave_sum(all);
  if (rank >= all) {
    t.tail = true;
    t.start = end;
    t.len = (int)a.tokens - t.start;
    t.row0 = rank - all < (t.len + bm - 1) / bm ? (rank - all) * bm : t.len;
    return t;
  }
  int lo = 1, hi = wave_max(most) + 1, above = 0;  // N(lo) > rank >= N(hi) = above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int n = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c) n += max(nt[c] - mid + 1, 0);
    n = wave_sum(n);
    if (n > rank) {
      lo = mid;
    } else {
      hi = mid;
      above = n;
    }
  }
  int j = rank - above;  // the j-th sequence of at least lo tiles
  t.tail = false;
  t.start = t.len = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const uint64_t m = __ballot(nt[c] >= lo);
    const int n = __popcll(m);
    if (j >= 0 && j < n) {
      const uint64_t hit = __ballot(((m >> lane) & 1) && __popcll(m & ((1ull << lane) - 1)) == j);
      const int l = __ffsll((unsigned long long)hit) - 1;
      t.start = __builtin_amdgcn_readlane(from[c], l);
      t.len = max(__builtin_amdgcn_readlane(to[c], l) - t.start, 0);
    }
    j -= n;
  }
  t.row0 = (keys ? (t.len + bm - 1) / bm - lo : lo - 1) * bm;
  return t;
}
// Block `i` of `n` along the tiles: heaviest first.  With more sequences than
// that, each is short beside the whole, and the slots are taken backwards
// (forwards for keys), heaviest first within a sequence.
__device__ __forceinline__ SeqTile block_tile(const AttnArgs& a, int i, int n, int bm, int lane, bool keys) {
  return a.seqs <= kRankSeqs ? ranked_tile(a, i, bm, lane, keys) : find_tile(a, keys ? i : n - 1 - i, bm, lane);
}

template <class T>
__device__ __forceinline__ void zero_rows(const HeadView& v, int head, int row0, int rows, int dim, int tid) {
  const int dw = dim * (int)sizeof(T) / 16;
  for (int i = tid; i < rows * dw; i += (int)blockDim.x) {
    T* p = (T*)v.data + (int64_t)(row0 + i / dw) * v.token + head * v.head;
    gv<u32x4>(p)[i % dw] = u32x4{0, 0, 0, 0};
  }
}

// ----------------------------------------------------------------- forward --
// NG groups of WR waves: the block's rows are 32 WR, wave w of each group
// holds rows 32 w .. +31, and the groups take the tiles of keys in turn, with
// softmax statistics of their own that the first group joins at the end.
//
// One pass over the keys, with the running maximum and sum in registers (fp32);
// p is rounded to bf16 for its product only (l sums the fp32 values).  Bound by
// vector operations at heads of 64 (per 64 keys and 32 rows: 156 of them, 740
// clocks, against 512 of MFMA; 64 keys at a time rather than 32: 67 and 82 us
// on 16384 packed tokens) and by the overlap of both at 128.  Times: 16384
// tokens in 24 sequences, 12 heads of 64: 64 us (614 TFLOP/s of the visible
// pairs); 16384 tokens, 16/4 heads of 128: 1077 us (1021 TFLOP/s).
template <class T>
struct Cfg {
  static constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;  // rows of a streamed tile
};

template <class T, int DP, int WR, int NG>
__global__ __launch_bounds__(NG * WR * 64, (kForwardWaves<T, DP, NG>)) void attention_forward_kernel(AttnArgs a) {
  typedef typename Elem<T>::Frag Frag;
  typedef Tiles<T, DP> Tl;
  constexpr int BM = 32 * WR, KT = Cfg<T>::kKeys, MT = KT / 32, ST = DP / 16, DT = DP / 32;
  constexpr int kTile = KT * Tl::kRow;
  __shared__ __align__(256) char lds[NG][2][2][kTile];
  __shared__ int flags[NG * WR];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, col = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6) % WR, grp = __builtin_amdgcn_readfirstlane(tid >> 6) / WR;
  const int head = blockIdx.x % a.q_heads, kvh = head / a.group;
  const SeqTile st =
      block_tile(a, (int)(blockIdx.x / a.q_heads), (int)(gridDim.x / a.q_heads), BM, lane, false);
  if (st.row0 >= st.len) return;
  if (st.tail) {
    const int rows = min(BM, st.len - st.row0), r0 = st.start + st.row0;
    if (a.zero_tail & kZeroOut) zero_rows<T>(a.o, head, r0, rows, a.dim, tid);
    if ((a.zero_tail & kZeroLse) && tid < rows) a.lse[(int64_t)head * a.tokens + r0 + tid] = 0.f;
    return;
  }
  const int qw = st.row0 + 32 * w, qi = qw + col;
  const int wend = qw < st.len ? min(st.len, qw + 32) : 0;  // keys this wave looks at
  const int ntile = (min(st.len, st.row0 + BM) + NG * KT - 1) / (NG * KT);  // of each group
  const float c = a.scale * kLog2e;

  Frag qf[ST];
  load_frags<T, DP>(qf, (const T*)a.q.data + (st.start + (int64_t)qi) * a.q.token + head * a.q.head, qi < st.len,
                    a.dim, h);
  f32x16 o[DT];
  float m, l;
  PairCopier<T, DP, KT, WR> cp;
  cp.init(a.k, a.v, a.dim, w, lane);
  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < DT; ++t) o[t] = f32x16{};
    m = -__FLT_MAX__, l = 0.f;  // not -inf: scores of -inf before the first finite one have weight 0, not NaN

    cp.seek(a.k, kvh, a.v, kvh, st.start + (int64_t)grp * KT, st.len - grp * KT, w);
    cp.template copy<NG>(lds[grp][0][0], w, lane);
    wait_tiles();
    for (int kt = 0; kt < ntile; ++kt) {
      const char *kl = lds[grp][kt & 1][0], *vl = lds[grp][kt & 1][1];
      const int k0 = (kt * NG + grp) * KT;  // first key of this group's tile
      if (kt + 1 < ntile) cp.template copy<NG>(lds[grp][(kt + 1) & 1][0], w, lane);
      if (k0 < wend) {
        f32x16 s[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          s[j] = f32x16{};
#pragma unroll
          for (int q = 0; q < ST; ++q) s[j] = Elem<T>::mma(Tl::row_frag(kl, 32 * j + col, q, h), qf[q], s[j]);
        }
        if (k0 + KT - 1 > qw) {
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (k0 + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3) > qi) s[j][i] = -__builtin_inff();
        }
        float top = s[0][0];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[j][i]);
        top = halves_max(top) * c;
        // The running maximum only has to keep exp2's arguments small: it is
        // raised (and the sums rescaled) when a score passes it by more than
        // kLazy, so p <= 2^kLazy, and most tiles rescale nothing.
        if (__any(top > m + kLazy)) {
          const float mn = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] *= f;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          float p[16], sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], c, -m));
            sum += p[i];
          }
          l += sum;  // 16 at a time: the error of a long sum grows with its number of additions
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const Frag pf = Elem<T>::pack(p + 8 * u);
#pragma unroll
            for (int t = 0; t < DT; ++t) {
              Frag vf = Tl::col_frag(vl, 32 * j + 16 * u, t, lane);
              if (careful.value) vf = finite_part<T>(vf, k0 + KT - 1 > qw);
              o[t] = Elem<T>::mma(vf, pf, o[t]);
            }
          }
        }
      }
      wait_tiles();
    }
  };
  pass(std::false_type{});
  if (any_nan<NG * WR>(not_finite(o), flags, grp * WR + w)) {
    pass(std::true_type{});
    const int k0 = qw / KT * KT;
    if (grp == 0 && qi < st.len)
      add_not_finite<T, DP>(o, (const T*)a.v.data + (st.start + (int64_t)k0) * a.v.token + kvh * a.v.head, a.v.token,
                            min(KT, st.len - k0), 0, qi - k0, 1.f, a.dim, h);
  }
  l = halves_sum(l);
  if constexpr (NG > 1) {  // the other groups hand their sums to the first
    constexpr int kOne = (16 * DT + 2) * 64;
    static_assert((NG - 1) * WR * kOne * sizeof(float) <= sizeof(lds), "the sums fit the tiles");
    float* sum = (float*)lds + w * kOne + lane;
    if (grp) {
      float* to = sum + (grp - 1) * WR * kOne;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) to[(16 * t + i) * 64] = o[t][i];
      to[16 * DT * 64] = m;
      to[(16 * DT + 1) * 64] = l;
    }
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int g = 0; g < NG - 1; ++g, sum += WR * kOne) {
      const float m2 = sum[16 * DT * 64], mn = fmaxf(m, m2);
      const float f1 = __builtin_amdgcn_exp2f(m - mn), f2 = __builtin_amdgcn_exp2f(m2 - mn);
      m = mn;
      l = l * f1 + sum[(16 * DT + 1) * 64] * f2;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = o[t][i] * f1 + sum[(16 * t + i) * 64] * f2;
    }
  }
  if (qi < st.len) {
    const int64_t tok = st.start + (int64_t)qi;
    store_row<T, DP>((T*)a.o.data + tok * a.o.token + head * a.o.head, o, 1.f / l, a.dim, h);
    if (h == 0) a.lse[(int64_t)head * a.tokens + tok] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// ---------------------------------------------------------------- backward --
// dQ; and for the next kernel delta and lse: in fp32, delta and lse / log 2;
// in bf16, -delta and -lse / scale, from which it starts its products' sums.
// The forward kernel's layout, with dO's fragments in registers beside Q's and
// no running maximum; ds is rounded to bf16 for its product.  Times: 16384
// tokens in 24 sequences, 12 heads of 64: 89 us (661 TFLOP/s); 8192 tokens,
// 16/4 heads of 128: 392 us (1051).
template <class T, int DP, int WR, int NG>
__global__ __launch_bounds__(NG * WR * 64, (kDqWaves<T, DP, NG>)) void attention_dq_kernel(AttnArgs a) {
  typedef typename Elem<T>::Frag Frag;
  typedef Tiles<T, DP> Tl;
  constexpr int BM = 32 * WR, KT = Cfg<T>::kKeys, MT = KT / 32, ST = DP / 16, DT = DP / 32;
  constexpr int kTile = KT * Tl::kRow;
  constexpr bool kFix = sizeof(T) == 2;
  __shared__ __align__(256) char lds[NG][2][2][kTile];
  __shared__ float offs[NG][WR][kFix ? 64 : 1];
  __shared__ int flags[NG * WR];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, col = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6) % WR, grp = __builtin_amdgcn_readfirstlane(tid >> 6) / WR;
  const int head = blockIdx.x % a.q_heads, kvh = head / a.group;
  const SeqTile st =
      block_tile(a, (int)(blockIdx.x / a.q_heads), (int)(gridDim.x / a.q_heads), BM, lane, false);
  if (st.row0 >= st.len) return;
  if (st.tail) {
    if (a.zero_tail & kZeroDq)
      zero_rows<T>(a.dq, head, st.start + st.row0, min(BM, st.len - st.row0), a.dim, tid);
    return;
  }
  const int qw = st.row0 + 32 * w, qi = qw + col;
  const int wend = qw < st.len ? min(st.len, qw + 32) : 0;
  const int ntile = (min(st.len, st.row0 + BM) + NG * KT - 1) / (NG * KT);
  const float c = a.scale * kLog2e;
  const bool valid = qi < st.len;
  const int64_t tok = st.start + (int64_t)qi;

  Frag qf[ST], df[ST];
  load_frags<T, DP>(qf, (const T*)a.q.data + tok * a.q.token + head * a.q.head, valid, a.dim, h);
  load_frags<T, DP>(df, (const T*)a.dout.data + tok * a.dout.token + head * a.dout.head, valid, a.dim, h);
  float delta = 0.f, lse2 = 0.f;
  {
    Frag of[ST];
    load_frags<T, DP>(of, (const T*)a.o.data + tok * a.o.token + head * a.o.head, valid, a.dim, h);
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      float x[8], y[8];
      Elem<T>::unpack(of[s], x);
      Elem<T>::unpack(df[s], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf(x[e], y[e], delta);
    }
    delta = halves_sum(delta);
    if (valid) {
      lse2 = a.lse[(int64_t)head * a.tokens + tok] * kLog2e;
      if (h == 0 && grp == 0) a.lse2[(int64_t)head * a.tokens + tok] = kFix ? -lse2 / c : lse2;
    }
  }
  f32x16 dq[DT];
  PairCopier<T, DP, KT, WR> cp;
  cp.init(a.k, a.v, a.dim, w, lane);
  // out is rounded to bf16, and so delta is off; but the ds of a row must sum
  // to zero, so their sum is the difference, and the exact delta goes to the
  // next kernel.  In a sequence's first rows, where few terms average such
  // errors, dq is made again with it.
  auto pass = [&](auto careful) __attribute__((always_inline)) {
    float off = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) dq[t] = f32x16{};
    cp.seek(a.k, kvh, a.v, kvh, st.start + (int64_t)grp * KT, st.len - grp * KT, w);
    cp.template copy<NG>(lds[grp][0][0], w, lane);
    wait_tiles();
    for (int kt = 0; kt < ntile; ++kt) {
      const char *kl = lds[grp][kt & 1][0], *vl = lds[grp][kt & 1][1];
      const int k0 = (kt * NG + grp) * KT;
      if (kt + 1 < ntile) cp.template copy<NG>(lds[grp][(kt + 1) & 1][0], w, lane);
      if (k0 < wend) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
          for (int q = 0; q < ST; ++q) s = Elem<T>::mma(Tl::row_frag(kl, 32 * j + col, q, h), qf[q], s);
#pragma unroll
          for (int q = 0; q < ST; ++q) dp = Elem<T>::mma(Tl::row_frag(vl, 32 * j + col, q, h), df[q], dp);
          float ds[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            ds[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2)) * (dp[i] - delta);
          if (k0 + 32 * j + 31 > qw) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (k0 + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3) > qi) ds[i] = 0.f;
          }
          if constexpr (kFix) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += ds[i];
            off += sum;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const Frag pf = Elem<T>::pack(ds + 8 * u);
#pragma unroll
            for (int t = 0; t < DT; ++t) {
              Frag kf = Tl::col_frag(kl, 32 * j + 16 * u, t, lane);
              if (careful.value) kf = finite_part<T>(kf, k0 + KT - 1 > qw);
              dq[t] = Elem<T>::mma(kf, pf, dq[t]);
            }
          }
        }
      }
      wait_tiles();
    }
    if constexpr (kFix) {
      off = halves_sum(off);
      if constexpr (NG > 1) {
        offs[grp][w][lane] = off;
        __syncthreads();
        off = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) off += offs[g][w][lane];
        __syncthreads();
      }
    }
    return off;
  };
  if (kFix && st.row0 == 0) delta += pass(std::false_type{});
  float off = pass(std::false_type{});
  if (any_nan<NG * WR>(not_finite(dq), flags, grp * WR + w)) {
    off = pass(std::true_type{});
    const int k0 = qw / KT * KT;
    if (grp == 0 && valid)
      add_not_finite<T, DP>(dq, (const T*)a.k.data + (st.start + (int64_t)k0) * a.k.token + kvh * a.k.head, a.k.token,
                            min(KT, st.len - k0), 0, qi - k0, 0.f, a.dim, h);
  }
  delta += off;
  if (valid && h == 0 && grp == 0) a.delta[(int64_t)head * a.tokens + tok] = kFix ? -delta : delta;
  if constexpr (NG > 1) {
    static_assert(kJoin<DT, WR, NG> <= sizeof(lds), "the sums fit the tiles");
    if (join_groups<WR, NG>(dq, (float*)lds, grp, w, lane)) return;
  }
  if (valid) store_row<T, DP>((T*)a.dq.data + tok * a.dq.token + head * a.dq.head, dq, a.scale, a.dim, h);
}

// dK and dV of 32 WR keys of one key/value head, over the query heads of its
// group (or of one part of it) and the query rows from the keys on, in fp32.
// Bound by the fp32 MFMA (157 TFLOP/s): 2048 tokens in 5 sequences, 12 heads of
// 64, 73 us with NG = 4 (MFMA busy 40%).
template <int DP, int WR, int NG>
__global__ __launch_bounds__(NG * WR * 64, DP <= 64 ? 2 : 1) void attention_dkv_kernel(AttnArgs a) {
  typedef float T;
  typedef typename Elem<T>::Frag Frag;
  typedef Tiles<T, DP> Tl;
  constexpr int BN = 32 * WR, QR = Cfg<T>::kKeys, MT = QR / 32, ST = DP / 16, DT = DP / 32;
  constexpr int kTile = QR * Tl::kRow;
  __shared__ __align__(256) char lds[NG][2][2][kTile];
  __shared__ __align__(256) float stat[NG][2][2][64];  // lse2 and delta of the tile's rows
  __shared__ int flags[NG * WR];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, col = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6) % WR, grp = __builtin_amdgcn_readfirstlane(tid >> 6) / WR;
  const int per = a.kv_heads * a.splits;
  const int kvh = (int)(blockIdx.x % per) / a.splits, part = (int)(blockIdx.x % per) % a.splits;
  const SeqTile st = block_tile(a, (int)(blockIdx.x / per), (int)(gridDim.x / per), BN, lane, true);
  if (st.row0 >= st.len) return;
  if (st.tail) {
    const int rows = min(BN, st.len - st.row0), r0 = st.start + st.row0;
    if (part == 0 && (a.zero_tail & kZeroDk)) zero_rows<T>(a.dk, kvh, r0, rows, a.dim, tid);
    if (part == 0 && (a.zero_tail & kZeroDv)) zero_rows<T>(a.dv, kvh, r0, rows, a.dim, tid);
    return;
  }
  const int kw = st.row0 + 32 * w, ki = kw + col;
  const bool valid = ki < st.len;
  const int64_t tok = st.start + (int64_t)ki;
  const float c = a.scale * kLog2e;
  const int hpp = a.group / a.splits, head0 = kvh * a.group + part * hpp;  // this block's query heads

  Frag kf[ST], vf[ST];
  load_frags<T, DP>(kf, (const T*)a.k.data + tok * a.k.token + kvh * a.k.head, valid, a.dim, h);
  load_frags<T, DP>(vf, (const T*)a.v.data + tok * a.v.token + kvh * a.v.head, valid, a.dim, h);
  f32x16 dk[DT], dv[DT];
  const int qt0 = st.row0 / QR, nq = (st.len + QR - 1) / QR - qt0, total = nq * hpp;
  PairCopier<T, DP, QR, WR> cp;
  cp.init(a.q, a.dout, a.dim, w, lane);
  auto copy = [&](int it) {
    const int n = it * NG + grp, b = it & 1;
    const int head = head0 + min(n / nq, hpp - 1), row0 = n < total ? (qt0 + n % nq) * QR : st.len;
    cp.seek(a.q, head, a.dout, head, st.start + (int64_t)row0, st.len - row0, w);
    cp.template copy<1>(lds[grp][b][0], w, lane);
    if (w < 2)
      dma_b32(buffer_of((w ? a.delta : a.lse2) + (int64_t)head * a.tokens + st.start + row0,
                        4 * min(st.len - row0, QR)), lds_offset(stat[grp][b][w]), 4 * lane);
  };
  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[t] = f32x16{}, dv[t] = f32x16{};
    copy(0);
    wait_tiles();
    for (int it = 0; it * NG < total; ++it) {
      const char *ql = lds[grp][it & 1][0], *dl = lds[grp][it & 1][1];
      const float *ll = stat[grp][it & 1][0], *el = stat[grp][it & 1][1];
      const int q0 = (qt0 + (it * NG + grp) % nq) * QR;
      const int end = it * NG + grp < total ? st.len : 0;  // of the rows in this tile
      if ((it + 1) * NG < total) copy(it + 1);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (q0 + 32 * j + 31 < kw || q0 + 32 * j >= end) continue;  // rows before every key of this wave, or none
        f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
        for (int q = 0; q < ST; ++q) s = Elem<T>::mma(Tl::row_frag(ql, 32 * j + col, q, h), kf[q], s);
#pragma unroll
        for (int q = 0; q < ST; ++q) dp = Elem<T>::mma(Tl::row_frag(dl, 32 * j + col, q, h), vf[q], dp);
        float p[16], ds[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 lse2 = *(const f32x4*)(ll + 32 * j + 8 * g + 4 * h);
          const f32x4 del = *(const f32x4*)(el + 32 * j + 8 * g + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * g + e;
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse2[e]));
            ds[i] = p[i] * (dp[i] - del[e]);
          }
        }
        // A row before some key, or past the last one: it is all zeros, but 0 times a key's infinity is NaN.
        if (q0 + 32 * j < kw + 31 || q0 + 32 * j + 32 > end) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = q0 + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3);
            if (row < ki || row >= end) p[i] = ds[i] = 0.f;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const Frag pf = Elem<T>::pack(p + 8 * u), sf = Elem<T>::pack(ds + 8 * u);
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            Frag of = Tl::col_frag(dl, 32 * j + 16 * u, t, lane), qf = Tl::col_frag(ql, 32 * j + 16 * u, t, lane);
            if (careful.value) {
              const bool diag = q0 + 32 * j < kw + 31;
              of = finite_part<T>(of, diag), qf = finite_part<T>(qf, diag);
            }
            dv[t] = Elem<T>::mma(of, pf, dv[t]);
            dk[t] = Elem<T>::mma(qf, sf, dk[t]);
          }
        }
      }
      wait_tiles();
    }
  };
  pass(std::false_type{});
  if (any_nan<NG * WR>(not_finite(dk) + not_finite(dv), flags, grp * WR + w)) {
    pass(std::true_type{});
    if (grp == 0 && valid)
      for (int head = head0; head < head0 + hpp; ++head) {
        const int64_t t0 = st.start + (int64_t)kw;
        const int rows = min(32, st.len - kw);
        add_not_finite<T, DP>(dk, (const T*)a.q.data + t0 * a.q.token + head * a.q.head, a.q.token, rows, col, 31, 0.f,
                              a.dim, h);
        add_not_finite<T, DP>(dv, (const T*)a.dout.data + t0 * a.dout.token + head * a.dout.head, a.dout.token, rows,
                              col, 31, 1.f, a.dim, h);
      }
  }
  if constexpr (NG > 1) {
    static_assert(kJoin<DT, WR, NG> <= sizeof(lds), "the sums fit the tiles");
    join_groups<WR, NG>(dk, (float*)lds, grp, w, lane);
    if (join_groups<WR, NG>(dv, (float*)lds, grp, w, lane)) return;
  }
  if (!valid) return;
  if (a.splits == 1) {
    store_row<T, DP>((T*)a.dk.data + tok * a.dk.token + kvh * a.dk.head, dk, a.scale, a.dim, h);
    store_row<T, DP>((T*)a.dv.data + tok * a.dv.token + kvh * a.dv.head, dv, 1.f, a.dim, h);
  } else {
    float* p = a.part + (((int64_t)part * a.tokens + tok) * a.kv_heads + kvh) * 2 * a.dim;
    store_row<float, DP>(p, dk, a.scale, a.dim, h);
    store_row<float, DP>(p + a.dim, dv, 1.f, a.dim, h);
  }
}

// The same in bf16.  Query rows stream through a ring of slots, 32 at a time
// into the products; their scores' sums start from -lse / scale and -delta, so
// p = exp2(c s) and ds = p dp.  Two blocks or three share a CU, as many waves a
// SIMD: with head sizes above 64, V's fragments are read from LDS again and
// again to fit the registers (held, they leave one wave a SIMD: 757 us on 8192
// tokens, 16/4 heads of 128, against 507, 1085 TFLOP/s).  At heads of 64, 64
// rows a step take 106 us on 16384 packed tokens, 32 rows 116.
template <int DP, int NG>
__global__ __launch_bounds__(NG * kThreads, kDkvWaves<DP>) void attention_dkv_bf16_kernel(AttnArgs a) {
  typedef __bf16 T;
  typedef Elem<T>::Frag Frag;
  typedef Tiles<T, DP> Tl;
  constexpr bool kHoldV = DP <= 64;
  constexpr int WR = 4, BN = 32 * WR, ST = DP / 16, DT = DP / 32, QR = DP <= 64 ? 64 : 32, kSlots = DP == 96 ? 4 : 2;
  typedef PairCopier<T, DP, QR, WR> Pair;
  constexpr int kSlot = 2 * Pair::kTile + 512;  // Q rows, dO rows, and two words a row
  __shared__ __align__(256) char lds[NG * kSlots * kSlot + (kHoldV ? 0 : BN * Tl::kRow)];
  __shared__ int flags[NG * WR];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, col = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6) % WR, grp = __builtin_amdgcn_readfirstlane(tid >> 6) / WR;
  char* const ring = lds + grp * kSlots * kSlot;
  const int per = a.kv_heads * a.splits;
  const int kvh = (int)(blockIdx.x % per) / a.splits, part = (int)(blockIdx.x % per) % a.splits;
  const SeqTile st = block_tile(a, (int)(blockIdx.x / per), (int)(gridDim.x / per), BN, lane, true);
  if (st.row0 >= st.len) return;
  if (st.tail) {
    const int rows = min(BN, st.len - st.row0), r0 = st.start + st.row0;
    if (part == 0 && (a.zero_tail & kZeroDk)) zero_rows<T>(a.dk, kvh, r0, rows, a.dim, tid);
    if (part == 0 && (a.zero_tail & kZeroDv)) zero_rows<T>(a.dv, kvh, r0, rows, a.dim, tid);
    return;
  }
  const int kw = st.row0 + 32 * w, ki = kw + col;
  const bool valid = ki < st.len;
  const int64_t tok = st.start + (int64_t)ki;
  const float c = a.scale * kLog2e;
  const int hpp = a.group / a.splits, head0 = kvh * a.group + part * hpp;  // this block's query heads

  char* const vt = lds + NG * kSlots * kSlot;
  Frag kf[ST], vf[kHoldV ? ST : 1];
  load_frags<T, DP>(kf, (const T*)a.k.data + tok * a.k.token + kvh * a.k.head, valid, a.dim, h);
  if constexpr (kHoldV) {
    load_frags<T, DP>(vf, (const T*)a.v.data + tok * a.v.token + kvh * a.v.head, valid, a.dim, h);
  } else {  // two tiles of V's rows, by a copier of its own
    PairCopier<T, DP, BN / 2, WR> cv;
    cv.init(a.v, a.v, a.dim, w, lane);
    cv.seek(a.v, kvh, a.v, kvh, st.start + (int64_t)st.row0 + (w < 2 ? 0 : BN / 2),
            st.len - st.row0 - (w < 2 ? 0 : BN / 2), w);
    if (grp == 0) cv.template copy<1>(vt, w, lane);
  }
  f32x16 dk[DT], dv[DT];

  // The rows to copy next: their slot, head and words (even waves copy the first, odd ones the second).
  Pair cp;
  cp.init(a.q, a.dout, a.dim, w, lane);
  int cslot, chead, crow;
  const float* words;
  auto next = [&](int& head, int& row) {
    row += QR;
    if (row >= st.len) row = st.row0, ++head;
  };
  auto seek = [&]() {
    const int64_t t0 = st.start + (int64_t)crow;
    cp.seek(a.q, chead, a.dout, chead, t0, chead < head0 + hpp ? st.len - crow : 0, w);
    words = (w & 1 ? a.delta : a.lse2) + (int64_t)chead * a.tokens + t0;
  };
  auto copy = [&]() {
    char* sl = ring + cslot * kSlot;
    dma_b32(buffer_of(words, 4 * max(min(cp.left, QR), 0)), lds_offset(sl + 2 * Pair::kTile + 256 * (w & 1)),
            4 * lane);
    words += NG * QR;
    cp.template copy<NG>(sl, w, lane);
    cslot = (cslot + 1) & (kSlots - 1);
    const int head = chead;
#pragma unroll
    for (int i = 0; i < NG; ++i) next(chead, crow);
    if (chead != head) seek();
  };
  auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < DT; ++t) dk[t] = f32x16{}, dv[t] = f32x16{};
    cslot = 0, chead = head0, crow = st.row0;
    int row = st.row0, rhead = head0;  // the rows in hand
    if (grp) next(chead, crow), next(rhead, row);
    seek();
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) copy();
    const int total = ((st.len - st.row0 + QR - 1) / QR * hpp + NG - 1) / NG;
    for (int i = 0; i < total; ++i) {
      wait_but<(kSlots - 2) * (Pair::kN + 1)>();
      copy();
      const char* sl = ring + (i & (kSlots - 1)) * kSlot;
      const int end = NG > 1 && rhead >= head0 + hpp ? 0 : st.len;  // of the rows in this slot
#pragma unroll 1
      for (int j = 0; j < QR; j += 32) {
        if (careful.value && row + j + 31 < kw) continue;  // rows before every key of this wave
        const char *ql = sl + j * Tl::kRow, *ol = ql + Pair::kTile;
        f32x16 s, dp;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 x = *(const f32x4*)(sl + 2 * Pair::kTile + 4 * j + 32 * g + 16 * h);
          const f32x4 y = *(const f32x4*)(sl + 2 * Pair::kTile + 256 + 4 * j + 32 * g + 16 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[4 * g + e] = x[e], dp[4 * g + e] = y[e];
        }
#pragma unroll
        for (int q = 0; q < ST; ++q) {
          s = Elem<T>::mma(Tl::row_frag(ql, col, q, h), kf[q], s);
          if constexpr (kHoldV)
            dp = Elem<T>::mma(Tl::row_frag(ol, col, q, h), vf[q], dp);
          else
            dp = Elem<T>::mma(Tl::row_frag(ol, col, q, h), Tl::row_frag(vt, 32 * w + col, q, h), dp);
        }
        // A row before some key, or past the last one: it is all zeros, but 0 times a key's infinity is NaN.
        if (row + j < kw + 31 || row + j + 32 > end) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = row + j + 8 * (e >> 2) + 4 * h + (e & 3) - ki;  // rows behind the lane's key
            if ((uint32_t)r >= (uint32_t)max(end - ki, 0)) s[e] = -__builtin_inff(), dp[e] = 0.f;
          }
        }
        float p[16], ds[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          p[e] = __builtin_amdgcn_exp2f(s[e] * c);
          ds[e] = p[e] * dp[e];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const Frag pf = Elem<T>::pack(p + 8 * u), sf = Elem<T>::pack(ds + 8 * u);
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            Frag of = Tl::col_frag(ol, 16 * u, t, lane), qf = Tl::col_frag(ql, 16 * u, t, lane);
            if (careful.value) of = finite_part<T>(of, row + j < kw + 31), qf = finite_part<T>(qf, row + j < kw + 31);
            dv[t] = Elem<T>::mma(of, pf, dv[t]);
            dk[t] = Elem<T>::mma(qf, sf, dk[t]);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) next(rhead, row);
    }
  };
  pass(std::false_type{});
  if (any_nan<NG * WR>(not_finite(dk) + not_finite(dv), flags, grp * WR + w)) {
    wait_tiles();  // the copies of rows past the last
    pass(std::true_type{});
    if (grp == 0 && valid)
      for (int head = head0; head < head0 + hpp; ++head) {
        const int64_t t0 = st.start + (int64_t)kw;
        const int rows = min(32, st.len - kw);
        add_not_finite<T, DP>(dk, (const T*)a.q.data + t0 * a.q.token + head * a.q.head, a.q.token, rows, col, 31, 0.f,
                              a.dim, h);
        add_not_finite<T, DP>(dv, (const T*)a.dout.data + t0 * a.dout.token + head * a.dout.head, a.dout.token, rows,
                              col, 31, 1.f, a.dim, h);
      }
  }
  if constexpr (NG > 1) {
    static_assert(kJoin<DT, WR, NG> <= sizeof(lds), "the sums fit the tiles");
    join_groups<WR, NG>(dk, (float*)lds, grp, w, lane);
    if (join_groups<WR, NG>(dv, (float*)lds, grp, w, lane)) return;
  }
  if (!valid) return;
  if (a.splits == 1) {
    store_row<T, DP>((T*)a.dk.data + tok * a.dk.token + kvh * a.dk.head, dk, a.scale, a.dim, h);
    store_row<T, DP>((T*)a.dv.data + tok * a.dv.token + kvh * a.dv.head, dv, 1.f, a.dim, h);
  } else {
    float* p = a.part + (((int64_t)part * a.tokens + tok) * a.kv_heads + kvh) * 2 * a.dim;
    store_row<float, DP>(p, dk, a.scale, a.dim, h);
    store_row<float, DP>(p + a.dim, dv, 1.f, a.dim, h);
  }
}

// Sums the parts of a split group in their order: part[split][token][kv head][dK, dV][dim].
// Bound by memory: 4 parts of 8192 tokens and 4 heads of 128 (134 MB) in 22 us, 6.1 TB/s (most of it from the Infinity Cache).
template <class T>
__global__ __launch_bounds__(kThreads) void attention_sum_kernel(AttnArgs a) {
  const int per = a.kv_heads * 2 * a.dim / 4;  // groups of 4 elements a token
  const int64_t total = (int64_t)(token_at(a, a.seqs) - token_at(a, 0)) * per, first = (int64_t)token_at(a, 0) * per;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t tok = (first + i) / per;
    const int at = (int)((first + i) % per), kvh = at / (a.dim / 2), e = at % (a.dim / 2) * 4;
    f32x4 s = f32x4{};
    for (int p = 0; p < a.splits; ++p) {
      const f32x4 x = *gv<f32x4>(a.part + ((int64_t)p * a.tokens * per + first + i) * 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += x[q];
    }
    const HeadView& v = e < a.dim ? a.dk : a.dv;
    T* row = (T*)v.data + tok * v.token + kvh * v.head + (e < a.dim ? e : e - a.dim);
    if constexpr (sizeof(T) == 2)
      *gv<u32x2>(row) = pack4_bf16(s[0], s[1], s[2], s[3]);
    else
      *gv<f32x4>(row) = s;
  }
}

// Blocks of two groups of waves, which share a tile's streamed side and join
// their sums, halve a block's run: worth it while the grid is about what the
// 256 CUs hold at once and the longest block decides.  Forward and backward, 12
// heads of 64 (one group / two): 4096 tokens 76 / 54 and 171 / 127 us; 8192
// tokens (792 blocks) 157 / 135 and 419 / 414; 16 heads of 128, 8192 tokens
// (1056 blocks) 281 / 295 and 927 / 948.  Short sequences only pay for the
// join: 32 of 512 tokens 35 / 42 and 100 / 142.
inline bool two_groups(const AttnArgs& a, int64_t blocks) {
  return blocks <= 800 && a.tokens >= 256 * (int64_t)a.seqs;
}
// fp32 products are 16 times slower than bf16 ones, so a block of 128 rows runs
// long, and K and V need not be shared by as many rows: up to head size 64, a
// block takes 64 rows and four groups of two waves (2048 tokens in 5
// sequences, 12 heads of 64: forward and backward 71 and 226 us with 128 rows
// and two groups, 43 and 138 with this).
template <class T, int DP>
constexpr bool kNarrow = sizeof(T) == 4 && DP <= 64;
constexpr int64_t grid_of(const AttnArgs& a, int heads, int bm) { return slots_of(a.tokens, a.seqs, bm) * heads; }

template <class T, int DP>
hipError_t forward_dp(const AttnArgs& a, hipStream_t stream) {
  if constexpr (kNarrow<T, DP>) {
    return launch_kernel(attention_forward_kernel<T, DP, 2, 4>, grid_of(a, a.q_heads, 64), 512, a, stream);
  } else {
    const int64_t grid = grid_of(a, a.q_heads, 128);
    return two_groups(a, grid) ? launch_kernel(attention_forward_kernel<T, DP, 4, 2>, grid, 512, a, stream)
                               : launch_kernel(attention_forward_kernel<T, DP, 4, 1>, grid, 256, a, stream);
  }
}

template <class T, int DP>
hipError_t backward_dp(const AttnArgs& a, hipStream_t stream) {
  hipError_t e;
  if constexpr (kNarrow<T, DP>) {
    e = launch_kernel(attention_dq_kernel<T, DP, 2, 4>, grid_of(a, a.q_heads, 64), 512, a, stream);
    if (e == hipSuccess)
      e = launch_kernel(attention_dkv_kernel<DP, 2, 4>, grid_of(a, a.kv_heads * a.splits, 64), 512, a, stream);
  } else {
    const int64_t gq = grid_of(a, a.q_heads, 128), gk = grid_of(a, a.kv_heads * a.splits, 128);
    // fp32 at heads of 128: one group and one wave a SIMD.  With two of either, 145 registers spill: 2048 tokens of
    // 12 heads 977 and 1079 us backward, 128 tokens of 8/2 heads 188 and 202.
    if constexpr (sizeof(T) == 4 && DP == 128)
      e = launch_kernel(attention_dq_kernel<T, DP, 4, 1>, gq, 256, a, stream);
    else
      e = two_groups(a, gq) ? launch_kernel(attention_dq_kernel<T, DP, 4, 2>, gq, 512, a, stream)
                            : launch_kernel(attention_dq_kernel<T, DP, 4, 1>, gq, 256, a, stream);
    if (e != hipSuccess) return e;
    if constexpr (sizeof(T) == 2)
      e = two_groups(a, gk) ? launch_kernel(attention_dkv_bf16_kernel<DP, 2>, gk, 512, a, stream)
                            : launch_kernel(attention_dkv_bf16_kernel<DP, 1>, gk, 256, a, stream);
    else  // two groups do not fit the registers of two waves a SIMD
      e = launch_kernel(attention_dkv_kernel<DP, 4, 1>, gk, 256, a, stream);
  }
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t blocks = (a.tokens * a.kv_heads * 2 * a.dim / 4 + kThreads - 1) / kThreads;
  return launch_kernel(attention_sum_kernel<T>, blocks < 4096 ? blocks : 4096, kThreads, a, stream);
}

template <class T>
hipError_t by_dim(const AttnArgs& a, bool backward, hipStream_t s) {
  switch ((a.dim + 31) / 32) {
    case 1: return backward ? backward_dp<T, 32>(a, s) : forward_dp<T, 32>(a, s);
    case 2: return backward ? backward_dp<T, 64>(a, s) : forward_dp<T, 64>(a, s);
    case 3: return backward ? backward_dp<T, 96>(a, s) : forward_dp<T, 96>(a, s);
    default: return backward ? backward_dp<T, 128>(a, s) : forward_dp<T, 128>(a, s);
  }
}

}  // namespace

// Query heads that share a key/value head are split over several blocks when
// the whole groups give too few blocks for the 256 CUs, and the sequences are
// long enough to pay for the sum's launch (a block's steps of 64 rows, 0.6 us
// each, against 4 us).
int attention_splits(int64_t tokens, int seqs, int q_heads, int kv_heads) {
  const int group = q_heads / kv_heads;
  if (tokens * group < 2048 * (int64_t)seqs) return 1;
  const int64_t blocks = (tokens / 128 + 1) * kv_heads;
  int s = 1;
  for (int d = 1; d <= group && blocks * s < 1024; ++d)
    if (group % d == 0) s = d;
  return s;
}

int64_t attention_threads(int64_t tokens, int seqs, int q_heads, int dim, bool bf16) {
  const bool narrow = !bf16 && dim <= 64;  // kNarrow
  return slots_of(tokens, seqs, narrow ? 64 : 128) * q_heads * (narrow ? 512 : 256);
}

hipError_t launch_attention_forward(const AttnArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? by_dim<__bf16>(a, false, stream) : by_dim<float>(a, false, stream);
}
hipError_t launch_attention_backward(const AttnArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? by_dim<__bf16>(a, true, stream) : by_dim<float>(a, true, stream);
}

}  // namespace muon
