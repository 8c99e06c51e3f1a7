// gfx950 (CDNA4) embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: y[t] = scale * table[id_t]; an id outside the table gives a row of zeros.
// Backward: dtable[v] = scale * sum of dout[t] over the tokens t with id_t = v, in
// fp32 and in an order that only the ids and sizes decide: the tokens are sorted
// by id (stable radix sort, so in token order within an id), groups of lanes sum
// chunks of the sorted list, and ids that reach over a chunk's end are joined in
// order.
//
// Bound by memory: forward, 65536 rows of 768 in bf16 out of 50304 take 26 to 31
// us (126 MB, 4.1 to 4.9 TB/s).  Backward, the table's zeros (77 MB: 12 us alone)
// are written while the tokens are sorted, 26 us in four launches that latency
// bounds; sums 30 us (100 MB read in the ids' order, 25 written, 4.2 TB/s), joining 8.
#include "block_internal.h"
#include "device_common.h"
#include "row_vectors.h"
#include "wave.h"

namespace muon {
namespace {

// The id of a token as the table's row, or `vocab` outside it.
__device__ __forceinline__ int64_t load_id(const void* ids, bool id64, int64_t t) {
  return id64 ? *gv<int64_t>((const int64_t*)ids + t) : *gv<int32_t>((const int32_t*)ids + t);
}
__device__ __forceinline__ uint32_t row_of(int64_t id, int64_t vocab) {
  return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}
__device__ __forceinline__ uint32_t id_at(const void* ids, bool id64, int64_t t, int64_t vocab) {
  return row_of(load_id(ids, id64, t), vocab);
}

// ---------------------------------------------------------------- forward --
// A block takes a.rows tokens, whose ids it holds in LDS, and its threads the
// vectors of those rows in turn.
constexpr int kMaxRows = 256;
template <class T, class O, bool PART>
__global__ __launch_bounds__(kThreads) void embed_forward_kernel(EmbedArgs a) {
  constexpr int VEC = sizeof(T) == 4 && sizeof(O) == 4 ? 4 : 8, AHEAD = 4;
  __shared__ uint32_t id[kMaxRows];
  const uint32_t vectors = (uint32_t)(a.cols + VEC - 1) / VEC;
  for (int64_t first = (int64_t)blockIdx.x * a.rows; first < a.tokens; first += (int64_t)gridDim.x * a.rows) {
    const int rows = (int)min((int64_t)a.rows, a.tokens - first);
    __syncthreads();  // the ids before have been read
    for (int i = threadIdx.x; i < rows; i += kThreads) id[i] = id_at(a.ids, a.id64, first + i, a.vocab);
    __syncthreads();
    const uint32_t count = rows * vectors;
    for (uint32_t j0 = threadIdx.x; j0 < count; j0 += AHEAD * kThreads) {
      float v[AHEAD][VEC];
      uint32_t row[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const uint32_t j = j0 + q * kThreads;
        row[q] = a.rows == 1 ? 0 : vectors == 1 ? j : __umulhi(j, a.magic);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[q][e] = 0.f;
        if (j >= count || id[row[q]] >= (uint32_t)a.vocab) continue;
        const int c = (int)(j - row[q] * vectors) * VEC;
        load_part<T, VEC, PART>((const T*)a.table + id[row[q]] * a.ld_table + c, PART ? min(a.cols - c, VEC) : VEC, v[q]);
      }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        const uint32_t j = j0 + q * kThreads;
        if (j >= count) break;
        const int c = (int)(j - row[q] * vectors) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[q][e] *= a.scale;
        store_part<O, VEC, PART>((O*)a.out + (first + row[q]) * a.ld_out + c, PART ? min(a.cols - c, VEC) : VEC, v[q]);
      }
    }
  }
}

// ------------------------------------------------------------------- zeros --
// Rows that no token has are zero, so the launches that sort, which leave most
// of the GPU idle, set the whole gradient to zero in their other blocks: `part`
// of `parts`.  What the sums write over is written twice, which costs less than
// knowing it first.
__device__ __forceinline__ void zero_table(const EmbedGradArgs& a, int es, int64_t block, int64_t blocks, int part,
                                           int parts) {
  const bool whole = a.ld_dtable == a.cols;  // one row of everything
  const int64_t rows = whole ? 1 : a.vocab, bytes = (whole ? a.vocab : 1) * a.cols * es;
  const int lane = threadIdx.x % 64, waves = blockDim.x / 64;
  constexpr int kPiece = 64 * 16 * 4;  // of a wave
  const int64_t pieces = (bytes + kPiece - 1) / kPiece, all = rows * pieces;
  const int64_t end = all * (part + 1) / parts;
  for (int64_t i = all * part / parts + block * waves + threadIdx.x / 64; i < end; i += blocks * waves) {
    const int64_t row = whole ? 0 : i / pieces, at = (whole ? i : i - row * pieces) * kPiece;
    char* p = (char*)a.dtable + row * a.ld_dtable * es + at;
    const int64_t n = bytes - at;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = (q * 64 + lane) * 16;
      if (o + 16 <= n) *gv<u32x4_any>(p + o) = u32x4{};
      else
        for (int e = o; e < n; e += 2) *gv<uint16_t>(p + e) = 0;
    }
  }
}

// ------------------------------------------------------------------- sort --
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// The rank of a lane's digit among equal ones of lower lanes, and their number in the wave.
__device__ __forceinline__ int rank_of(uint32_t d, int bits, bool on, int& count) {
  const uint64_t all = __ballot(on);
  uint32_t lo = (uint32_t)all, hi = (uint32_t)(all >> 32);
  for (int b = 0; b < bits; ++b) {
    const uint32_t bit = (uint32_t)__builtin_amdgcn_sbfe((int)d, b, 1);  // 0 or all ones
    const uint64_t set = __ballot(bit);
    lo &= ~((uint32_t)set ^ bit);
    hi &= ~((uint32_t)(set >> 32) ^ bit);
  }
  count = __popc(lo) + __popc(hi);
  return __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
}

// Exclusive sums over the block's threads.
__device__ __forceinline__ uint32_t scan_threads(uint32_t v, uint32_t* wave_sum) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  uint32_t scan = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t n = __shfl_up(scan, o);
    if (lane >= o) scan += n;
  }
  if (lane == 63) wave_sum[wave] = scan;
  __syncthreads();
  uint32_t lower = scan - v;
  for (int w = 0; w < wave; ++w) lower += wave_sum[w];
  return lower;
}

// Not many tokens: one block sorts them in LDS, in as many passes as the ids' bits
// need.  A wave counts the digits of its own part of the list, so that the block
// only meets to add the waves' counts and to move the entries.  The whole
// backward pass of 4096 tokens takes 23 us for 50304 x 768 in bf16 and 20 for
// 5000 x 64 (35 and 26 with the launches below), of 8192 tokens 30 and 24 (35
// and 25; for a small table of 64 x 768 22 and 19).
template <int ITEMS>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(EmbedGradArgs a) {
  __shared__ EmbedEntry list[ITEMS * kSortThreads];
  __shared__ uint16_t place[kSortWaves][1 << kMaxDigit];
  __shared__ uint32_t wave_sum[kSortWaves];
  if (blockIdx.x > 0) return zero_table(a, a.table_size, blockIdx.x - 1, gridDim.x - 1, 0, 1);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, bins = 1 << a.digit, n = (int)a.tokens;
  const int rounds = (n + kSortThreads - 1) / kSortThreads, first = wave * rounds * 64 + lane;
  EmbedEntry e[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = first + i * 64;
    e[i] = EmbedEntry{0, (uint32_t)at};
    if (i < rounds && at < n) e[i].id = id_at(a.ids, a.id64, at, a.vocab);
  }
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit;
    int rank[ITEMS];
    for (int i = lane; i < bins; i += 64) place[wave][i] = 0;
    wave_fence();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (i >= rounds) break;
      const bool on = first + i * 64 < n;
      const uint32_t d = e[i].id >> shift & (bins - 1);
      int count;
      const int r = rank_of(d, a.digit, on, count), before = place[wave][d];
      wave_fence();
      if (on && r == 0) place[wave][d] = (uint16_t)(before + count);
      wave_fence();
      rank[i] = before + r;
    }
    __syncthreads();
    uint32_t total = 0;
    if ((int)threadIdx.x < bins)
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) total += place[w][threadIdx.x];
    uint32_t base = scan_threads(total, wave_sum);
    if ((int)threadIdx.x < bins)
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = place[w][threadIdx.x];
        place[w][threadIdx.x] = (uint16_t)base;
        base += c;
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (i < rounds && first + i * 64 < n) list[place[wave][e[i].id >> shift & (bins - 1)] + rank[i]] = e[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (i < rounds && first + i * 64 < n) e[i] = list[first + i * 64];
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (i < rounds && first + i * 64 < n) a.sorted[first + i * 64] = e[i];
}

// More tokens: a pass of two launches for each digit.  Every block counts its
// segment's digits, then every block finds its places from all blocks' counts
// and moves its entries there.  The tokens' order is kept among equals.
__device__ __forceinline__ EmbedEntry entry_at(const EmbedGradArgs& a, int64_t i) {
  if (a.pass == 0) return EmbedEntry{id_at(a.ids, a.id64, i, a.vocab), (uint32_t)i};
  return a.entry[(a.pass + 1) & 1][i];
}

__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedGradArgs a) {
  if ((int)blockIdx.x >= a.blocks)
    return zero_table(a, a.table_size, blockIdx.x - a.blocks, gridDim.x - a.blocks, 2 * a.pass, 2 * a.passes);
  __shared__ uint32_t count[1 << kMaxDigit];
  const int bins = 1 << a.digit;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.segment, last = min(first + a.segment, a.tokens);
  for (int64_t i = first + threadIdx.x; i < last; i += kSortThreads)
    atomicAdd(&count[entry_at(a, i).id >> (a.pass * a.digit) & (bins - 1)], 1u);
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) a.hist[(int64_t)blockIdx.x * bins + i] = count[i];
}

__global__ __launch_bounds__(kSortThreads) void embed_move_kernel(EmbedGradArgs a) {
  if ((int)blockIdx.x >= a.blocks)
    return zero_table(a, a.table_size, blockIdx.x - a.blocks, gridDim.x - a.blocks, 2 * a.pass + 1, 2 * a.passes);
  __shared__ uint32_t base[1 << kMaxDigit];               // where the digit's next entry goes
  __shared__ uint16_t place[kSortWaves][1 << kMaxDigit];  // a wave's count of a digit, then its place after base
  __shared__ uint32_t wave_sum[kSortWaves];
  __shared__ uint32_t sums[2][kSortThreads];
  const int bins = 1 << a.digit, lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  {
    // entries of lower digits, and of the same digit in earlier blocks: kSortThreads / bins threads a digit
    const int bin = threadIdx.x & (bins - 1), share = threadIdx.x >> a.digit, shares = kSortThreads >> a.digit;
    uint32_t before = 0, total = 0;
#pragma unroll 16
    for (int b = share; b < a.blocks; b += shares) {
      const uint32_t n = a.hist[(int64_t)b * bins + bin];
      before += b < (int)blockIdx.x ? n : 0;
      total += n;
    }
    sums[0][threadIdx.x] = before, sums[1][threadIdx.x] = total;
    __syncthreads();
    before = total = 0;
    if ((int)threadIdx.x < bins)
      for (int i = threadIdx.x; i < kSortThreads; i += bins) before += sums[0][i], total += sums[1][i];
    const uint32_t lower = scan_threads(total, wave_sum);
    if ((int)threadIdx.x < bins) base[threadIdx.x] = lower + before;
  }
  EmbedEntry* to = a.pass == a.passes - 1 ? a.sorted : a.entry[a.pass & 1];
  const int64_t first = (int64_t)blockIdx.x * a.segment, last = min(first + a.segment, a.tokens);
  for (int64_t at = first; at < last; at += kSortThreads) {
    const int64_t i = at + threadIdx.x;
    const bool on = i < last;
    const EmbedEntry e = on ? entry_at(a, i) : EmbedEntry{};
    for (int b = lane; b < bins; b += 64) place[wave][b] = 0;
    wave_fence();
    const uint32_t d = e.id >> (a.pass * a.digit) & (bins - 1);
    int count;
    const int rank = rank_of(d, a.digit, on, count);
    if (on && rank == 0) place[wave][d] = (uint16_t)count;
    __syncthreads();
    uint32_t sum = 0;
    if ((int)threadIdx.x < bins) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t n = place[w][threadIdx.x];
        place[w][threadIdx.x] = (uint16_t)sum;
        sum += n;
      }
    }
    __syncthreads();
    if (on) to[base[d] + place[wave][d] + rank] = e;
    __syncthreads();  // base and place have been read
    if ((int)threadIdx.x < bins) base[threadIdx.x] += sum;
  }
}

// -------------------------------------------------------------------- sums --
template <class T, int VEC, bool PART>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, uint32_t id, int c, int n, float* v) {
  T* p = (T*)a.dtable + id * a.ld_dtable + c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= a.scale;
  if (a.accumulate) {
    float old[VEC];
    load_part<T, VEC, PART>(p, n, old);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] += old[e];
  }
  store_part<T, VEC, PART>(p, n, v);
}

// A vector of a row as it was loaded: whole ones of bf16 stay packed, in half the
// registers.  Rows of more than the caches keep are read past them (whole
// vectors): 65536 x 768 in bf16 30 us instead of 35, but 32768 x 128, which the
// caches hold, 12 instead of 11 (96 and 8 MiB; the rule's 32 lies between them, no
// size between was measured).
template <class O, bool PART, bool STREAM>
struct Held {
  float v[kVec<O>];
  __device__ __forceinline__ void load(const O* p, int n) {
    if constexpr (STREAM) {
#pragma unroll
      for (int e = 0; e < kVec<O>; e += 4) {
        const f32x4 r = __builtin_nontemporal_load(gv<f32x4_any>(p + e));
        v[e] = r[0], v[e + 1] = r[1], v[e + 2] = r[2], v[e + 3] = r[3];
      }
    } else {
      load_part<O, kVec<O>, PART>(p, n, v);
    }
  }
  __device__ __forceinline__ void add_to(float* acc) const {
#pragma unroll
    for (int e = 0; e < kVec<O>; ++e) acc[e] += v[e];
  }
};
template <bool STREAM>
struct Held<__bf16, false, STREAM> {
  u32x4 r;
  __device__ __forceinline__ void load(const __bf16* p, int) {
    if constexpr (STREAM) r = __builtin_nontemporal_load(gv<u32x4_any>(p));
    else r = *gv<u32x4_any>(p);
  }
  __device__ __forceinline__ void add_to(float* acc) const {
    float v[8];
    unpack8_bf16(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += v[e];
  }
};

// A block sums a chunk of the sorted list over LPR vectors of columns: each group
// of LPR lanes EACH entries, whose rows it loads at once.  An id's run that lies
// within a group goes to its row of the table; parts of longer ones go to LDS,
// where the group in which a run starts adds the others' (in order).  A run that
// came in from the chunk before ends in part[chunk][0], one that goes on from
// here in part[chunk][1].
template <class T, class O, bool PART, int LPR, int EACH, bool STREAM>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<O>, GROUPS = kThreads / LPR, CHUNK = GROUPS * EACH;
  __shared__ EmbedEntry list[CHUNK + 2];  // one entry before and behind the chunk
  __shared__ __align__(16) float parts[2][GROUPS][LPR * VEC];  // of a group's run that came in, of one that goes on
  const int u = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const uint32_t none = (uint32_t)a.vocab;  // ids outside the table are sorted last, and what is behind the list follows
  const int slices = (a.cols + LPR * VEC - 1) / (LPR * VEC);
  const int64_t chunks = (a.tokens + CHUNK - 1) / CHUNK;
  auto came_in = [&](int g) { return list[g * EACH].id == list[g * EACH + 1].id; };
  auto goes_on = [&](int g) {  // and the run
    const uint32_t id = list[(g + 1) * EACH].id;
    return id == list[(g + 1) * EACH + 1].id && id < none;
  };
  auto passes = [&](int g) { return goes_on(g) && list[g * EACH + 1].id == list[(g + 1) * EACH].id; };
  for (int64_t unit = blockIdx.x; unit < chunks * slices; unit += gridDim.x) {
    const int64_t chunk = unit / slices, first = chunk * CHUNK - 1;
    const int c = ((int)(unit % slices) * LPR + u) * VEC, n = min(a.cols - c, VEC);
    __syncthreads();  // the unit before is done
    for (int k = threadIdx.x; k < CHUNK + 2; k += kThreads)
      list[k] = first + k >= 0 && first + k < a.tokens ? a.sorted[first + k] : EmbedEntry{none + 1 + (k == 0), 0};
    __syncthreads();
    const EmbedEntry* mine = list + group * EACH + 1;
    Held<O, PART, STREAM> v[EACH];
    float acc[VEC];
#pragma unroll
    for (int q = 0; q < EACH; ++q)
      if (mine[q].id < none && n > 0) v[q].load((const O*)a.dout + mine[q].token * a.ld_dout + c, n);
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    bool started = !came_in(group);  // the run, in this group
#pragma unroll
    for (int q = 0; q < EACH; ++q) {
      const uint32_t id = mine[q].id, next = mine[q + 1].id;
      if (id >= none) break;
      v[q].add_to(acc);
      if (next == id && q + 1 < EACH) continue;
      if (!started || next == id) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) parts[started][group][u * VEC + e] = acc[e];
      } else if (n > 0) {
        write_row<T, VEC, PART>(a, id, c, n, acc);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      started = true;
    }
    __syncthreads();
    auto add = [&](int g) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += parts[0][g][u * VEC + e];
    };
    if (goes_on(group) && !(came_in(group) && passes(group))) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = parts[1][group][u * VEC + e];
      int g = group;
      bool on = true;
      while (on && ++g < GROUPS) add(g), on = passes(g);
      if (n > 0) {
        if (on) store_part<float, VEC, PART>(a.part + (chunk * 2 + 1) * a.cols + c, n, acc);
        else write_row<T, VEC, PART>(a, mine[EACH - 1].id, c, n, acc);
      }
    }
    if (group == 0 && came_in(0) && mine[0].id < none) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      int g = 0;
      do add(g);
      while (passes(g) && ++g < GROUPS);
      if (n > 0) store_part<float, VEC, PART>(a.part + chunk * 2 * a.cols + c, n, acc);
    }
  }
}

// Adds the parts of the ids that reach over chunks: a block for the chunk where
// an id's run starts, and a slice of the columns; its groups share the parts
// between them.
template <class T, class O, bool PART, int LPR, int EACH>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<O>, GROUPS = kThreads / LPR, CHUNK = GROUPS * EACH;
  __shared__ __align__(16) float red[GROUPS][LPR * VEC];
  const int lane = threadIdx.x % 64, u = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int slices = (a.cols + LPR * VEC - 1) / (LPR * VEC);
  for (int64_t unit = blockIdx.x;; unit += gridDim.x) {
    const int64_t chunk = unit / slices, first = chunk * CHUNK, end = first + CHUNK;
    if (end >= a.tokens) return;
    const uint32_t before = first > 0 ? a.sorted[first - 1].id : 0xFFFFFFFFu, start = a.sorted[first].id,
                   id = a.sorted[end - 1].id, next = a.sorted[end].id;
    if (id == (uint32_t)a.vocab || next != id || (start == id && before == id)) continue;  // not the first of several
    int64_t parts = 1;
    for (;; parts += 64) {
      const int64_t i = (chunk + parts + lane) * CHUNK;
      const uint64_t on = __ballot(i < a.tokens && a.sorted[i].id == id);
      if (~on) {
        parts += __builtin_ctzll(~on);
        break;
      }
    }
    const int c = ((int)(unit % slices) * LPR + u) * VEC, n = min(a.cols - c, VEC);
    float acc[VEC], v[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    if (n > 0)
#pragma unroll 8
      for (int64_t k = group; k < parts; k += GROUPS) {
        load_part<float, VEC, PART>(a.part + ((chunk + k) * 2 + (k == 0 ? 1 : 0)) * a.cols + c, n, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      }
    __syncthreads();  // the unit before has been read
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[group][u * VEC + e] = acc[e];
    __syncthreads();
    if (group == 0 && n > 0) {
      for (int g = 1; g < GROUPS && g < parts; ++g)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += red[g][u * VEC + e];
      write_row<T, VEC, PART>(a, id, c, n, acc);
    }
  }
}

// ------------------------------------------------------------------ direct --
// Few tokens: one launch, whose blocks each take some rows of the table, look
// through all ids for those of their rows (stably sorted by row in LDS, as
// above), and write every row, zeros first.  A row of many tokens is shared by
// all groups of lanes.  Alone on the GPU, against the launches that sort: 512
// tokens for 50304 x 768 in bf16 16 us instead of 22, for 5000 x 256 7 instead
// of 17, for 64 x 768 8 instead of 12; all of them of one id 32 instead of 23
// (50304 x 768; 256 tokens 22 and 22).  1024 tokens took 19 instead of 23 and 61
// instead of 23, so they are sorted.  The tokens alone decide, which loses for
// tables of few wide rows (512 tokens of 2 x 4096 61 us, 513, which are sorted, 14)
// and for adding to very large ones (one token into 2^24 x 64 in fp32 143 us, 513
// tokens 15; into 2^20 x 64 12 and 14).
constexpr int kDirectItems = kDirect / kThreads, kDirectWaves = kThreads / 64, kShared = 8;
template <class T, class O, bool PART, int LPR>
__global__ __launch_bounds__(kThreads) void embed_direct_kernel(EmbedGradArgs a) {
  constexpr int VEC = kVec<O>, GROUPS = kThreads / LPR;
  __shared__ uint16_t place[kDirectWaves][kDirectRows];
  __shared__ uint16_t start[kDirectRows + 1];
  __shared__ uint16_t list[kDirect];  // tokens by row
  __shared__ uint16_t present[kDirectRows];
  __shared__ uint32_t counts[2];
  __shared__ uint32_t wave_sum[kDirectWaves];
  __shared__ __align__(16) float red[GROUPS][LPR * VEC];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, u = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int n = (int)a.tokens, rows = (int)min((int64_t)a.segment, a.vocab - (int64_t)blockIdx.x * a.segment);
  const uint32_t row0 = blockIdx.x * (uint32_t)a.segment;
  int64_t id[kDirectItems];
#pragma unroll
  for (int i = 0; i < kDirectItems; ++i) {
    const int t = (wave * kDirectItems + i) * 64 + lane;
    id[i] = t < n ? load_id(a.ids, a.id64, t) : -1;
  }
  if (!a.accumulate) {  // all of the block's rows, while the ids are on their way; sums are written over them
    char* p = (char*)a.dtable + row0 * a.ld_dtable * a.table_size;
    const int64_t width = (int64_t)a.cols * a.table_size, bytes = rows * width;
    if (a.ld_dtable == a.cols) {
      for (int64_t o = threadIdx.x * 16; o < bytes; o += kThreads * 16) {
        if (o + 16 <= bytes) *gv<u32x4_any>(p + o) = u32x4{};
        else
          for (int64_t e = o; e < bytes; e += 2) *gv<uint16_t>(p + e) = 0;
      }
    } else {
      const float zero[VEC] = {};
      for (int r = group; r < rows; r += GROUPS)
        for (int c = u * VEC; c < a.cols; c += LPR * VEC)
          store_part<T, VEC, PART>((T*)p + r * a.ld_dtable + c, min(a.cols - c, VEC), zero);
    }
  }
  uint32_t row[kDirectItems];
  bool on[kDirectItems];
#pragma unroll
  for (int i = 0; i < kDirectItems; ++i) {
    row[i] = row_of(id[i], a.vocab) - row0;
    on[i] = row[i] < (uint32_t)rows;
    row[i] = on[i] ? row[i] : 0;
  }
  for (int i = lane; i < rows; i += 64) place[wave][i] = 0;
  if (threadIdx.x < 2) counts[threadIdx.x] = 0;
  wave_fence();
  int rank[kDirectItems];
#pragma unroll
  for (int i = 0; i < kDirectItems; ++i) {
    int count;
    const int r = rank_of(row[i], a.digit, on[i], count), before = place[wave][row[i]];
    wave_fence();
    if (on[i] && r == 0) place[wave][row[i]] = (uint16_t)(before + count);
    wave_fence();
    rank[i] = before + r;
  }
  __syncthreads();
  constexpr int EACH = kDirectRows / kThreads;  // rows of a thread
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i)
#pragma unroll
    for (int w = 0; w < kDirectWaves; ++w)
      if ((int)threadIdx.x * EACH + i < rows) mine += place[w][threadIdx.x * EACH + i];
  uint32_t base = scan_threads(mine, wave_sum);
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = threadIdx.x * EACH + i;
    if (b >= rows) continue;
    start[b] = (uint16_t)base;
#pragma unroll
    for (int w = 0; w < kDirectWaves; ++w) {
      const uint32_t c = place[w][b];
      place[w][b] = (uint16_t)base;
      base += c;
    }
    if (b == rows - 1) start[rows] = (uint16_t)base;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDirectItems; ++i)
    if (on[i]) list[place[wave][row[i]] + rank[i]] = (uint16_t)((wave * kDirectItems + i) * 64 + lane);
  __syncthreads();
  // rows with tokens, the shared ones from the end (in any order: each is a result of its own)
  for (int r = threadIdx.x; r < rows; r += kThreads) {
    const int count = start[r + 1] - start[r];
    if (count > 0 && count <= kShared) present[atomicAdd(&counts[0], 1)] = (uint16_t)r;
    if (count > kShared) present[kDirectRows - 1 - atomicAdd(&counts[1], 1)] = (uint16_t)r;
  }
  __syncthreads();
  auto sum = [&](auto ahead, int from, int to, int step, int c, int cn, float* acc) {
    constexpr int AHEAD = decltype(ahead)::value;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    for (int k = from; k < to; k += step * AHEAD) {
      Held<O, PART, false> v[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
        if (k + q * step < to) v[q].load((const O*)a.dout + list[k + q * step] * a.ld_dout + c, cn);
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
        if (k + q * step < to) v[q].add_to(acc);
    }
  };
  const int slices = (a.cols + LPR * VEC - 1) / (LPR * VEC);
  for (int i = group; i < (int)counts[0] * slices; i += GROUPS) {
    const int r = present[i / slices], c = (i % slices * LPR + u) * VEC, cn = min(a.cols - c, VEC);
    if (cn <= 0) continue;
    float acc[VEC];
    sum(std::integral_constant<int, 4>{}, start[r], start[r + 1], 1, c, cn, acc);
    write_row<T, VEC, PART>(a, row0 + r, c, cn, acc);
  }
  for (int i = 0; i < (int)counts[1]; ++i) {
    const int r = present[kDirectRows - 1 - i];
    for (int c0 = 0; c0 < a.cols; c0 += LPR * VEC) {
      const int c = c0 + u * VEC, cn = min(a.cols - c, VEC);
      float acc[VEC];
      sum(std::integral_constant<int, 16>{}, start[r] + group, cn > 0 ? start[r + 1] : 0, GROUPS, c, cn, acc);
      __syncthreads();  // the columns before have been read
#pragma unroll
      for (int e = 0; e < VEC; ++e) red[group][u * VEC + e] = acc[e];
      __syncthreads();
      if (group > 0 || cn <= 0) continue;
      for (int g = 1; g < GROUPS; ++g)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += red[g][u * VEC + e];
      write_row<T, VEC, PART>(a, row0 + r, c, cn, acc);
    }
  }
}

// The gradient of no tokens.
__global__ __launch_bounds__(kSortThreads) void embed_zero_kernel(EmbedGradArgs a) {
  zero_table(a, a.table_size, blockIdx.x, gridDim.x, 0, 1);
}

// ----------------------------------------------------------------- launch --
constexpr int64_t kMostBlocks = 1 << 20;  // what is left is taken in turn: a launch holds fewer than 2^32 threads
template <class T, class O>
hipError_t run_forward(const EmbedArgs& args, hipStream_t s) {
  constexpr int VEC = sizeof(T) == 4 && sizeof(O) == 4 ? 4 : 8;
  EmbedArgs a = args;
  const int vectors = (a.cols + VEC - 1) / VEC;
  // about four vectors a thread; a block's vectors, below 2048, are divided exactly by the multiplication
  a.rows = vectors >= 4 * kThreads ? 1 : (4 * kThreads + vectors - 1) / vectors;
  if (a.rows > kMaxRows) a.rows = kMaxRows;
  a.magic = (uint32_t)(((1ull << 32) + vectors - 1) / vectors);
  const int64_t blocks = (a.tokens + a.rows - 1) / a.rows;
  const int64_t grid = blocks < kMostBlocks ? blocks : kMostBlocks;
  return a.cols % VEC ? launch_kernel(embed_forward_kernel<T, O, true>, grid, kThreads, a, s)
                      : launch_kernel(embed_forward_kernel<T, O, false>, grid, kThreads, a, s);
}

// Blocks that set a launch's share of the table to zero: up to two for each CU, 64 KiB at least for each.
int64_t zero_blocks(const EmbedGradArgs& a, int launches) {
  if (a.accumulate) return 0;
  const int64_t need = (a.vocab * a.cols * a.table_size / launches + 65535) / 65536;
  return need < 512 ? need : 512;
}

hipError_t run_sort(EmbedGradArgs a, hipStream_t s) {
  if (!a.tokens) {
    const int64_t grid = zero_blocks(a, 1);
    return grid ? launch_kernel(embed_zero_kernel, grid, kSortThreads, a, s) : hipSuccess;
  }
  if (a.tokens <= kOneBlock) return launch_kernel(embed_sort_kernel<kOneBlock / kSortThreads>, 1 + zero_blocks(a, 1), kSortThreads, a, s);
  const int64_t grid = a.blocks + zero_blocks(a, 2 * a.passes);
  hipError_t e = hipSuccess;
  for (a.pass = 0; a.pass < a.passes && e == hipSuccess; ++a.pass) {
    e = launch_kernel(embed_count_kernel, grid, kSortThreads, a, s);
    if (e == hipSuccess) e = launch_kernel(embed_move_kernel, grid, kSortThreads, a, s);
  }
  return e;
}

template <class T, class O, bool PART, int LPR, int EACH, bool STREAM>
hipError_t run_sums(const EmbedGradArgs& a, hipStream_t s) {
  const int64_t chunks = (a.tokens + a.chunk - 1) / a.chunk, slices = (a.cols + LPR * kVec<O> - 1) / (LPR * kVec<O>);
  auto grid = [](int64_t units) { return units < kMostBlocks ? units : kMostBlocks; };
  hipError_t e = launch_kernel(embed_sum_kernel<T, O, PART, LPR, EACH, STREAM>, grid(chunks * slices), kThreads, a, s);
  if (e == hipSuccess && chunks > 1)
    e = launch_kernel(embed_join_kernel<T, O, PART, LPR, EACH>, grid((chunks - 1) * slices), kThreads, a, s);
  return e;
}
template <class T, class O, bool PART, int LPR>
hipError_t pick_sums(const EmbedGradArgs& a, hipStream_t s) {
  if (a.chunk == kThreads / LPR * kFewEach) return run_sums<T, O, PART, LPR, kFewEach, false>(a, s);
  return a.stream && !PART ? run_sums<T, O, PART, LPR, kEmbedEach, !PART>(a, s)
                           : run_sums<T, O, PART, LPR, kEmbedEach, false>(a, s);
}
template <class T, class O, bool PART>
hipError_t pick_lanes(const EmbedGradArgs& a, hipStream_t s) {
  if (a.direct) {
    const int64_t grid = (a.vocab + a.segment - 1) / a.segment;
    switch (a.lanes) {
      case 64: return launch_kernel(embed_direct_kernel<T, O, PART, 64>, grid, kThreads, a, s);
      case 32: return launch_kernel(embed_direct_kernel<T, O, PART, 32>, grid, kThreads, a, s);
      case 16: return launch_kernel(embed_direct_kernel<T, O, PART, 16>, grid, kThreads, a, s);
      default: return launch_kernel(embed_direct_kernel<T, O, PART, 8>, grid, kThreads, a, s);
    }
  }
  hipError_t e = run_sort(a, s);
  if (e != hipSuccess || !a.tokens) return e;
  switch (a.lanes) {
    case 64: return pick_sums<T, O, PART, 64>(a, s);
    case 32: return pick_sums<T, O, PART, 32>(a, s);
    case 16: return pick_sums<T, O, PART, 16>(a, s);
    default: return pick_sums<T, O, PART, 8>(a, s);
  }
}
template <class T, class O>
hipError_t pick_part(const EmbedGradArgs& a, hipStream_t s) {
  return a.cols % kVec<O> ? pick_lanes<T, O, true>(a, s) : pick_lanes<T, O, false>(a, s);
}

}  // namespace

void plan_embed(EmbedGradArgs& a, bool table_bf16, bool out_bf16) {
  a.table_size = table_bf16 ? 2 : 4;
  const int64_t want = (a.tokens + kSortThreads - 1) / kSortThreads;
  const int64_t blocks = want < 1 ? 1 : want < 256 ? want : 256;
  const int64_t each = (a.tokens + blocks - 1) / blocks;
  a.segment = (int32_t)((each + kSortThreads - 1) / kSortThreads * kSortThreads);
  a.blocks = (int32_t)blocks;
  int bits = 1;
  while (bits < 31 && a.vocab >> bits) ++bits;  // ids 0 .. vocab
  a.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  a.digit = (bits + a.passes - 1) / a.passes;
  // the most lanes a row of which no more than an eighth stand idle
  const int vectors = (a.cols + (out_bf16 ? 7 : 3)) / (out_bf16 ? 8 : 4);
  a.lanes = 64;
  while (a.lanes > 8 && (vectors + a.lanes - 1) / a.lanes * a.lanes * 8 > vectors * 9) a.lanes /= 2;
  // fewer entries a group while blocks are few: sums of 32768 x 128 in bf16 8.6 us instead of 11.0 (256 blocks of 8),
  // of 4099 x 1001 in fp32 8.0 instead of 10.5 (516); but with the runs' joining, 42 us instead of 37 for 65536 x 768
  // (over 3000; nothing between 516 and 3000 was measured)
  a.chunk = kThreads / a.lanes * kEmbedEach;
  const int64_t blocks8 = (a.tokens + a.chunk - 1) / a.chunk * ((vectors + a.lanes - 1) / a.lanes);
  if (blocks8 < 1024) a.chunk = kThreads / a.lanes * kFewEach;
  a.direct = a.tokens > 0 && a.tokens <= kDirect;
  if (a.direct) {
    // rows of a block: 64 KiB of the table, but at least 512 blocks
    const int64_t row = (int64_t)a.cols * a.table_size;
    int64_t rows = 65536 / row < a.vocab / 512 ? 65536 / row : a.vocab / 512;
    rows = rows < 1 ? 1 : rows < kDirectRows ? rows : kDirectRows;
    a.segment = (int32_t)rows;
    a.digit = 0;
    while (1 << a.digit < rows) ++a.digit;
  }
  a.stream = a.tokens * a.cols * (out_bf16 ? 2 : 4) >= (int64_t)32 << 20;  // 1024 blocks of 8 at least
}

hipError_t launch_embed_forward(const EmbedArgs& a, bool table_bf16, bool out_bf16, hipStream_t s) {
  if (table_bf16) return out_bf16 ? run_forward<__bf16, __bf16>(a, s) : run_forward<__bf16, float>(a, s);
  return out_bf16 ? run_forward<float, __bf16>(a, s) : run_forward<float, float>(a, s);
}
hipError_t launch_embed_backward(const EmbedGradArgs& a, bool table_bf16, bool out_bf16, hipStream_t s) {
  if (table_bf16) return out_bf16 ? pick_part<__bf16, __bf16>(a, s) : pick_part<__bf16, float>(a, s);
  return out_bf16 ? pick_part<float, __bf16>(a, s) : pick_part<float, float>(a, s);
}

}  // namespace muon
