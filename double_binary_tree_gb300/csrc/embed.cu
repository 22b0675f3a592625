// Embedding lookup with scaling (vr_embedding) and the gradient of the table
// (vr_embedding_grad).
//
//   out_t = scale w[id_t];  dw_v (+)= scale sum_{t: id_t = v} dout_t
//
// The lookup is a gather: a warp takes a piece of a token's row.  16384 tokens of
// 4096 in bf16, of 131072 words, take 32.6 us; the distinct rows once and the
// result are 191 MB, 28.6 us at the copy bandwidth.
//
// The gradient sorts the tokens by word, stably, by the words' digits from the
// lowest up (each pass counts the digits of every warp's run of tokens, adds
// the counts up and moves the tokens), so that a word's rows are summed in
// token order: the same bits on every run, without atomic additions.  Up to 8192
// tokens (16384 where word and token fit 32 bits) can be sorted by one CTA in
// shared memory; else two launches make a pass.  The sorted tokens are cut into
// chunks; a warp sums a slice of the columns of a chunk in fp32 and writes each
// word's row that lies in the chunk as a whole; a word that goes on over the
// chunk's end leaves a partial sum, and a last launch adds the partial sums up in
// chunk order.
//
// Rows of words that do not occur are most of what is written.  They are zeroed
// by the CTAs beside the one that sorts, each of which marks the words of its
// part of the table for itself; after a sort over all SMs, by the launch that
// sums, where a lane looks its word up among the sorted ones.
//
// The same 16384 tokens: 208 us, 180 us of them its 1.2 GB at the copy bandwidth.
// 159 us zero rows (6.0 TB/s to DRAM, the sort beside them), 40 us sum (rows on
// their way through shared memory; 43 us with eight of them in registers, which
// leaves room for half the warps), 11 us join.
//
// Few tokens are summed by one launch without sorting (embed_few_kernel): 777 tokens
// x 1000 added to a table take 6.3 us in a graph, 7.5 us where a few
// words are frequent.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "common.h"
#include "fold.cuh"
#include "gemm_host.h"

namespace vr {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// `N` consecutive elements of a row as one access, or one element.
template <typename T, int N>
struct Pack {
  using Bits = typename Ty<T>::Bits;
  using Raw = typename Select<
      N * sizeof(Bits) == 16, uint4,
      typename Select<N * sizeof(Bits) == 4, uint32_t, Bits>::type>::type;
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[N]) {
    const Bits* b = reinterpret_cast<const Bits*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Ty<T>::widen(b[i]);
  }
  static __device__ __forceinline__ Raw narrow(const float (&x)[N]) {
    Raw r;
    Bits* b = reinterpret_cast<Bits*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = Ty<T>::narrow(x[i]);
    return r;
  }
};

// ---------------------------------------------------------------- lookup
struct LookupArgs {
  const void* weight;
  const long long* ids;
  void* out;
  long long weightStride, outStride, units, ignore;
  int dim, vocab, slices;  // slices of kLookupLoads accesses a lane
  float scale;
  unsigned* status;
};
constexpr int kLookupLoads = 4;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) embed_lookup_kernel(
    const __grid_constant__ LookupArgs a) {
  using Raw = typename Pack<T, N>::Raw;
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const long long step = (long long)gridDim.x * kWarps;
  for (long long u = (long long)blockIdx.x * kWarps + threadIdx.x / 32; u < a.units; u += step) {
    const long long t = u / a.slices;
    const int slice = (int)(u - t * a.slices);
    const long long id = a.ids[t];
    const bool there = id >= 0 && id < a.vocab && id != a.ignore;
    if (!there && id != a.ignore && lane == 0 && slice == 0)
      atomicCAS(a.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
    const T* in = static_cast<const T*>(a.weight) + (there ? id : 0) * a.weightStride;
    T* out = static_cast<T*>(a.out) + t * a.outStride;
    const int c0 = (slice * kLookupLoads * 32 + lane) * N;
    Raw r[kLookupLoads];
#pragma unroll
    for (int i = 0; i < kLookupLoads; ++i) {
      const int c = c0 + i * 32 * N;
      if (there && c < a.dim) r[i] = *reinterpret_cast<const Raw*>(in + c);
    }
#pragma unroll
    for (int i = 0; i < kLookupLoads; ++i) {
      const int c = c0 + i * 32 * N;
      if (c >= a.dim) break;
      float x[N];
      if (there) Pack<T, N>::widen(r[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = there ? x[j] * a.scale : 0.0f;
      *reinterpret_cast<Raw*>(out + c) = Pack<T, N>::narrow(x);
    }
  }
}

// ------------------------------------------------------------------ sorting
// An item is a word and, in the lowest tokenBits bits, the token that has it; a
// token that does not count has the word `vocab`, behind all others.
using Item = unsigned long long;
constexpr int kItemBits = 32;  // tokenBits of the sorted items
__device__ __forceinline__ unsigned word_of(Item x) { return (unsigned)(x >> kItemBits); }
__device__ __forceinline__ unsigned token_of(Item x) { return (unsigned)x; }

constexpr int kMaxBits = 9, kDigits = 1 << kMaxBits;  // of one pass
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr size_t kSmallBytes = 64 << 10;  // of items that one CTA sorts

struct SortArgs {
  const long long* ids;
  long long ignore;
  int tokens, vocab;
  int passes, bits;   // of each pass
  int tokenBits;
  int shift;          // this pass's lowest bit (large)
  int ctas, run;      // large: CTAs, and tokens of each
  const Item* in;     // large: null in the first pass
  Item* out;
  int* counts;        // large: [ctas][kDigits]
  unsigned* status;
  // the table, whose rows of words that do not occur are zeroed (not large)
  char* table;
  long long rowBytes;
  int access;
};

__device__ __forceinline__ bool counts_as_word(const SortArgs& a, long long id) {
  return id >= 0 && id < a.vocab && id != a.ignore;
}
template <typename K>
__device__ __forceinline__ K item_of(const SortArgs& a, int t) {
  const long long id = a.ids[t];
  const bool there = counts_as_word(a, id);
  if (!there && id != a.ignore) atomicCAS(a.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
  return (K)(unsigned)(there ? (int)id : a.vocab) << a.tokenBits | (unsigned)t;
}

// Counts the digits (from bit `shift` of an item) of a warp's run [lo, hi) of
// items into its row of counters, or (MOVE) sends each to the place that its
// digit's counter gives.  Equal digits of 32 items take consecutive places, so
// the order is kept.
template <typename K, bool MOVE, class Get, class Put>
__device__ __forceinline__ void digits_of_run(unsigned* row, int lo, int hi, int shift,
                                              unsigned mask, Get get, Put put) {
  const int lane = threadIdx.x % 32;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const bool live = i0 + lane < hi;
    const K x = live ? get(i0 + lane) : 0;
    const unsigned d = (unsigned)(x >> shift) & mask;
    // the live lanes with the same digit, bit by bit (__match_any_sync: 43 us instead
    // of 28 for 8192 tokens)
    unsigned same = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int b = 0; b < kMaxBits; ++b) {
      const unsigned set = __ballot_sync(0xffffffffu, d >> b & 1);
      same &= d >> b & 1 ? set : ~set;
    }
    const int first = __ffs(same) - 1;
    unsigned base = 0;
    if (live && lane == first) {
      base = row[d];
      row[d] = base + __popc(same);
    }
    if (MOVE) {
      base = __shfl_sync(0xffffffffu, base, first);
      if (live) put(base + __popc(same & ((1u << lane) - 1)), x);
    }
    __syncwarp();
  }
}

// The counters of the warps made into places: of each digit, the items of lower
// digits and of its earlier warps before it.  `base(d, n)` adds what lies
// before this CTA's n items of the digit, as a whole sum over lower digits
// (the CTAs' totals) and earlier CTAs.
template <class Base>
__device__ __forceinline__ void places(unsigned (*rows)[kDigits], int warps, unsigned* sScan,
                                       Base base) {
  const int d = threadIdx.x;
  unsigned total = 0;
  if (d < kDigits) {
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const unsigned n = rows[w][d];
      rows[w][d] = total;
      total += n;
    }
  }
  // exclusive sum over the digits of all items that have them
  unsigned all = total, before = 0;
  if (d < kDigits) base(d, &all, &before);
  unsigned sum = all;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const unsigned up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) sScan[warp] = d < kDigits ? sum : 0;
  __syncthreads();
  if (d < kDigits) {
    unsigned start = sum - all + before;
    for (int w = 0; w < warp; ++w) start += sScan[w];
#pragma unroll 8
    for (int w = 0; w < warps; ++w) rows[w][d] += start;
  }
  __syncthreads();
}

__device__ __forceinline__ void clear(unsigned (*rows)[kDigits], int warps) {
  unsigned* p = &rows[0][0];
  for (int i = threadIdx.x; i < warps * kDigits; i += kSortThreads) p[i] = 0;
  __syncthreads();
}

// The rows of a part of the table whose words do not occur, zeroed by one CTA.
constexpr int kMarked = 8192;  // words that are marked at a time
__device__ __forceinline__ void zero_row(char* row, long long bytes, int access) {
  const int lane = threadIdx.x % 32;
  if (access == 16) {
#pragma unroll 4
    for (long long i = lane * 16; i < bytes; i += 32 * 16)
      *reinterpret_cast<uint4*>(row + i) = make_uint4(0, 0, 0, 0);
  } else if (access == 4) {
#pragma unroll 4
    for (long long i = lane * 4; i < bytes; i += 32 * 4) *reinterpret_cast<unsigned*>(row + i) = 0;
  } else {
#pragma unroll 4
    for (long long i = lane * 2; i < bytes; i += 32 * 2)
      *reinterpret_cast<unsigned short*>(row + i) = 0;
  }
}
template <int THREADS>
__device__ __forceinline__ void zero_rows(const SortArgs& a, unsigned* marks, int part, int parts) {
  const int lo = (int)((long long)a.vocab * part / parts);
  const int hi = (int)((long long)a.vocab * (part + 1) / parts);
  for (int v0 = lo; v0 < hi; v0 += kMarked) {
    const int n = min(kMarked, hi - v0);
    for (int i = threadIdx.x; i < kMarked / 32; i += THREADS) marks[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int t = threadIdx.x; t < a.tokens; t += THREADS) {
      const long long id = a.ids[t];
      if (id >= v0 && id < v0 + n && id != a.ignore)
        atomicOr(&marks[(id - v0) / 32], 1u << ((id - v0) % 32));
    }
    __syncthreads();
    for (int i = threadIdx.x / 32; i < n; i += THREADS / 32)
      if (!(marks[i / 32] >> (i % 32) & 1))
        zero_row(a.table + (long long)(v0 + i) * a.rowBytes, a.rowBytes, a.access);
    __syncthreads();
  }
}

// CTA 0 sorts the tokens in shared memory, the others zero rows.
constexpr size_t kSmallSmem = 2 * kSmallBytes + kSortWarps * kDigits * 4;
template <typename K>
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(
    const __grid_constant__ SortArgs a) {
  extern __shared__ Item smem[];
  __shared__ unsigned sScan[kSortWarps];
  K *from = reinterpret_cast<K*>(smem), *to = from + kSmallBytes / sizeof(K);
  unsigned(*rows)[kDigits] =
      reinterpret_cast<unsigned(*)[kDigits]>(reinterpret_cast<char*>(smem) + 2 * kSmallBytes);
  pdl_launch();
  pdl_wait();
  if (blockIdx.x > 0) {
    zero_rows<kSortThreads>(a, &rows[0][0], (int)blockIdx.x - 1, (int)gridDim.x - 1);
    return;
  }
  for (int t = threadIdx.x; t < a.tokens; t += kSortThreads) from[t] = item_of<K>(a, t);
  const int warp = threadIdx.x / 32;
  // (128 tokens a warp at least: every warp has counters to be added up)
  const int run = max((a.tokens + kSortWarps * 32 - 1) / (kSortWarps * 32), 4) * 32;
  const int warps = (a.tokens + run - 1) / run;
  const int lo = min(warp * run, a.tokens), hi = min(lo + run, a.tokens);
  const unsigned mask = (1u << a.bits) - 1;
  for (int p = 0; p < a.passes; ++p) {
    clear(rows, warps);
    const int shift = a.tokenBits + p * a.bits;
    auto get = [&](int i) { return from[i]; };
    digits_of_run<K, false>(rows[warp], lo, hi, shift, mask, get, [](unsigned, K) {});
    __syncthreads();
    places(rows, warps, sScan, [](int, unsigned*, unsigned*) {});
    if (p + 1 == a.passes) {
      digits_of_run<K, true>(rows[warp], lo, hi, shift, mask, get, [&](unsigned at, K x) {
        a.out[at] = (Item)(x >> a.tokenBits) << kItemBits | (unsigned)(x & ((K)1 << a.tokenBits) - 1);
      });
    } else {
      digits_of_run<K, true>(rows[warp], lo, hi, shift, mask, get,
                             [&](unsigned at, K x) { to[at] = x; });
    }
    __syncthreads();
    K* t = from;
    from = to;
    to = t;
  }
}

// One pass over many tokens: a launch that counts every CTA's digits, one that
// moves the items.
template <bool MOVE>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(
    const __grid_constant__ SortArgs a) {
  extern __shared__ Item smem[];
  __shared__ unsigned sScan[kSortWarps];
  unsigned(*rows)[kDigits] = reinterpret_cast<unsigned(*)[kDigits]>(smem);
  pdl_launch();
  clear(rows, kSortWarps);
  pdl_wait();
  const int warp = threadIdx.x / 32;
  const int begin = (int)min((long long)blockIdx.x * a.run, (long long)a.tokens);
  const int n = min(a.run, a.tokens - begin);
  const int run = (n + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;
  const int lo = begin + min(warp * run, n), hi = min(lo + run, begin + n);
  const unsigned mask = (1u << a.bits) - 1;
  auto get = [&](int i) { return a.in ? a.in[i] : item_of<Item>(a, i); };
  digits_of_run<Item, false>(rows[warp], lo, hi, a.shift, mask, get, [](unsigned, Item) {});
  __syncthreads();
  if (!MOVE) {
    if (threadIdx.x < kDigits) {
      unsigned total = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) total += rows[w][threadIdx.x];
      a.counts[blockIdx.x * kDigits + threadIdx.x] = (int)total;
    }
    return;
  }
  places(rows, kSortWarps, sScan, [&](int d, unsigned* all, unsigned* before) {
    unsigned sum = 0, mine = 0;
#pragma unroll 16
    for (int c = 0; c < a.ctas; ++c) {
      const unsigned k = (unsigned)a.counts[c * kDigits + d];
      sum += k;
      mine += c < (int)blockIdx.x ? k : 0;
    }
    *all = sum;
    *before = mine;
  });
  digits_of_run<Item, true>(rows[warp], lo, hi, a.shift, mask, get,
                            [&](unsigned at, Item x) { a.out[at] = x; });
}

// --------------------------------------------------------------------- sums
struct SumArgs {
  const void* dout;
  void* dweight;
  const Item* items;
  float* parts;      // [chunks][2][dim]: of the word that a chunk begins and ends with
  long long stride;  // of dout
  long long fillUnits, units;
  int tokens, dim, vocab, add;
  int chunk, chunks, slices;
  float scale;
};
constexpr int kFillRows = 8;  // rows of the table that a warp zeroes at a time

// A slice of a row: REP accesses of N elements a lane.
template <typename T, int N, int REP>
struct Slice {
  using Raw = typename Pack<T, N>::Raw;
  static constexpr int kCols = 32 * N * REP;
  // rows of a warp on their way, where they are whole 16-byte units
  static constexpr int kRing = sizeof(Raw) == 16 ? 8 / REP : 0;
  static __device__ __forceinline__ int col(int slice, int i) {
    return slice * kCols + (i * 32 + (int)threadIdx.x % 32) * N;
  }
  // the final row of a word: scaled, added to what is there, rounded once
  static __device__ __forceinline__ T* row(const SumArgs& a, unsigned word) {
    return static_cast<T*>(a.dweight) + (long long)word * a.dim;
  }
  static __device__ __forceinline__ void load_old(const SumArgs& a, unsigned word, int slice,
                                                  Raw (&old)[REP]) {
    if (!a.add) return;
#pragma unroll
    for (int i = 0; i < REP; ++i)
      if (col(slice, i) < a.dim) old[i] = *reinterpret_cast<const Raw*>(row(a, word) + col(slice, i));
  }
  static __device__ __forceinline__ void write(const SumArgs& a, unsigned word, int slice,
                                               const float (&sum)[REP][N], const Raw (&old)[REP]) {
#pragma unroll
    for (int i = 0; i < REP; ++i) {
      if (col(slice, i) >= a.dim) break;
      float x[N];
      if (a.add) Pack<T, N>::widen(old[i], x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = fmaf(sum[i][j], a.scale, a.add ? x[j] : 0.0f);
      *reinterpret_cast<Raw*>(row(a, word) + col(slice, i)) = Pack<T, N>::narrow(x);
    }
  }
  static __device__ __forceinline__ void write(const SumArgs& a, unsigned word, int slice,
                                               const float (&sum)[REP][N]) {
    Raw old[REP];
    load_old(a, word, slice, old);
    write(a, word, slice, sum, old);
  }
  static __device__ __forceinline__ float* part(const SumArgs& a, int chunk, int end) {
    return a.parts + ((long long)chunk * 2 + end) * a.dim;
  }
  static __device__ __forceinline__ void store_part(const SumArgs& a, int chunk, int end,
                                                    int slice, const float (&sum)[REP][N]) {
    float* p = part(a, chunk, end);
#pragma unroll
    for (int i = 0; i < REP; ++i) {
      if (col(slice, i) >= a.dim) break;
#pragma unroll
      for (int j = 0; j < N; j += kWide)
        *reinterpret_cast<Wide*>(p + col(slice, i) + j) =
            *reinterpret_cast<const Wide*>(&sum[i][j]);
    }
  }
  // (dim is a multiple of N, the partial sums begin at 16 bytes)
  using Wide = typename Select<N % 4 == 0, float4, typename Select<N == 2, float2, float>::type>::type;
  static constexpr int kWide = N % 4 == 0 ? 4 : N;
  // the partial sums of chunks `from` to `to` that begin with the word, in order,
  // up to eight of them on their way
  static __device__ __forceinline__ void add_parts(const SumArgs& a, int from, int to, int slice,
                                                   float (&sum)[REP][N]) {
    constexpr int kUnits = N / kWide, kAtOnce = 8;
    const long long step = 2LL * a.dim;
#pragma unroll
    for (int i = 0; i < REP; ++i) {
      if (col(slice, i) >= a.dim) break;
      const float* p = part(a, from, 0) + col(slice, i);
      for (int k = from; k <= to; k += kAtOnce) {
        Wide w[kAtOnce][kUnits];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
          for (int j = 0; j < kUnits; ++j)
            if (k + q <= to) w[q][j] = *reinterpret_cast<const Wide*>(p + q * step + j * kWide);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
          if (k + q <= to) {
#pragma unroll
            for (int j = 0; j < N; ++j)
              sum[i][j] += reinterpret_cast<const float*>(&w[q][j / kWide])[j % kWide];
          }
        p += kAtOnce * step;
      }
    }
  }
  static __device__ __forceinline__ void load_part(const SumArgs& a, int chunk, int end, int slice,
                                                   float (&sum)[REP][N]) {
    const float* p = part(a, chunk, end);
#pragma unroll
    for (int i = 0; i < REP; ++i) {
      if (col(slice, i) >= a.dim) break;
#pragma unroll
      for (int j = 0; j < N; j += kWide)
        *reinterpret_cast<Wide*>(&sum[i][j]) =
            *reinterpret_cast<const Wide*>(p + col(slice, i) + j);
    }
  }
};

// Whether `word` occurs among the sorted items.
__device__ __forceinline__ bool occurs(const SumArgs& a, unsigned word) {
  int lo = 0, hi = a.tokens;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (word_of(a.items[mid]) < word) lo = mid + 1;
    else hi = mid;
  }
  return lo < a.tokens && word_of(a.items[lo]) == word;
}

template <typename T, int N, int REP>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const __grid_constant__ SumArgs a) {
  using S = Slice<T, N, REP>;
  using Raw = typename S::Raw;
  __shared__ uint4 rings[S::kRing ? kWarps : 1][S::kRing ? S::kRing : 1][REP][32];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x % 32;
  const long long step = (long long)gridDim.x * kWarps;
  for (long long u = (long long)blockIdx.x * kWarps + threadIdx.x / 32; u < a.units; u += step) {
    if (u < a.fillUnits) {  // rows of words that do not occur
      const long long v = u * kFillRows + lane;
      const bool zero = lane < kFillRows && v < a.vocab && !occurs(a, (unsigned)v);
      unsigned rows = __ballot_sync(0xffffffffu, zero);
      Raw none = {};
      while (rows) {
        T* out = static_cast<T*>(a.dweight) + (u * kFillRows + __ffs(rows) - 1) * a.dim;
        rows &= rows - 1;
#pragma unroll 4
        for (int c = lane * N; c < a.dim; c += 32 * N) *reinterpret_cast<Raw*>(out + c) = none;
      }
      continue;
    }
    const long long at = u - a.fillUnits;
    const int chunk = (int)(at / a.slices), slice = (int)(at - (long long)chunk * a.slices);
    const int lo = chunk * a.chunk, hi = min(lo + a.chunk, a.tokens);
    unsigned word = word_of(a.items[lo]);
    if (word >= (unsigned)a.vocab) continue;  // tokens that do not count are last
    bool head = lo > 0 && word_of(a.items[lo - 1]) == word;  // goes on from the last chunk
    float sum[REP][N] = {};
    unsigned before = word;  // of the item before the next 32
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const Item mine = i0 + lane < hi ? a.items[i0 + lane] : (Item)~0u << kItemBits;
      const unsigned w = word_of(mine);
      const unsigned up = __shfl_up_sync(0xffffffffu, w, 1);
      const unsigned starts = __ballot_sync(0xffffffffu, w != (lane ? up : before));
      const int n = __popc(__ballot_sync(0xffffffffu, w < (unsigned)a.vocab));  // those first
      before = __shfl_sync(0xffffffffu, w, 31);
      auto start = [&](int j) {  // item j begins a word: the last one is written
        if (head) S::store_part(a, chunk, 0, slice, sum);
        else S::write(a, word, slice, sum);
        head = false;
        word = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
        for (int i = 0; i < REP; ++i)
#pragma unroll
          for (int k = 0; k < N; ++k) sum[i][k] = 0.0f;
      };
      auto add = [&](const Raw(&r)[REP]) {
#pragma unroll
        for (int i = 0; i < REP; ++i) {
          float x[N];
          Pack<T, N>::widen(r[i], x);
#pragma unroll
          for (int k = 0; k < N; ++k) sum[i][k] += x[k];
        }
      };
      auto row_of = [&](int j) {
        const unsigned token = __shfl_sync(0xffffffffu, token_of(mine), j);
        return static_cast<const T*>(a.dout) + (long long)token * a.stride;
      };
      if constexpr (S::kRing > 0) {
        // a lane's 16 bytes of the next rows on their way through shared memory
        uint4(*ring)[REP][32] = rings[threadIdx.x / 32];
        auto fetch = [&](int j) {
          if (j < n) {
            const T* in = row_of(j);
#pragma unroll
            for (int i = 0; i < REP; ++i)
              if (S::col(slice, i) < a.dim)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_addr(&ring[j % S::kRing][i][lane])),
                             "l"(in + S::col(slice, i))
                             : "memory");
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int j = 0; j < S::kRing - 1; ++j) fetch(j);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          fetch(j + S::kRing - 1);  // (into the place that was read in the last round)
          asm volatile("cp.async.wait_group %0;" ::"n"(S::kRing - 1) : "memory");
          if (starts >> j & 1) start(j);
          Raw r[REP];
#pragma unroll
          for (int i = 0; i < REP; ++i)
            r[i] = *reinterpret_cast<const Raw*>(&ring[j % S::kRing][i][lane]);
          add(r);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      } else {
        constexpr int kAhead = 8 / REP;
        for (int j0 = 0; j0 < n; j0 += kAhead) {
          Raw r[kAhead][REP];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= n) break;
            const T* in = row_of(j0 + k);
#pragma unroll
            for (int i = 0; i < REP; ++i)
              if (S::col(slice, i) < a.dim)
                r[k][i] = *reinterpret_cast<const Raw*>(in + S::col(slice, i));
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (j0 + k >= n) break;
            if (starts >> (j0 + k) & 1) start(j0 + k);
            add(r[k]);
          }
        }
      }
    }
    const bool tail = hi < a.tokens && word_of(a.items[hi]) == word;
    if (head) S::store_part(a, chunk, 0, slice, sum);
    else if (tail) S::store_part(a, chunk, 1, slice, sum);
    else S::write(a, word, slice, sum);
  }
}

// The words that go on over a chunk's end: a warp adds the partial sums of a
// slice of one up, in chunk order.
template <typename T, int N, int REP>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ SumArgs a) {
  using S = Slice<T, N, REP>;
  pdl_launch();
  pdl_wait();
  const long long step = (long long)gridDim.x * kWarps;
  const long long units = (long long)(a.chunks - 1) * a.slices;
  const int lane = threadIdx.x % 32;
  for (long long u = (long long)blockIdx.x * kWarps + threadIdx.x / 32; u < units; u += step) {
    const int chunk = (int)(u / a.slices), slice = (int)(u - (long long)chunk * a.slices);
    const int lo = chunk * a.chunk, hi = lo + a.chunk;  // not the last chunk
    const unsigned word = word_of(a.items[hi - 1]);
    if (word >= (unsigned)a.vocab || word_of(a.items[hi]) != word) continue;
    // it begins in this chunk
    if (lo > 0 && word_of(a.items[lo]) == word && word_of(a.items[lo - 1]) == word) continue;
    // the chunks that it goes on into: every lane looks at the end of one
    int last = chunk + 1;
    for (;; last += 32) {
      const long long end = (long long)(last + lane + 1) * a.chunk;
      const bool on = end < a.tokens && word_of(a.items[end]) == word;
      const unsigned stops = ~__ballot_sync(0xffffffffu, on);
      if (stops) {
        last += __ffs(stops) - 1;
        break;
      }
    }
    float sum[REP][N] = {};
    S::load_part(a, chunk, 1, slice, sum);
    S::add_parts(a, chunk + 1, last, slice, sum);
    S::write(a, word, slice, sum);
  }
}

// ---------------------------------------------------------------- few tokens
// No sorting: a warp takes a slice of a token's columns, compares the token's word
// with all others, and where the token is the first that has it, adds up the
// rows of those that do, in token order.  A word that more than kHot tokens have
// is left to all warps of the CTA, an eighth of the tokens each, whose sums are
// added in order.  The first CTAs zero rows.
//
// One launch instead of three, and no partial sums in memory.  Comparisons grow
// with the tokens' square: 1024 tokens x 4096 columns added to a table take 17 us
// (sorted: 16; half of them one word: 22 and 27), x 8192 29 us (20), which is
// sorted; 777 x 1000 6.3 us (14.7), all of one word 16 us (30), 64 x 1024 2.5 us
// (10).  (With several slices a warp, to compare once for them, a frequent word's
// are summed by few CTAs: 64 us instead of 21.)
constexpr size_t kFewTokens = 1024, kFewSlices = 16384;  // slices of 256 columns of all tokens
constexpr int kHot = 32;
struct FewArgs {
  SortArgs sort;
  SumArgs sum;
  int zeroing;  // CTAs that zero rows
};

template <typename T, int N, int REP>
__global__ void __launch_bounds__(kThreads) embed_few_kernel(const __grid_constant__ FewArgs f) {
  using S = Slice<T, N, REP>;
  using Raw = typename S::Raw;
  __shared__ unsigned words[kFewTokens];  // of the tokens; of one that does not count: vocab
  __shared__ alignas(16) float parts[kWarps][S::kCols];
  __shared__ long long hot[kWarps];
  static_assert(sizeof(parts) >= kMarked / 8, "the marks of the words");
  const SumArgs& a = f.sum;
  pdl_launch();
  pdl_wait();
  if ((int)blockIdx.x < f.zeroing) {
    zero_rows<kThreads>(f.sort, reinterpret_cast<unsigned*>(&parts[0][0]), (int)blockIdx.x,
                        f.zeroing);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = (int)blockIdx.x - f.zeroing, ctas = (int)gridDim.x - f.zeroing;
  const int blocks = (a.tokens + 31) / 32;  // of 32 tokens: at most one for each lane
  for (int t = threadIdx.x; t < blocks * 32; t += kThreads) {
    const long long id = t < a.tokens ? f.sort.ids[t] : f.sort.ignore;
    const bool there = counts_as_word(f.sort, id);
    if (!there && id != f.sort.ignore && cta == 0)
      atomicCAS(f.sort.status, 0u, (unsigned)VR_ERR_INVALID_ARGUMENT);
    words[t] = there ? (unsigned)id : (unsigned)a.vocab;
  }
  __syncthreads();
  // the tokens that have the word: lane b has those of block b, in [from, to)
  auto tokens_of = [&](unsigned word, int from, int to) {
    unsigned mine = 0;
#pragma unroll 8
    for (int b = from; b < to; ++b) {
      const unsigned same = __ballot_sync(0xffffffffu, words[b * 32 + lane] == word);
      if (lane == b) mine = same;
    }
    return mine;
  };
  // the sum of their rows
  auto add_rows = [&](unsigned mine, int slice, float(&sum)[REP][N]) {
    constexpr int kRows = 8 / REP;  // on their way
    unsigned left = __ballot_sync(0xffffffffu, mine != 0), bits = 0;
    int block = 0;
    for (bool more = left != 0; more;) {
      Raw r[kRows][REP];
      int n = 0;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (!bits) {
          if (!left) break;
          block = __ffs(left) - 1;
          left &= left - 1;
          bits = __shfl_sync(0xffffffffu, mine, block);
        }
        const int token = block * 32 + __ffs(bits) - 1;
        bits &= bits - 1;
        const T* in = static_cast<const T*>(a.dout) + (long long)token * a.stride;
#pragma unroll
        for (int i = 0; i < REP; ++i)
          if (S::col(slice, i) < a.dim) r[k][i] = *reinterpret_cast<const Raw*>(in + S::col(slice, i));
        n = k + 1;
      }
      more = bits || left;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < REP; ++i) {
          float x[N];
          Pack<T, N>::widen(r[k][i], x);
#pragma unroll
          for (int j = 0; j < N; ++j) sum[i][j] += x[j];
        }
      }
    }
  };
  const long long step = (long long)ctas * kWarps;
  for (long long u0 = 0; u0 < a.units; u0 += step) {
    // (the slices of a token in CTAs beside each other)
    const long long u = u0 + (long long)warp * ctas + cta;
    bool whole = false;
    if (u < a.units) {
      const int t = (int)(u / a.slices), slice = (int)(u - (long long)t * a.slices);
      const unsigned word = words[t];
      if (word < (unsigned)a.vocab) {
        const unsigned mine = tokens_of(word, 0, blocks);
        const int count = (int)__reduce_add_sync(0xffffffffu, (unsigned)__popc(mine));
        // the first token that has it: in the first block that has one
        const bool earlier = lane < t / 32 ? mine != 0
                                           : lane == t / 32 && (mine & ((1u << (t % 32)) - 1)) != 0;
        const bool first = !__any_sync(0xffffffffu, earlier);
        whole = first && count > kHot;
        if (first && !whole) {
          Raw old[REP];
          float sum[REP][N] = {};
          S::load_old(a, word, slice, old);
          add_rows(mine, slice, sum);
          S::write(a, word, slice, sum, old);
        }
      }
    }
    if (lane == 0) hot[warp] = whole ? u : -1;
    if (!__syncthreads_or(whole)) continue;  // (nobody reads `hot`)
    for (int w = 0; w < kWarps; ++w) {
      const long long h = hot[w];
      if (h < 0) continue;
      const int t = (int)(h / a.slices), slice = (int)(h - (long long)t * a.slices);
      const unsigned word = words[t];
      float sum[REP][N] = {};
      add_rows(tokens_of(word, blocks * warp / kWarps, blocks * (warp + 1) / kWarps), slice, sum);
#pragma unroll
      for (int i = 0; i < REP; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) parts[warp][(i * N + j) * 32 + lane] = sum[i][j];
      __syncthreads();
      if (warp == w) {
#pragma unroll
        for (int i = 0; i < REP; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            float x = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) x += parts[k][(i * N + j) * 32 + lane];
            sum[i][j] = x;
          }
        S::write(a, word, slice, sum);
      }
      __syncthreads();
    }
    __syncthreads();  // (all have read `hot`)
  }
}

// ------------------------------------------------------------- host side
constexpr size_t kMostTokens = (size_t)1 << 30, kMostVocab = (size_t)1 << 30,
                 kMostDim = (size_t)1 << 24, kMostStride = (size_t)1 << 31;
constexpr int kMostCtas = 152;
constexpr size_t kSortRun = 2048;  // the fewest tokens that a CTA of a large sort takes

int bits_of(size_t n) {
  int b = 1;
  while (n >> b) ++b;
  return b;
}

// Items of a chunk: as few as four where that makes no more warps than are
// resident at once (a warp writes the rows of its words one after the other: 777
// tokens x 1000 columns, sorted, in 7 us instead of 27 with 32).
size_t chunk_of(size_t tokens, size_t dim) {
  const size_t slices = (dim + 255) / 256;
  size_t c = 4;
  while (tokens / c * slices > 8192) c *= 2;
  return c;
}

struct EmbedPlan {
  bool few;            // no sorting
  bool small, narrow;  // one CTA may sort; with items of 32 bits
  int passes, bits, tokenBits;
  size_t run, ctas, chunk, chunks;
  size_t items, other, counts, parts, bytes;  // offsets into the workspace
};
bool make_plan(size_t tokens, size_t dim, size_t vocab, int dtype, EmbedPlan* p) {
  if (!op_elem_size(dtype) || tokens > kMostTokens || dim < 1 || dim > kMostDim || vocab < 1 ||
      vocab > kMostVocab)
    return false;
  *p = EmbedPlan{};
  // (a workspace of the same size either way: which way is no caller's concern)
  p->few = tokens <= kFewTokens && tokens * ((dim + 255) / 256) <= kFewSlices;
  const int words = bits_of(vocab);  // of the words 0 .. vocab
  p->passes = (words + kMaxBits - 1) / kMaxBits;
  p->bits = (words + p->passes - 1) / p->passes;
  p->tokenBits = bits_of(tokens ? tokens - 1 : 0);
  p->narrow = tokens <= kSmallBytes / 4 && words + p->tokenBits <= 32;
  p->small = p->narrow || tokens <= kSmallBytes / sizeof(Item);
  p->run = std::max(kSortRun, (tokens + kMostCtas - 1) / kMostCtas);
  p->ctas = (tokens + p->run - 1) / p->run;
  p->chunk = chunk_of(tokens, dim);
  p->chunks = (tokens + p->chunk - 1) / p->chunk;
  size_t at = 0;
  auto take = [&at](size_t n) {
    const size_t here = at;
    at += op_round(n);
    return here;
  };
  p->items = take(tokens * sizeof(Item));
  p->other = take(tokens * sizeof(Item));
  p->counts = take(p->ctas * kDigits * 4);
  p->parts = take(p->chunks * 2 * dim * 4);
  p->bytes = at + kOpSlack;
  return true;
}

// Which sort.  One CTA's takes 28 us for 8192 tokens, 47 us for 16384 (two passes), the
// other way 21 and 23 us, but nothing is zeroed meanwhile.
// So it goes by whether the difference is more than zeroing `bytes` at 6 TB/s takes.
// Whole gradients in a graph, one CTA / all SMs (us, bf16):
//                                  2048     4096     6000     8192    12000    16384 tokens
//   x 1024, added, 5 % one word  17 / 24  26 / 27  34 / 31  43 / 36  53 / 35  67 / 42
//   x 4096, added                22 / 29  34 / 35  44 / 40  71 / 62  91 / 72  127 / 98
//   x 1024 of 32000, whole       17 / 32  24 / 33  29 / 34  37 / 36  48 / 38  62 / 41
//   x 1024 of 131072, whole      50 / 64  52 / 67  55 / 71  59 / 78  59 / 78  69 / 82
// The rule takes the quicker one everywhere but at 8192 of 32000 (37).
void choose_sort(EmbedPlan* p, size_t tokens, double bytes) {
  const double longer = 1.05e-3 * p->passes * ((double)tokens - 4900.0);  // us
  p->small = p->small && longer <= bytes / 6e6;
  p->narrow = p->narrow && p->small;
  if (!p->narrow) p->tokenBits = kItemBits;
}

// The widest access that all rows allow: 16 bytes, 4 or one element.
int access_bytes(uintptr_t bits, size_t elem) {
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : (int)elem;
}

template <typename T, int N, int REP>
vr_result_t launch_sums(const EmbedPlan& p, const OpDevice& dev, SumArgs& a, void* stream) {
  a.slices = (a.dim + Slice<T, N, REP>::kCols - 1) / Slice<T, N, REP>::kCols;
  a.fillUnits = a.add || p.small ? 0 : ((long long)a.vocab + kFillRows - 1) / kFillRows;
  a.units = a.fillUnits + (long long)p.chunks * a.slices;
  void* args[] = {&a};
  auto grid = [&](long long units) {
    return dim3((unsigned)std::min<long long>((units + kWarps - 1) / kWarps, dev.sms * 8LL));
  };
  vr_result_t e = op_launch((const void*)embed_sum_kernel<T, N, REP>, grid(a.units),
                            dim3(kThreads), args, 0, stream);
  if (e != VR_SUCCESS || p.chunks < 2) return e;
  return op_launch((const void*)embed_join_kernel<T, N, REP>,
                   grid((long long)(p.chunks - 1) * a.slices), dim3(kThreads), args, 0, stream);
}

template <typename T, int N, int REP>
vr_result_t launch_few(const SortArgs& s, const OpDevice& dev, SumArgs& a, void* stream) {
  FewArgs f = {s, a, 0};
  f.sum.slices = (a.dim + Slice<T, N, REP>::kCols - 1) / Slice<T, N, REP>::kCols;
  f.sum.units = (long long)a.tokens * f.sum.slices;
  if (!a.add) f.zeroing = std::min(dev.sms * 4, a.vocab);
  const long long ctas = std::min<long long>((f.sum.units + kWarps - 1) / kWarps, dev.sms * 4LL);
  void* args[] = {&f};
  return op_launch((const void*)embed_few_kernel<T, N, REP>, dim3((unsigned)(f.zeroing + ctas)),
                   dim3(kThreads), args, 0, stream);
}

template <typename T>
vr_result_t sums(const EmbedPlan& p, const SortArgs& s, const OpDevice& dev, SumArgs& a, int access,
                 void* stream) {
  auto go = [&](auto n, auto rep) {
    constexpr int N = decltype(n)::value, REP = decltype(rep)::value;
    return p.few ? launch_few<T, N, REP>(s, dev, a, stream)
                 : launch_sums<T, N, REP>(p, dev, a, stream);
  };
  using std::integral_constant;
  constexpr int kElem = (int)sizeof(T), kWide = 16 / kElem;
  if (access == 16) return go(integral_constant<int, kWide>(), integral_constant<int, 8 / kWide>());
  if constexpr (kElem == 2)
    if (access == 4) return go(integral_constant<int, 2>(), integral_constant<int, 4>());
  return go(integral_constant<int, 1>(), integral_constant<int, 4>());
}

template <typename T>
const void* lookup(int access, int* n) {
  constexpr int kElem = (int)sizeof(T);
  *n = access / kElem;
  if (access == 16) return (const void*)embed_lookup_kernel<T, 16 / kElem>;
  if constexpr (kElem == 2)
    if (access == 4) return (const void*)embed_lookup_kernel<T, 2>;
  return (const void*)embed_lookup_kernel<T, 1>;
}

}  // namespace
}  // namespace vr

using namespace vr;

extern "C" {

vr_result_t vr_embedding(const void* weight, size_t weightStride, const long long* ids,
                         size_t tokens, size_t dim, size_t vocab, vr_dtype_t dtype,
                         long long ignoreIndex, float scale, void* out, size_t outStride,
                         void* stream) {
  const size_t E = op_elem_size(dtype);
  EmbedPlan p;
  if (!make_plan(tokens, dim, vocab, dtype, &p) || weightStride < dim || outStride < dim ||
      weightStride > kMostStride || outStride > kMostStride || !weight ||
      (tokens && (!ids || !out)) || ((uintptr_t)ids & 7) ||
      ((uintptr_t)weight | (uintptr_t)out) % E)
    return VR_ERR_INVALID_ARGUMENT;
  // (an output listed before the inputs may be none of them)
  const OpBuffer buf[3] = {{out, tokens, dim * E, outStride * E, true},
                           {weight, vocab, dim * E, weightStride * E, false},
                           {ids, 1, tokens * 8, tokens * 8, false}};
  if (!op_buffers_ok(buf, 3)) return VR_ERR_INVALID_ARGUMENT;
  if (!tokens) return VR_SUCCESS;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, 3, dev.device)) != VR_SUCCESS) return e;
  const int access = access_bytes((uintptr_t)weight | (uintptr_t)out | (uintptr_t)(dim * E) |
                                      (uintptr_t)(weightStride * E) | (uintptr_t)(outStride * E),
                                  E);
  int n = 0;
  const void* fn = dtype == VR_FLOAT32   ? lookup<float>(access, &n)
                   : dtype == VR_FLOAT16 ? lookup<__half>(access, &n)
                                         : lookup<__nv_bfloat16>(access, &n);
  LookupArgs a = {};
  a.weight = weight;
  a.ids = ids;
  a.out = out;
  a.weightStride = (long long)weightStride;
  a.outStride = (long long)outStride;
  a.ignore = ignoreIndex;
  a.dim = (int)dim;
  a.vocab = (int)vocab;
  a.slices = (int)((dim + kLookupLoads * 32 * n - 1) / (kLookupLoads * 32 * n));
  a.units = (long long)tokens * a.slices;
  a.scale = scale;
  a.status = dev.status;
  void* args[] = {&a};
  return op_launch(fn,
                   dim3((unsigned)std::min<long long>((a.units + kWarps - 1) / kWarps,
                                                      dev.sms * 8LL)),
                   dim3(kThreads), args, 0, stream);
}

vr_result_t vr_embedding_grad_workspace_bytes(size_t tokens, size_t dim, size_t vocab,
                                              vr_dtype_t dtype, size_t* bytes) {
  EmbedPlan p;
  if (!bytes || !make_plan(tokens, dim, vocab, dtype, &p)) return VR_ERR_INVALID_ARGUMENT;
  *bytes = p.bytes;
  return VR_SUCCESS;
}

vr_result_t vr_embedding_grad(const void* dOut, size_t dOutStride, const long long* ids,
                              size_t tokens, size_t dim, size_t vocab, vr_dtype_t dtype,
                              long long ignoreIndex, float scale, int accumulate, void* dWeight,
                              void* workspace, size_t workspaceBytes, void* stream) {
  const size_t E = op_elem_size(dtype);
  EmbedPlan p;
  if (!make_plan(tokens, dim, vocab, dtype, &p) || dOutStride < dim || dOutStride > kMostStride ||
      !dWeight || !workspace || (tokens && (!ids || !dOut)) || ((uintptr_t)ids & 7) ||
      ((uintptr_t)dOut | (uintptr_t)dWeight) % E || ((uintptr_t)workspace & 15) ||
      workspaceBytes < p.bytes)
    return VR_ERR_INVALID_ARGUMENT;
  const OpBuffer buf[4] = {{workspace, 1, workspaceBytes, workspaceBytes, true},
                           {dWeight, 1, vocab * dim * E, vocab * dim * E, true},
                           {dOut, tokens, dim * E, dOutStride * E, false},
                           {ids, 1, tokens * 8, tokens * 8, false}};
  if (!op_buffers_ok(buf, 4)) return VR_ERR_INVALID_ARGUMENT;
  OpDevice dev;
  vr_result_t e = op_device(&dev);
  if (e != VR_SUCCESS || (e = op_reachable(buf, 4, dev.device)) != VR_SUCCESS) return e;
  if (!tokens) {
    if (accumulate) return VR_SUCCESS;
    return cudaMemsetAsync(dWeight, 0, vocab * dim * E, (cudaStream_t)stream) == cudaSuccess
               ? VR_SUCCESS
               : VR_ERR_CUDA;
  }
  choose_sort(&p, tokens, accumulate ? 0.0 : (double)vocab * (double)(dim * E));
  char* w = op_workspace(workspace);
  SortArgs s = {};
  s.ids = ids;
  s.ignore = ignoreIndex;
  s.tokens = (int)tokens;
  s.vocab = (int)vocab;
  s.status = dev.status;
  s.passes = p.passes;
  s.bits = p.bits;
  s.tokenBits = p.tokenBits;
  const int access = access_bytes((uintptr_t)dOut | (uintptr_t)dWeight | (uintptr_t)(dim * E) |
                                      (uintptr_t)(dOutStride * E),
                                  E);
  Item* items = reinterpret_cast<Item*>(w + p.items);
  s.table = static_cast<char*>(dWeight);
  s.rowBytes = (long long)(dim * E);
  s.access = access;
  if (p.few) {  // (the launch that sums is all)
  } else if (p.small) {
    s.out = items;
    void* args[] = {&s};
    const void* fn = p.narrow ? (const void*)embed_sort_small_kernel<unsigned>
                              : (const void*)embed_sort_small_kernel<Item>;
    const unsigned grid =
        accumulate ? 1 : 1 + (unsigned)std::min<size_t>(std::max(dev.sms - 1, 1), vocab);
    if ((e = gemm_prepare(fn, dev.device, kSmallSmem)) != VR_SUCCESS ||
        (e = op_launch(fn, dim3(grid), dim3(kSortThreads), args, kSmallSmem, stream)) != VR_SUCCESS)
      return e;
  } else {
    Item* other = reinterpret_cast<Item*>(w + p.other);
    constexpr size_t kSmem = (size_t)kSortWarps * kDigits * 4;
    const void *count = (const void*)embed_sort_kernel<false>,
               *move = (const void*)embed_sort_kernel<true>;
    if ((e = gemm_prepare(count, dev.device, kSmem)) != VR_SUCCESS ||
        (e = gemm_prepare(move, dev.device, kSmem)) != VR_SUCCESS)
      return e;
    s.counts = reinterpret_cast<int*>(w + p.counts);
    s.ctas = (int)p.ctas;
    s.run = (int)p.run;
    for (int i = 0; i < s.passes; ++i) {
      s.shift = s.tokenBits + i * s.bits;
      // the last pass ends in `items`
      s.out = (s.passes - 1 - i) % 2 ? other : items;
      void* args[] = {&s};
      if ((e = op_launch(count, dim3((unsigned)p.ctas), dim3(kSortThreads), args, kSmem,
                         stream)) != VR_SUCCESS ||
          (e = op_launch(move, dim3((unsigned)p.ctas), dim3(kSortThreads), args, kSmem,
                         stream)) != VR_SUCCESS)
        return e;
      s.in = s.out;
    }
  }
  SumArgs a = {};
  a.dout = dOut;
  a.dweight = dWeight;
  a.items = items;
  a.parts = reinterpret_cast<float*>(w + p.parts);
  a.stride = (long long)dOutStride;
  a.tokens = (int)tokens;
  a.dim = (int)dim;
  a.vocab = (int)vocab;
  a.add = accumulate != 0;
  a.chunk = (int)p.chunk;
  a.chunks = (int)p.chunks;
  a.scale = scale;
  return dtype == VR_FLOAT32   ? sums<float>(p, s, dev, a, access, stream)
         : dtype == VR_FLOAT16 ? sums<__half>(p, s, dev, a, access, stream)
                               : sums<__nv_bfloat16>(p, s, dev, a, access, stream);
}

}  // extern "C"
