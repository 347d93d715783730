// Tokens sorted by expert and back: the stable counting sort of a router's choices, the copy of
// token rows into that order, the weighted sum of the experts' rows back into tokens, and the
// gradients of the last two.
//
// Slot s = token * top_k + j holds the id of the token's j-th expert. Position p of slot s in the
// sorted order is offsets[id] + (slots before s with the same id). Ids outside [0, E) count as one
// more group behind the last, so that `rows` (slot -> position) is always a permutation and a slot
// is kept exactly when its position lies below offsets[E].
//
// All of it is integer work and streaming; no atomics decide an order and none touch global memory,
// so every result is the same bits on every run.
//
// What bounds it. The sort moves a few bytes per slot: 32 slots of 8 experts take 3.2 us and 49146 slots of 64
// experts 4.7 + 5.8 us, launches and dependent loads, not bandwidth. The row kernels are bound by HBM, with 16
// bytes per lane and access (a large copy reaches 5156 GB/s): 8191 tokens of 2048 16-bit columns to 6 experts
// each gathered in 40 us (234 MB, 5.8 TB/s, part of it left in the caches); 8192 tokens of 4096 columns with 4
// experts each combined in 67 us (336 MB, 5.0 TB/s), both gradients in 105 us (604 MB, 5.7 TB/s). 37
// tokens with 8 experts each take 5.1 us: 3 for the launch, the rest two rounds of four slots, whose positions, then
// rows and weights, each wait for a trip to memory.
#include "spt_device.h"
#include "spt_experts.h"

namespace spt {

// ------------------------------------------------------------------------------ counting sort
constexpr int kSortThreads = 1024, kSortWaves = 16;

// Slot numbers are unsigned in loops: a step past the last may pass 2^31.
__device__ __forceinline__ int slot_key(const SortArgs& a, unsigned i) {
  if (a.id64) {
    const int64_t v = ((const int64_t*)a.ids)[i];
    return v >= 0 && v < a.experts ? (int)v : a.experts;
  }
  const int v = ((const int*)a.ids)[i];
  return v >= 0 && v < a.experts ? v : a.experts;
}

// Lanes of the wave that hold the same key (key < 2^bits), among the `active` ones.
__device__ __forceinline__ unsigned long long same_key(int key, int bits, unsigned long long active) {
  unsigned long long m = active;
  for (int b = 0; b < bits; ++b) {
    const unsigned long long set = __ballot((key >> b) & 1);
    m &= (key >> b) & 1 ? set : ~set;
  }
  return m;
}

// Exclusive prefix sum of v over the workgroup's threads; `total` receives the sum. `tmp`: 16 ints.
__device__ __forceinline__ int block_prefix(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) tmp[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int t = tmp[w];
    before += w < wave ? t : 0;
    total += t;
  }
  return before + s - v;
}

// Places the slots [first, last) of one workgroup. cnt[w][e] holds wave w's count of key e on entry
// and start[e] the position of the workgroup's first slot with key e. Each wave owns a contiguous
// run of slots, so the order inside a key is the order of the slots.
__device__ __forceinline__ void place_slots(const SortArgs& a, unsigned first, unsigned last, unsigned run, int* cnt, const int* start) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int keys = a.experts + 1;
  for (int e = threadIdx.x; e < keys; e += kSortThreads) {
    int at = start[e];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = cnt[w * keys + e];
      cnt[w * keys + e] = at;
      at += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.experts);  // keys 0 .. experts
  const unsigned lo = first + wave * run, hi = lo + run < last ? lo + run : last;
  for (unsigned i0 = lo; i0 < hi; i0 += 64) {
    const unsigned i = i0 + lane;
    const bool on = i < hi;
    const unsigned long long active = __ballot(on);
    const int key = on ? slot_key(a, i) : 0;
    const unsigned long long same = same_key(key, bits, active);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int at = 0;
    if (on && rank == 0) at = atomicAdd(&cnt[wave * keys + key], __popcll(same));  // LDS, one lane per key
    at = __shfl(at, same ? __builtin_ctzll(same) : 0) + rank;
    if (on) {
      a.slots[at] = (int)i;
      a.rows_of[i] = at;
    }
  }
}

__device__ __forceinline__ void count_slots(const SortArgs& a, unsigned first, unsigned last, unsigned run, int* cnt) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int keys = a.experts + 1;
  for (int i = threadIdx.x; i < kSortWaves * keys; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const unsigned lo = first + wave * run, hi = lo + run < last ? lo + run : last;
  for (unsigned i = lo + lane; i < hi; i += 64) atomicAdd(&cnt[wave * keys + slot_key(a, i)], 1);
  __syncthreads();
}

// One workgroup sorts everything.
__global__ void __launch_bounds__(kSortThreads) sort_one_kernel(SortArgs a) {
  extern __shared__ int lds[];
  const int keys = a.experts + 1;
  int* cnt = lds;                       // [16][keys]
  int* start = lds + kSortWaves * keys;  // [keys]
  int* tmp = start + keys;              // [16]
  const unsigned run = ((unsigned)(a.rows + kSortWaves - 1) / kSortWaves + 63) & ~63u;
  count_slots(a, 0, a.rows, run, cnt);
  const int e = threadIdx.x;
  int mine = 0, total = 0;
  if (e < a.experts)
    for (int w = 0; w < kSortWaves; ++w) mine += cnt[w * keys + e];
  const int at = block_prefix(mine, tmp, total);
  if (e < a.experts) {
    start[e] = at;
    a.offsets[e] = at;
  }
  if (e == 0) {
    start[a.experts] = total;
    a.offsets[a.experts] = total;
  }
  __syncthreads();
  place_slots(a, 0, a.rows, run, cnt, start);
}

// Many slots: each workgroup counts its keys ...
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(SortArgs a) {
  extern __shared__ int lds[];
  const int keys = a.experts + 1;
  for (int i = threadIdx.x; i < keys; i += kSortThreads) lds[i] = 0;
  __syncthreads();
  const unsigned first = blockIdx.x * a.per_block;
  const unsigned last = a.rows - first < (unsigned)a.per_block ? a.rows : first + a.per_block;
  for (unsigned i = first + threadIdx.x; i < last; i += kSortThreads) atomicAdd(&lds[slot_key(a, i)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < keys; i += kSortThreads) a.counts[(int64_t)blockIdx.x * keys + i] = lds[i];
}

// ... and then places them: the counts of the workgroups before it, and of all of them, give where
// each key of this workgroup starts.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
  extern __shared__ int lds[];
  const int keys = a.experts + 1;
  int* cnt = lds;
  int* start = lds + kSortWaves * keys;
  int* tmp = start + keys;
  int* tot = tmp + kSortWaves;  // [keys]
  for (int i = threadIdx.x; i < keys; i += kSortThreads) start[i] = tot[i] = 0;
  __syncthreads();
  // the threads split into teams of 2^s >= keys threads (one key each); a team adds up every
  // (1024 / 2^s)-th workgroup's counts, and the teams' sums meet in LDS (integers: any order)
  const int s = 32 - __builtin_clz(a.experts);  // 2^s > experts
  if (s < 10) {
    const int e = threadIdx.x & ((1 << s) - 1), team = threadIdx.x >> s, teams = kSortThreads >> s;
    if (e < keys) {
      int all = 0, before = 0;
#pragma unroll 4
      for (int b = team; b < a.blocks; b += teams) {
        const int c = a.counts[(int64_t)b * keys + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&tot[e], all);
      atomicAdd(&start[e], before);
    }
  } else {
    for (int e = threadIdx.x; e < keys; e += kSortThreads) {
      int all = 0, before = 0;
#pragma unroll 4
      for (int b = 0; b < a.blocks; ++b) {
        const int c = a.counts[(int64_t)b * keys + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      tot[e] = all;
      start[e] = before;
    }
  }
  const unsigned first = blockIdx.x * a.per_block;
  const unsigned last = a.rows - first < (unsigned)a.per_block ? a.rows : first + a.per_block;
  const unsigned run = a.per_block / kSortWaves;
  count_slots(a, first, last, run, cnt);  // its barriers also publish tot and start
  const int e = threadIdx.x;
  int total = 0;
  const int at = block_prefix(e < a.experts ? tot[e] : 0, tmp, total);
  if (e < a.experts) {
    start[e] += at;
    if (blockIdx.x == 0) a.offsets[e] = at;
  }
  if (e == 0) {
    start[a.experts] += total;
    if (blockIdx.x == 0) a.offsets[a.experts] = total;
  }
  __syncthreads();
  place_slots(a, first, last, run, cnt, start);
}

// ------------------------------------------------------------------------------ rows
// Eight elements of a row, 16 bytes (32 for fp32), at any element alignment: global accesses of
// these widths need no more than the element's own.
typedef unsigned u32x4u __attribute__((ext_vector_type(4), aligned(2)));
template <int T>
struct Elem {
  static constexpr int size = T == 2 ? 4 : 2;
};
struct Raw8 {
  u32x4 lo, hi;  // hi: fp32 only
};

template <int T>
__device__ __forceinline__ Raw8 load8(const char* row, int col, int width) {
  Raw8 r;
  r.lo = r.hi = u32x4{0, 0, 0, 0};
  const char* p = row + (int64_t)col * Elem<T>::size;
  if (col + 8 <= width) {
    r.lo = *(const u32x4u*)p;
    if constexpr (T == 2) r.hi = *(const u32x4u*)(p + 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + e < width) {
        if constexpr (T == 2) {
          const unsigned v = ((const unsigned*)p)[e];
          if (e < 4) r.lo[e & 3] = v;
          else r.hi[e & 3] = v;
        } else {
          r.lo[e >> 1] |= (unsigned)((const unsigned short*)p)[e] << (16 * (e & 1));
        }
      }
    }
  }
  return r;
}

template <int T>
__device__ __forceinline__ void put8(const Raw8& r, char* row, int col, int width) {
  char* p = row + (int64_t)col * Elem<T>::size;
  if (col + 8 <= width) {
    *(u32x4u*)p = r.lo;
    if constexpr (T == 2) *(u32x4u*)(p + 16) = r.hi;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + e < width) {
        if constexpr (T == 2) ((unsigned*)p)[e] = e < 4 ? r.lo[e & 3] : r.hi[e & 3];
        else ((unsigned short*)p)[e] = (unsigned short)(r.lo[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

template <int T>
__device__ __forceinline__ void to_float(const Raw8& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned word = T == 2 ? (e < 4 ? r.lo[e & 3] : r.hi[e & 3]) : r.lo[e >> 1];
    if constexpr (T == 2) v[e] = __builtin_bit_cast(float, word);
    else if constexpr (T == 1) v[e] = __builtin_bit_cast(float, e & 1 ? word & 0xFFFF0000u : word << 16);
    else v[e] = (float)__builtin_bit_cast(f16x2, word)[e & 1];
  }
}

template <int T>
__device__ __forceinline__ Raw8 from_float(const float (&v)[8]) {
  Raw8 r;
  r.hi = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (T == 2) {
      r.lo[e] = __builtin_bit_cast(unsigned, v[e]);
      r.hi[e] = __builtin_bit_cast(unsigned, v[4 + e]);
    } else {
      r.lo[e] = T == 1 ? pack_bf16(v[2 * e], v[2 * e + 1]) : pack_f16(v[2 * e], v[2 * e + 1]);
    }
  }
  return r;
}

template <int W>
__device__ __forceinline__ float load_weight(const void* w, int64_t i) {
  if constexpr (W == 3) return 1.f;
  else if constexpr (W == 2) return ((const float*)w)[i];
  else if constexpr (W == 1) return __builtin_bit_cast(float, (unsigned)((const unsigned short*)w)[i] << 16);
  else return (float)((const _Float16*)w)[i];
}

// A thread's token and its first chunk of 8 columns: 2^lanes_log2 neighbouring threads share a token,
// blockIdx.y moves them along the row.
struct Place {
  int token, col;
};
__device__ __forceinline__ Place place_of(const RouteArgs& a) {
  const int l = a.lanes_log2;
  const int token = (int)blockIdx.x * (256 >> l) + (int)(threadIdx.x >> l);
  return Place{token, 8 * (int)((blockIdx.y << l) + (threadIdx.x & ((1u << l) - 1)))};
}

// Sorted rows from tokens. A thread reads its chunk of the token once and writes it to each of the
// token's positions: every byte of x is read once however many experts a token has, and the writes, which are
// most of the bytes, go out in whole rows.
template <int T>
__global__ void __launch_bounds__(256) gather_kernel(RouteArgs a) {
  const Place p = place_of(a);
  if (p.token >= a.tokens || p.col >= a.width) return;
  const int slots = a.tokens * a.top_k, kept = clampi(*a.kept, 0, slots);
  const Raw8 v = load8<T>(a.src + (int64_t)p.token * a.ld_src * Elem<T>::size, p.col, a.width);
  Raw8 zero;
  zero.lo = zero.hi = u32x4{0, 0, 0, 0};
  const int* rows = a.rows_of + (int64_t)p.token * a.top_k;
  for (int j = 0; j < a.top_k; ++j) {
    const int at = rows[j];
    char* dst = a.dst + (int64_t)at * a.ld_dst * Elem<T>::size;
    if ((unsigned)at < (unsigned)kept) put8<T>(v, dst, p.col, a.width);
    else if (a.zero_rest && (unsigned)at < (unsigned)slots) put8<T>(zero, dst, p.col, a.width);
  }
}

// Tokens from sorted rows: out[t] = sum over j, in that order, of w[t][j] * src[rows[t][j]], in fp32,
// rounded once. Four rows are loaded before the first is used.
template <int T, int W>
__global__ void __launch_bounds__(256) combine_kernel(RouteArgs a) {
  const Place p = place_of(a);
  if (p.token >= a.tokens || p.col >= a.width) return;
  const int kept = clampi(*a.kept, 0, a.tokens * a.top_k);
  const int64_t s0 = (int64_t)p.token * a.top_k;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    Raw8 r[4];
    float w[4];
    bool on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = j0 + i < a.top_k ? a.rows_of[s0 + j0 + i] : kept;
      on[i] = (unsigned)at < (unsigned)kept;
      if (on[i]) {
        w[i] = load_weight<W>(a.weights, s0 + j0 + i);
        r[i] = load8<T>(a.src + (int64_t)at * a.ld_src * Elem<T>::size, p.col, a.width);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (on[i]) {
        float v[8];
        to_float<T>(r[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = W == 3 ? acc[e] + v[e] : __builtin_fmaf(w[i], v[e], acc[e]);
      }
    }
  }
  put8<T>(from_float<T>(acc), a.dst + (int64_t)p.token * a.ld_dst * Elem<T>::size, p.col, a.width);
}

// Gradients of the weighted sum: dy[rows[t][j]] = w[t][j] * dout[t] and dw[t][j] = <dout[t],
// y[rows[t][j]]>. One workgroup per token: dout is read once per group of four slots (from L1 after the
// first), each row of y once, and the four dot products are added over the lanes, then the waves, in a
// fixed order.
template <int T, int W>
__global__ void __launch_bounds__(256) combine_grad_kernel(RouteArgs a) {
  __shared__ float part[4][4];
  const int token = blockIdx.x;
  const int slots = a.tokens * a.top_k, kept = clampi(*a.kept, 0, slots);
  const int64_t s0 = (int64_t)token * a.top_k;
  const char* drow = a.dout + (int64_t)token * a.ld_dout * Elem<T>::size;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < a.top_k; j0 += 4) {
    float dot[4] = {0.f, 0.f, 0.f, 0.f};
    int at[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at[i] = j0 + i < a.top_k ? a.rows_of[s0 + j0 + i] : -1;
      if (at[i] >= slots) at[i] = -1;
      w[i] = at[i] >= 0 ? load_weight<W>(a.weights, s0 + j0 + i) : 0.f;
    }
    for (int col = 8 * (int)threadIdx.x; col < a.width; col += 8 * 256) {
      const Raw8 d = load8<T>(drow, col, a.width);
      Raw8 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at[i] >= 0 && at[i] < kept) y[i] = load8<T>(a.src + (int64_t)at[i] * a.ld_src * Elem<T>::size, col, a.width);
      float dv[8];
      to_float<T>(d, dv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at[i] < 0) continue;
        float g[8];
        if (at[i] < kept) {
          float yv[8];
          to_float<T>(y[i], yv);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dot[i] = __builtin_fmaf(dv[e], yv[e], dot[i]);
            g[e] = W == 3 ? dv[e] : w[i] * dv[e];
          }
        } else {
          if (!a.zero_rest) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = 0.f;
        }
        put8<T>(from_float<T>(g), a.dst + (int64_t)at[i] * a.ld_dst * Elem<T>::size, col, a.width);
      }
    }
    if constexpr (W != 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 32; d; d >>= 1) dot[i] += __shfl_xor(dot[i], d);
        if (lane == 0) part[i][wave] = dot[i];
      }
      __syncthreads();
      if (threadIdx.x < 4 && j0 + (int)threadIdx.x < a.top_k) {
        const int i = threadIdx.x;
        const float s = ((part[i][0] + part[i][1]) + part[i][2]) + part[i][3];
        const int64_t o = s0 + j0 + i;
        if constexpr (W == 2) ((float*)a.dweights)[o] = s;
        else if constexpr (W == 1) ((unsigned short*)a.dweights)[o] = (unsigned short)pack_bf16(s, 0.f);
        else ((unsigned short*)a.dweights)[o] = (unsigned short)pack_f16(s, 0.f);
      }
      __syncthreads();
    }
  }
}

const void* sort_hist_fn() { return (const void*)&sort_hist_kernel; }
const void* sort_place_fn() { return (const void*)&sort_place_kernel; }
const void* sort_one_fn() { return (const void*)&sort_one_kernel; }

const void* gather_fn(int dtype) {
  static const void* const fn[3] = {(const void*)&gather_kernel<0>, (const void*)&gather_kernel<1>,
                                    (const void*)&gather_kernel<2>};
  return fn[dtype];
}

#define SPT_BY_WEIGHT(K, T) \
  { (const void*)&K<T, 0>, (const void*)&K<T, 1>, (const void*)&K<T, 2>, (const void*)&K<T, 3> }
const void* combine_fn(int dtype, int wtype) {
  static const void* const fn[3][4] = {SPT_BY_WEIGHT(combine_kernel, 0), SPT_BY_WEIGHT(combine_kernel, 1),
                                       SPT_BY_WEIGHT(combine_kernel, 2)};
  return fn[dtype][wtype];
}
const void* combine_grad_fn(int dtype, int wtype) {
  static const void* const fn[3][4] = {SPT_BY_WEIGHT(combine_grad_kernel, 0), SPT_BY_WEIGHT(combine_grad_kernel, 1),
                                       SPT_BY_WEIGHT(combine_grad_kernel, 2)};
  return fn[dtype][wtype];
}

}  // namespace spt
