// embed.cu — embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: Y[t] = scale * E[ids[t]].  Backward: dE[r] = scale * the sum over
// the tokens t with ids[t] = r of dY[t], in fp32, the same bit for bit on
// every run: the tokens are sorted by (id, t) with a stable radix sort, so
// that each touched row is one contiguous segment of the sorted order, and
// the segments are summed in that order.
//
// A user whose tokens are half actions gives segments of very different
// length (an action row holds thousands of tokens, most content rows one or
// two), so the sum is cut by sorted position, not by row: a block takes
// kRun = 96 consecutive positions and 256 columns, each of its 6 warps 16
// positions.  A segment inside one warp's positions is written at once; the
// parts of a segment that passes a warp's border are joined through shared
// memory, and the parts of one that passes a block's border through the
// workspace (at most two partial rows per block), by the last of its blocks.
#include <cuda_bf16.h>
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ptx.cuh"

namespace hstu {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kSortWarps = kSortThreads / 32;
static_assert(kSortWarps == 32, "sort_scan");
constexpr int kMaxCluster = 16;
constexpr int kDigitBits = 10;  // at most; bins of one pass
constexpr int kMaxBins = 1 << kDigitBits;

constexpr int kRunWarps = 6;
constexpr int kRunTokens = 16;                     // sorted positions of one warp
constexpr int kRun = kRunWarps * kRunTokens;       // of one block
constexpr int kColumns = 256;                      // columns of one block, 8 per lane

constexpr int64_t kMaxTokens = 0x7fffffffll - kSortTile;
constexpr int64_t kMaxRows = 0x7ffffffell;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

// ---------------------------------------------------------------- elements
// 8 elements of a row as fp32.  Vector form: the lane's 8 consecutive ones,
// 16 bytes (32 for fp32) at an aligned address.
template <int DT>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<HSTU_FP32> {
  uint4 a, b;
};
DEVI void load8(Raw8<HSTU_BF16>& r, const void* p, int64_t e) {
  r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + e));
}
DEVI void load8(Raw8<HSTU_FP16>& r, const void* p, int64_t e) {
  r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(p) + e));
}
DEVI void load8(Raw8<HSTU_FP32>& r, const void* p, int64_t e) {
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + e);
  r.a = __ldg(q);
  r.b = __ldg(q + 1);
}
// A lane's 8 elements from shared memory (fp32: their two halves 32 vectors apart).
DEVI void from_shared(Raw8<HSTU_BF16>& r, const uint4* p) { r.a = *p; }
DEVI void from_shared(Raw8<HSTU_FP16>& r, const uint4* p) { r.a = *p; }
DEVI void from_shared(Raw8<HSTU_FP32>& r, const uint4* p) {
  r.a = p[0];
  r.b = p[32];
}
DEVI void widen(const Raw8<HSTU_BF16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
DEVI void widen(const Raw8<HSTU_FP16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
DEVI void widen(const Raw8<HSTU_FP32>& r, float (&f)[8]) {
  f[0] = __uint_as_float(r.a.x);
  f[1] = __uint_as_float(r.a.y);
  f[2] = __uint_as_float(r.a.z);
  f[3] = __uint_as_float(r.a.w);
  f[4] = __uint_as_float(r.b.x);
  f[5] = __uint_as_float(r.b.y);
  f[6] = __uint_as_float(r.b.z);
  f[7] = __uint_as_float(r.b.w);
}
template <int DT>
DEVI float load1(const void* p, int64_t e) {
  if (DT == HSTU_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[e]);
  if (DT == HSTU_FP16) return __half2float(static_cast<const __half*>(p)[e]);
  return static_cast<const float*>(p)[e];
}
DEVI float load1_dyn(int dt, const void* p, int64_t e) {
  return dt == HSTU_BF16 ? load1<HSTU_BF16>(p, e)
                         : dt == HSTU_FP16 ? load1<HSTU_FP16>(p, e) : load1<HSTU_FP32>(p, e);
}
// The type of what is written is the same for the whole launch: a branch per
// store instead of a kernel per pair of types.
DEVI void store1(int dt, void* p, int64_t e, float x) {
  if (dt == HSTU_BF16)
    static_cast<__nv_bfloat16*>(p)[e] = __float2bfloat16_rn(x);
  else if (dt == HSTU_FP16)
    static_cast<__half*>(p)[e] = __float2half_rn(x);
  else
    static_cast<float*>(p)[e] = x;
}
DEVI void store8(int dt, void* p, int64_t e, const float (&f)[8]) {
  if (dt == HSTU_FP32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt == HSTU_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- lookup
struct LookupArgs {
  const int64_t* ids;
  const void* table;
  void* out;
  int* status;
  int64_t T, R, ldt, ldo, pad;
  float scale;
  int d, cols;          // cols: threads along a row; blockDim.x = cols * rows per block
  int check;            // block 0 only validates the ids; else every block reports its own
};

constexpr int kLookupUnroll = 4;
constexpr int64_t kCheckMax = 65536;

// Y[t] = scale * E[ids[t]].  38,070 x 1024 bf16 take 19.7 us: 78 MB written and
// as many read through L2, 36 MB of both through DRAM, 4.6 TB/s in all, with
// 54 % of the issue slots used (88 instructions per 8 elements, most of them ids
// and addresses), so neither memory nor issue alone bounds it.  Only setting 78 MB
// to zero takes 12.2; more loads ahead, places of rows in shared memory and other
// numbers of blocks gave 18.9 to 26.  A thread keeps one column group of 8
// elements (1 where a row is not a multiple of 8) and walks the tokens, 4 loads in
// flight, so that no index is divided inside the loop.
// Both types are compiled in: with a branch on the output's type per store the
// kernel was bound by instructions (12.5 per element).  A dropped token's
// loads are replaced by zeros.  (Some of the vector forms spill 4 bytes at their
// register limit.)
// A thread of one block cannot clear the status word before another one sets
// it, so up to kCheckMax tokens block 0 copies nothing and validates all ids
// itself; beyond that the word is cleared by a memset before the launch, 1.5 to
// 3 us.  Checking block against memset, bf16: 1,024 x 64 2.8 and 4.8 us;
// 16,384 x 8 3.3 and 5.0; 16,384 x 1032 12.9 and 14.5; 38,070 x 1024 19.7 and 22.8;
// 65,536 x 8 8.5 and 6.3; 65,536 x 1032 45 and 37: near the border the one block,
// whose time grows with the tokens, is what the launch waits for.
template <int DT, int OUT, bool VEC>
__global__ void __launch_bounds__(256, DT == HSTU_FP32 || OUT == HSTU_FP32 ? 4 : 5)
    k_embed_lookup(const LookupArgs a) {
  if (a.check && blockIdx.x == 0) {
    bool bad = false;
    for (int64_t t = threadIdx.x; t < a.T; t += blockDim.x) {
      const int64_t id = a.ids[t];
      bad |= id != a.pad && (id < 0 || id >= a.R);
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = any ? HSTU_ERR_BAD_IDS : HSTU_OK;
    return;
  }
  const int rows = blockDim.x / a.cols;
  const int c0 = threadIdx.x % a.cols, r0 = threadIdx.x / a.cols;
  const int64_t block = (int64_t)blockIdx.x - a.check, blocks = (int64_t)gridDim.x - a.check;
  const int n_cols = VEC ? a.d / 8 : a.d;
  for (int64_t t0 = block * rows * kLookupUnroll + r0; t0 < a.T;
       t0 += blocks * rows * kLookupUnroll) {
    int64_t from[kLookupUnroll];  // first element of the token's row, -1: none
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
      const int64_t t = t0 + (int64_t)u * rows;
      const int64_t id = t < a.T ? a.ids[t] : a.pad;
      const bool in = id >= 0 && id < a.R;
      if (!a.check && !in && id != a.pad && c0 == 0)
        atomicCAS(a.status, HSTU_OK, HSTU_ERR_BAD_IDS);
      from[u] = in && id != a.pad ? id * a.ldt : -1;
    }
    for (int c = c0; c < n_cols; c += a.cols) {
      if (VEC) {
        Raw8<DT> r[kLookupUnroll];
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u) {
          r[u] = Raw8<DT>{};
          if (from[u] >= 0) load8(r[u], a.table, from[u] + 8 * c);
        }
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u) {
          const int64_t t = t0 + (int64_t)u * rows;
          if (t >= a.T) break;
          float f[8];
          widen(r[u], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= a.scale;
          store8(OUT, a.out, t * a.ldo + 8 * c, f);
        }
      } else {
        float f[kLookupUnroll];
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u)
          f[u] = from[u] >= 0 ? load1<DT>(a.table, from[u] + c) * a.scale : 0.f;
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u) {
          const int64_t t = t0 + (int64_t)u * rows;
          if (t < a.T) store1(OUT, a.out, t * a.ldo + c, f[u]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- sort
// Exclusive scan over the block (kSortThreads threads) of one int per thread;
// *all receives the sum.
DEVI int sort_scan(int v, int* s_warp, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // s_warp is free (previous use done)
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int w = s_warp[lane];  // kSortWarps == 32
  *all = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + incl - v;
}

struct SortArgs {
  const int64_t* ids;
  int64_t pad;
  uint32_t n_rows;         // also the key of tokens that are dropped (pad, bad id)
  int T, tiles, passes, digit;
  uint32_t* key[2];        // ping-pong; keys of pass p in key[p & 1]
  uint32_t* val[2];        // token numbers (pass 0 reads none: position = token)
  uint32_t* hist;          // [tiles, bins] counts, then exclusive over tiles; [bins] totals behind
  int32_t* bad;            // per tile: an id outside the table was seen
  int32_t* heads;          // per tile: touched rows that start in it
  int32_t* sums;           // one-launch sort: per block (bad id seen, heads, live, -)
  uint32_t* rank;          // per sorted position: its segment
  uint32_t* seg_start;     // per segment: its first sorted position; behind the last: the end
  int64_t* row_ids;        // compact form: the touched rows (else null)
  int64_t* n_unique;       // compact form: their number (else null)
  int32_t* status;
  uint32_t* arrived;       // counters of the sums, cleared here
  int64_t n_arrived;
};

// Clears the sums' counters; block `b` of `n`.
DEVI void clear_arrived(const SortArgs& a, int b, int n) {
  for (int64_t i = b * kSortThreads + threadIdx.x; i < a.n_arrived; i += n * kSortThreads)
    a.arrived[i] = 0;
}

DEVI uint32_t token_key(const SortArgs& a, int64_t id, bool* bad) {
  const bool in = id >= 0 && id < (int64_t)a.n_rows;
  *bad = !in && id != a.pad;
  return in && id != a.pad ? (uint32_t)id : a.n_rows;
}

// Counts of one pass's digits in each tile; the first pass also turns ids
// into keys.
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const SortArgs a, int pass) {
  __shared__ uint32_t s_hist[kMaxBins];
  grid_dep_launch();
  grid_dep_wait();
  const int bins = 1 << a.digit, shift = pass * a.digit;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) s_hist[b] = 0;
  __syncthreads();
  const int base = blockIdx.x * kSortTile;
  bool any_bad = false;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * kSortThreads + threadIdx.x;
    if (i < a.T) {
      uint32_t key;
      if (pass == 0) {
        bool bad;
        key = token_key(a, a.ids[i], &bad);
        any_bad |= bad;
        a.key[0][i] = key;
      } else {
        key = a.key[pass & 1][i];
      }
      atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
    }
  }
  const int tile_bad = __syncthreads_or(any_bad);
  if (pass == 0 && threadIdx.x == 0) a.bad[blockIdx.x] = tile_bad;
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    a.hist[(size_t)blockIdx.x * bins + b] = s_hist[b];
}

// Counts -> exclusive sums over the tiles, per digit, and the digits' totals.
__global__ void k_sort_scan(const SortArgs a, int pass) {
  grid_dep_launch();
  grid_dep_wait();
  const int bins = 1 << a.digit;
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < bins) {
    uint32_t sum = 0;
    uint32_t* col = a.hist + b;
#pragma unroll 8
    for (int t = 0; t < a.tiles; ++t) {
      const uint32_t n = col[(size_t)t * bins];
      col[(size_t)t * bins] = sum;
      sum += n;
    }
    col[(size_t)a.tiles * bins] = sum;
  }
  if (pass == 0 && blockIdx.x == 0) {
    bool bad = false;
    for (int t = threadIdx.x; t < a.tiles; t += blockDim.x) bad |= a.bad[t] != 0;
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = any ? HSTU_ERR_BAD_IDS : HSTU_OK;
  }
}

// Ranks a tile's items among those of the same digit, in tile order: each
// warp counts its own 32 * items consecutive items (equal digits of one
// 32-item step found by match: 850 cycles a step of 32 warps, against 1300 with
// one ballot per bit), then the warps' counts are summed up per digit.  Every
// warp's counts (its row of hist, clear_counts) must be zero before.  On return
// hist[w][b] is the number of items of digit b in warps before w, rank[k] this
// thread's item's number inside its warp, and total[b] (if given) the tile's
// number of items of digits 2 b (low half) and 2 b + 1.
DEVI void clear_counts(uint16_t* hist, int bits) {
  const int row = 2 << bits;  // bytes
  uint8_t* mine = reinterpret_cast<uint8_t*>(hist) + (threadIdx.x >> 5) * row;
  for (int i = 4 * (threadIdx.x & 31); i < row; i += 128)
    *reinterpret_cast<uint32_t*>(mine + i) = 0;
  __syncwarp();
}
DEVI void rank_tile(const uint32_t (&digit)[kSortItems], const bool (&in)[kSortItems], int items,
                    int bits, uint16_t* hist, uint32_t (&rank)[kSortItems], uint32_t* total) {
  const int bins = 1 << bits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t* mine = hist + warp * bins;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (k >= items) break;
    const uint32_t d = digit[k];
    const uint32_t peers = __match_any_sync(0xffffffffu, in[k] ? d : 0xffffffffu);
    const uint32_t before = in[k] ? mine[d] : 0;
    rank[k] = before + __popc(peers & ((1u << lane) - 1));
    __syncwarp();
    if (in[k] && lane == __ffs(peers) - 1) mine[d] = (uint16_t)(before + __popc(peers));
    __syncwarp();
  }
  __syncthreads();
  // two digits per thread, as one 32-bit sum (a tile's counts fit 16 bits)
  uint32_t* two = reinterpret_cast<uint32_t*>(hist);
  for (int b = threadIdx.x; b < bins / 2; b += kSortThreads) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t n = two[w * (bins / 2) + b];
      two[w * (bins / 2) + b] = sum;
      sum += n;
    }
    if (total) total[b] = sum;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) k_sort_scatter(const SortArgs a, int pass) {
  extern __shared__ uint16_t s_warp_hist[];
  __shared__ uint32_t s_base[kMaxBins];
  __shared__ int s_scan[kSortWarps];
  grid_dep_launch();
  grid_dep_wait();
  const int bins = 1 << a.digit, shift = pass * a.digit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  {  // first position of each digit of this tile (bins <= threads)
    const int b = threadIdx.x;
    const int total = b < bins ? (int)a.hist[(size_t)a.tiles * bins + b] : 0;
    int all;
    const int base = sort_scan(total, s_scan, &all);
    if (b < bins) s_base[b] = base + a.hist[(size_t)blockIdx.x * bins + b];
  }
  uint32_t key[kSortItems], digit[kSortItems], rank[kSortItems];
  bool in[kSortItems];
  const int base = blockIdx.x * kSortTile + warp * (32 * kSortItems) + lane;
  const uint32_t* src = a.key[pass & 1];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * 32;
    in[k] = i < a.T;
    key[k] = in[k] ? src[i] : 0;
    digit[k] = (key[k] >> shift) & (bins - 1);
  }
  clear_counts(s_warp_hist, a.digit);
  rank_tile(digit, in, kSortItems, a.digit, s_warp_hist, rank, nullptr);
  uint32_t* dst_key = a.key[(pass + 1) & 1];
  uint32_t* dst_val = a.val[(pass + 1) & 1];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (!in[k]) continue;
    const int i = base + k * 32;
    const uint32_t to = s_base[digit[k]] + s_warp_hist[warp * bins + digit[k]] + rank[k];
    dst_key[to] = key[k];
    dst_val[to] = pass == 0 ? (uint32_t)i : a.val[pass & 1][i];
  }
}

// Whether a segment starts at sorted position i; dropped tokens start none.
DEVI bool seg_head(const uint32_t* key, uint32_t n_rows, int i) {
  const uint32_t k = key[i];
  return k < n_rows && (i == 0 || key[i - 1] != k);
}

__global__ void __launch_bounds__(kSortThreads) k_sort_heads(const SortArgs a) {
  __shared__ int s_scan[kSortWarps];
  grid_dep_launch();
  grid_dep_wait();
  clear_arrived(a, blockIdx.x, gridDim.x);
  const uint32_t* key = a.key[a.passes & 1];
  int n = 0;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = blockIdx.x * kSortTile + k * kSortThreads + threadIdx.x;
    n += i < a.T && seg_head(key, a.n_rows, i);
  }
  int all;
  sort_scan(n, s_scan, &all);
  if (threadIdx.x == 0) a.heads[blockIdx.x] = all;
}

// Segment number of every sorted position, each segment's start, the touched
// rows and the counts.
__global__ void __launch_bounds__(kSortThreads) k_sort_segments(const SortArgs a) {
  __shared__ int s_scan[kSortWarps];
  grid_dep_launch();
  grid_dep_wait();
  const uint32_t* key = a.key[a.passes & 1];
  int before = 0;
  for (int t = threadIdx.x; t < (int)blockIdx.x; t += kSortThreads) before += a.heads[t];
  int run;
  sort_scan(before, s_scan, &run);
  const bool last_tile = blockIdx.x == gridDim.x - 1;
  for (int k = 0; k < kSortItems; ++k) {
    const int i = blockIdx.x * kSortTile + k * kSortThreads + threadIdx.x;
    const bool valid = i < a.T && key[i] < a.n_rows;
    const bool h = i < a.T && seg_head(key, a.n_rows, i);
    int all;
    const int pre = sort_scan(h, s_scan, &all);
    if (valid) {
      const int seg = run + pre + h - 1;
      a.rank[i] = (uint32_t)seg;
      if (h) {
        a.seg_start[seg] = (uint32_t)i;
        if (a.row_ids) a.row_ids[seg] = (int64_t)key[i];
      }
      if (i + 1 == a.T || key[i + 1] >= a.n_rows) a.seg_start[seg + 1] = (uint32_t)(i + 1);
    }
    run += all;
  }
  if (last_tile && threadIdx.x == 0 && a.n_unique) *a.n_unique = run;
}

// ---------------------------------------------------------------- one-launch sort
// Up to kClusterTokens tokens are sorted by one cluster of up to 16 blocks,
// each holding its tile of (key, token) pairs in shared memory: a pass ranks
// the tile, adds up the blocks' digit counts and writes every pair into the
// shared memory of the block that its new position falls to.  The blocks'
// digit counts go through global memory: 16 blocks reading 1024 counts of each
// other are 64 KB per block, which took 10,300 cycles a pass as shared-memory
// reads across the cluster and takes 2,400 through L2.  The barriers of a pass
// are the cluster's own (they order global memory too), so the whole sort with
// the segments' numbers is one launch, where the kernels above are 3 per pass
// and 2 more.  It is bound by latency: 19 us for 38,070 tokens of a table of
// 1M rows (two passes of 10 bits, 5 us each), 27 for 82,351, 8 for 3,271 of 8
// rows, against 80 with the kernels above.
//
// The launch's other clusters clear the dense gradient meanwhile (if there is
// one to clear): the sort leaves the memory idle.  Where that leaves room in
// the L2 cache they ask it for dY, which the sums read next (touched rows of
// 38,070 x 1024: 50 -> 46 us).
constexpr int64_t kClusterTokens = (int64_t)kMaxCluster * kSortTile;

struct FillArgs {
  uint8_t* out;        // null: nothing to clear
  int64_t rows, row_bytes, pitch;
  int unit;            // bytes of one element
  const uint8_t* ask;  // null: nothing to ask the L2 cache for
  int64_t ask_bytes;   // a multiple of 16
};

// Asks the L2 cache for dY while the tokens are sorted: at most what leaves
// room in its 126 MB, nothing where it is too little to be worth the extra
// cluster, and nothing beside a larger gradient to clear, which would push it
// out again.  (16 KB per request instead of 4 took twice as long.)
constexpr int64_t kAskMost = (int64_t)96 << 20, kAskLeast = (int64_t)4 << 20,
                  kAskFill = (int64_t)32 << 20;
constexpr int kAskChunk = 4096;
DEVI void ask_l2(const FillArgs& f, int64_t block, int64_t blocks) {
  for (int64_t o = (block * kSortThreads + threadIdx.x) * kAskChunk; o < f.ask_bytes;
       o += blocks * kSortThreads * kAskChunk)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(f.ask + o),
                 "r"((uint32_t)min((int64_t)kAskChunk, f.ask_bytes - o))
                 : "memory");
}

DEVI void fill_zero(const FillArgs& f, int64_t block, int64_t blocks) {
  if (f.row_bytes == f.pitch) {
    const int64_t bytes = f.rows * f.row_bytes, n16 = bytes / 16;
    uint4* q = reinterpret_cast<uint4*>(f.out);
    for (int64_t i = block * kSortThreads + threadIdx.x; i < n16; i += blocks * kSortThreads)
      q[i] = make_uint4(0, 0, 0, 0);
    if (block == 0 && threadIdx.x < 16 && n16 * 16 + threadIdx.x < bytes)
      f.out[n16 * 16 + threadIdx.x] = 0;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t r = block * kSortWarps + warp; r < f.rows; r += blocks * kSortWarps) {
    uint8_t* row = f.out + r * f.pitch;
    for (int64_t c = (int64_t)lane * f.unit; c < f.row_bytes; c += 32 * f.unit) {
      if (f.unit == 4)
        *reinterpret_cast<uint32_t*>(row + c) = 0;
      else
        *reinterpret_cast<uint16_t*>(row + c) = 0;
    }
  }
}

size_t cluster_smem(int tile, int bins) {
  return (size_t)tile * 16 + (size_t)kSortWarps * bins * 2 + (size_t)bins * 4;
}

__global__ void __launch_bounds__(kSortThreads)
    k_embed_sort(const SortArgs a, const FillArgs f, int tile) {
  namespace cg = cooperative_groups;
  extern __shared__ uint4 s_mem[];
  __shared__ int s_scan[kSortWarps];
  __shared__ int s_before;
  grid_dep_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  if ((int)blockIdx.x >= nc) {
    const int64_t block = (int64_t)blockIdx.x - nc, blocks = (int64_t)gridDim.x - nc;
    if (f.out) fill_zero(f, block, blocks);
    if (f.ask) ask_l2(f, block, blocks);
    return;
  }
  clear_arrived(a, c, nc);
  const int bins = 1 << a.digit;
  uint2* pair = reinterpret_cast<uint2*>(s_mem);  // (key, token)
  uint2* pair2 = pair + tile;
  uint16_t* hist = reinterpret_cast<uint16_t*>(pair2 + tile);
  uint32_t* base = reinterpret_cast<uint32_t*>(hist + kSortWarps * bins);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = min(max(a.T - c * tile, 0), tile);
  const int items = (tile + kSortThreads - 1) / kSortThreads;
  const int w0 = warp * 32 * items + lane;  // this thread's items: w0 + 32 k
  uint2 x[kSortItems];
  bool in[kSortItems];
  bool bad = false;
  {
    int64_t id[kSortItems];
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      in[k] = k < items && w0 + 32 * k < n;
      id[k] = in[k] ? a.ids[c * tile + w0 + 32 * k] : 0;
    }
    clear_counts(hist, a.digit);
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      bool b;
      x[k] = make_uint2(token_key(a, id[k], &b), (uint32_t)(c * tile + w0 + 32 * k));
      bad |= in[k] && b;
    }
  }
  for (int p = 0; p < a.passes; ++p) {
    uint32_t digit[kSortItems], rank[kSortItems];
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      if (p > 0) x[k] = in[k] ? pair[w0 + 32 * k] : make_uint2(0, 0);
      digit[k] = (x[k].x >> (p * a.digit)) & (bins - 1);
    }
    rank_tile(digit, in, items, a.digit, hist, rank, a.hist + c * (bins / 2));
    cluster.sync();  // every block's totals
    uint32_t b0 = 0, b1 = 0, all0 = 0, all1 = 0;  // two digits: before this block, of all
    if (tid < bins / 2) {
      uint32_t t[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        t[r] = r < nc ? __ldcg(a.hist + r * (bins / 2) + tid) : 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        all0 += t[r] & 0xffffu;
        all1 += t[r] >> 16;
        b0 += r < c ? t[r] & 0xffffu : 0;
        b1 += r < c ? t[r] >> 16 : 0;
      }
    }
    int sum;
    const uint32_t first = (uint32_t)sort_scan((int)(all0 + all1), s_scan, &sum);
    if (tid < bins / 2) {
      base[2 * tid] = first + b0;
      base[2 * tid + 1] = first + all0 + b1;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSortItems; ++k) {
      if (!in[k]) continue;
      const uint32_t to = base[digit[k]] + hist[warp * bins + digit[k]] + rank[k];
      const uint32_t r = to / (uint32_t)tile;
      cluster.map_shared_rank(pair2, (int)r)[to - r * (uint32_t)tile] = x[k];
    }
    __syncwarp();
    if (p + 1 < a.passes) clear_counts(hist, a.digit);
    cluster.sync();  // every pair has arrived
    uint2* t = pair;
    pair = pair2;
    pair2 = t;
  }
  uint32_t* out_key = a.key[a.passes & 1] + c * tile;
  uint32_t* out_val = a.val[a.passes & 1] + c * tile;
  for (int i = tid; i < n; i += kSortThreads) {
    out_key[i] = pair[i].x;
    out_val[i] = pair[i].y;
  }
  // segments: this thread's `items` consecutive sorted positions
  const uint32_t left = c > 0 && n > 0 ? cluster.map_shared_rank(pair, c - 1)[tile - 1].x : 0;
  const int i0 = tid * items;
  int count = 0;  // heads in the low half, live tokens in the high half
  for (int k = 0; k < items; ++k) {
    const int i = i0 + k;
    if (i >= n) break;
    const uint32_t key = pair[i].x;
    const bool first = c == 0 && i == 0;
    if (key < a.n_rows)
      count += 0x10000 + (first || (i > 0 ? pair[i - 1].x : left) != key);
  }
  int all;
  int seg = sort_scan(count, s_scan, &all) & 0xffff;
  const int any_bad = __syncthreads_or(bad);
  if (tid == 0)
    *reinterpret_cast<int4*>(a.sums + 4 * c) = make_int4(any_bad, all & 0xffff, all >> 16, 0);
  cluster.sync();  // the blocks' sums; and no block's shared memory is read by another any more
  if (warp == 0) {
    const int4 o = lane < nc ? __ldcg(reinterpret_cast<const int4*>(a.sums) + lane)
                             : make_int4(0, 0, 0, 0);
    const int before = __reduce_add_sync(0xffffffffu, lane < c ? o.y : 0);
    const int bads = __reduce_add_sync(0xffffffffu, o.x);
    const int heads = __reduce_add_sync(0xffffffffu, o.y);
    const int live = __reduce_add_sync(0xffffffffu, o.z);
    if (lane == 0) {
      s_before = before;
      if (c == 0) {
        *a.status = bads ? HSTU_ERR_BAD_IDS : HSTU_OK;
        a.seg_start[heads] = (uint32_t)live;
        if (a.n_unique) *a.n_unique = heads;
      }
    }
  }
  __syncthreads();
  seg += s_before;
  // through the buffer that is free now, so that they are written side by side
  uint32_t* number = reinterpret_cast<uint32_t*>(pair2);
  for (int k = 0; k < items; ++k) {
    const int i = i0 + k;
    if (i >= n) break;
    const uint32_t key = pair[i].x;
    if (key >= a.n_rows) break;
    if ((c == 0 && i == 0) || (i > 0 ? pair[i - 1].x : left) != key) {
      a.seg_start[seg] = (uint32_t)(c * tile + i);
      if (a.row_ids) a.row_ids[seg] = (int64_t)key;
      ++seg;
    }
    number[i] = (uint32_t)(seg - 1);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kSortThreads) a.rank[c * tile + i] = number[i];
}

// ---------------------------------------------------------------- sums
struct SumArgs {
  int T;
  uint32_t n_rows;
  const uint32_t* key;
  const uint32_t* val;
  const uint32_t* rank;
  const uint32_t* seg_start;
  const void* dY;
  void* out;
  float* part;        // [runs, 2, ld_part]
  uint32_t* arrived;  // [runs, column blocks]: blocks of the segment starting there that are done
  int64_t ld_dy, ld_out;
  float scale;
  int d, ld_part, out_dt, compact, accumulate;
};

// Writes (or adds into) a row of the gradient, this lane's 8 columns: 8 lane +
// 0 .. 7 (VEC), or lane + 32 j.  PLAIN: fp32, not accumulated.
template <bool VEC, bool PLAIN>
DEVI void write_row(const SumArgs& a, uint32_t key, uint32_t rank, int c0, int lane,
                    const float (&acc)[8]) {
  const int64_t at = (int64_t)(a.compact ? rank : key) * a.ld_out + c0;
  if (VEC) {
    if (c0 + 8 * lane >= a.d) return;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = acc[j] * a.scale;
      if (!PLAIN && a.accumulate) f[j] += load1_dyn(a.out_dt, a.out, at + 8 * lane + j);
    }
    store8(PLAIN ? HSTU_FP32 : a.out_dt, a.out, at + 8 * lane, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 32 * j + lane;
      if (c0 + c < a.d) {
        float f = acc[j] * a.scale;
        if (!PLAIN && a.accumulate) f += load1_dyn(a.out_dt, a.out, at + c);
        store1(PLAIN ? HSTU_FP32 : a.out_dt, a.out, at + c, f);
      }
    }
  }
}

// Partial rows keep the lane's own order (8 floats per lane), in either form.
DEVI void put8(float* p, int lane, const float (&f)[8]) {
  float4* q = reinterpret_cast<float4*>(p + 8 * lane);
  q[0] = make_float4(f[0], f[1], f[2], f[3]);
  q[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <bool L2 = false>  // L2: written by another block of this launch
DEVI void add8(const float* p, int lane, float (&f)[8]) {
  const float4* q = reinterpret_cast<const float4*>(p + 8 * lane);
  const float4 x = L2 ? __ldcg(q) : q[0], y = L2 ? __ldcg(q + 1) : q[1];
  f[0] += x.x;
  f[1] += x.y;
  f[2] += x.z;
  f[3] += x.w;
  f[4] += y.x;
  f[5] += y.y;
  f[6] += y.z;
  f[7] += y.w;
}

// Where a segment that passes a block's border lies.
struct Chain {
  uint32_t key, seg;
  int start, end;  // sorted positions; start < 0: there is none
};

// Sums of one run of sorted positions and 256 columns.  A warp's 16 positions:
// lane i + 1 holds position i's key, token and segment, lane 0 the key before,
// lane 17 the key behind; one ballot tells where segments start, so the loop
// over the tokens has no exchange but the token's number.
template <int DT, bool VEC, bool PLAIN>
__global__ void __launch_bounds__(kRunWarps * 32, VEC ? 6 : 3) k_embed_sum(const SumArgs a) {
  __shared__ float s_pre[kRunWarps][kColumns], s_post[kRunWarps][kColumns];
  constexpr int kBatch = VEC && DT == HSTU_FP32 ? 2 : 4;  // rows
  constexpr int kVecs = DT == HSTU_FP32 ? 2 : 1;          // 16 bytes of a row per lane
  __shared__ uint4 s_rows[VEC ? kRunWarps : 1][2][kBatch][kVecs][32];
  __shared__ int s_flags[kRunWarps];  // 1: pre holds a part, 2: it goes on past this warp
  __shared__ Chain s_chain[2];        // of the run's first position, and of its last one
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b0 = blockIdx.x * kRun, c0 = blockIdx.y * kColumns;
  grid_dep_wait();
  const int pos = b0 + warp * kRunTokens + lane - 1;
  const bool mine = lane >= 1 && lane <= kRunTokens && pos < a.T;
  const uint32_t key = lane <= kRunTokens + 1 && pos >= 0 && pos < a.T ? a.key[pos] : 0xffffffffu;
  const uint32_t val = mine ? a.val[pos] : 0, rank = mine ? a.rank[pos] : 0;
  const uint32_t before = __shfl_up_sync(0xffffffffu, key, 1);
  const int n = __popc(__ballot_sync(0xffffffffu, mine && key < a.n_rows));  // the first n
  const uint32_t heads = __ballot_sync(0xffffffffu, mine && key != before) >> 1;
  const uint32_t last_key = __shfl_sync(0xffffffffu, key, n);
  const bool on = n > 0 && __shfl_sync(0xffffffffu, key, n + 1) == last_key;  // behind this warp
  bool open = n > 0 && !(heads & 1);  // the running segment began before this warp's positions
  const uint32_t last_rank = __shfl_sync(0xffffffffu, rank, n);
  // the segments at the run's borders, which its first and its last warp see: lanes 0 and 1 read
  // where they start and end
  const bool edge = warp == 0 || warp == kRunWarps - 1;
  const bool chained = warp == 0 ? open : on && n == kRunTokens;
  const uint32_t edge_seg = warp == 0 ? __shfl_sync(0xffffffffu, rank, 1) : last_rank;
  int bound = -1;
  if (edge && chained && lane < 2) bound = (int)a.seg_start[edge_seg + lane];
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  int flags = 0;
  // Vector form: rows are copied into shared memory, each lane its own 16 bytes (32 of fp32), two
  // groups of 2 KB ahead of the sums, where they take no registers: 6 warps a block, 6 blocks a
  // SM, 56 registers (dense gradient of 65,536 x 512: 1.6 us less than with 4 rows in registers;
  // 7 blocks spill, 6 us more).  A lane reads what it copied itself, so no exchange is needed.
  const bool col = c0 + 8 * lane < a.d;
  auto ask = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t t = __shfl_sync(0xffffffffu, val, (i0 + u + 1) & 31);
      if (i0 + u < n && col) {
        const uint8_t* src = static_cast<const uint8_t*>(a.dY) +
                             ((int64_t)t * a.ld_dy + c0 + 8 * lane) * (DT == HSTU_FP32 ? 4 : 2);
#pragma unroll
        for (int q = 0; q < kVecs; ++q)
          copy16(&s_rows[warp][(i0 / kBatch) & 1][u][q][lane], src + 16 * q);
      }
    }
    copy_commit();
  };
  if (VEC) {
    ask(0);
    ask(kBatch);
  }
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float one[VEC ? 1 : kBatch][8];
    if (VEC) {
      copy_wait_but_one();
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t row = (int64_t)__shfl_sync(0xffffffffu, val, i0 + u + 1) * a.ld_dy + c0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = 32 * j + lane;
          one[u][j] = 0.f;
          if (c0 + 32 * j < a.d && i0 + u < n && c0 + c < a.d) one[u][j] = load1<DT>(a.dY, row + c);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      if (i > 0 && (heads >> i & 1)) {  // the running segment ended with token i - 1
        if (open) {
          put8(s_pre[warp], lane, acc);
          flags = 1;
        } else {
          write_row<VEC, PLAIN>(a, __shfl_sync(0xffffffffu, key, i),
                                __shfl_sync(0xffffffffu, rank, i), c0, lane, acc);
        }
        open = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
      }
      if (VEC) {
        Raw8<DT> r;
        float x[8];
        from_shared(r, &s_rows[warp][(i0 / kBatch) & 1][u][0][lane]);
        widen(r, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += x[j];  // columns past the end: not written
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += one[u][j];
      }
    }
    if (VEC) ask(i0 + 2 * kBatch);
  }
  bool post = false;
  if (n > 0) {
    if (open) {
      put8(s_pre[warp], lane, acc);
      flags = on ? 3 : 1;
    } else if (on) {
      put8(s_post[warp], lane, acc);
      post = true;
    } else {
      write_row<VEC, PLAIN>(a, last_key, last_rank, c0, lane, acc);
    }
  }
  if (lane == 0) s_flags[warp] = flags;
  if (edge) {
    const int end = __shfl_sync(0xffffffffu, bound, 1);
    // (a segment that fills the run is the first border's; its key is also lane 0's)
    if (lane == 0)
      s_chain[warp != 0] = Chain{warp == 0 ? key : last_key, edge_seg,
                                 warp == 0 || bound >= b0 ? bound : -1, end};
  }
  __syncthreads();
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.ld_part + c0;
  // the part that began before this block, and this warp's own segment that goes on
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !(warp == 0 && (flags & 1)) : !post) continue;
    int w = which == 0 ? 0 : warp;
    bool done = which == 0 && !(flags & 2);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    add8(which == 0 ? s_pre[0] : s_post[warp], lane, acc);
    while (!done && ++w < kRunWarps) {
      add8(s_pre[w], lane, acc);
      done = !(s_flags[w] & 2);
    }
    if (which == 0)
      put8(part, lane, acc);
    else if (done)
      write_row<VEC, PLAIN>(a, last_key, last_rank, c0, lane, acc);
    else
      put8(part + a.ld_part, lane, acc);
  }
  // Segments that pass this block's borders: the last of a segment's blocks to
  // get here joins its parts (in their order, whoever it is).
  for (int which = 0; which < 2; ++which) {
    const Chain x = s_chain[which];
    if (x.start < 0) continue;
    const int first = x.start / kRun, last = (x.end - 1) / kRun;
    __syncthreads();  // the parts are written, and s_flags is free
    if (threadIdx.x == 0) {
      __threadfence();
      s_flags[0] = (int)atomicAdd(&a.arrived[(int64_t)first * gridDim.y + blockIdx.y], 1u) ==
                   last - first;
    }
    __syncthreads();
    if (!s_flags[0]) continue;
    __threadfence();
    const int per = (last - first + kRunWarps) / kRunWarps;  // of the runs behind the first
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if (warp == 0) add8<true>(a.part + ((int64_t)first * 2 + 1) * a.ld_part + c0, lane, acc);
    const int r1 = min(first + 1 + (warp + 1) * per, last + 1);
#pragma unroll 8
    for (int r = first + 1 + warp * per; r < r1; ++r)
      add8<true>(a.part + (int64_t)r * 2 * a.ld_part + c0, lane, acc);
    put8(s_pre[warp], lane, acc);
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kRunWarps; ++w) add8(s_pre[w], lane, acc);
      write_row<VEC, PLAIN>(a, x.key, x.seg, c0, lane, acc);
    }
  }
}

// ---------------------------------------------------------------- host
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool dtype_ok(int32_t t) { return t == HSTU_BF16 || t == HSTU_FP32 || t == HSTU_FP16; }
size_t dsize(int32_t t) { return t == HSTU_FP32 ? 4 : 2; }

struct BwdLayout {
  size_t head, key[2], val[2], hist, bad, heads, sums, rank, seg_start, arrived, part, total;
  int tiles, passes, digit, runs, ld_part;
  int64_t n_arrived;
};

bool bwd_layout(int64_t T, int64_t R, int32_t d, BwdLayout* L) {
  if (T < 0 || T > kMaxTokens || R < 1 || R > kMaxRows || d < 1 || d > (1 << 20)) return false;
  int bits = 1;
  while (bits < 31 && ((int64_t)1 << bits) <= R) ++bits;  // keys 0 .. R (R: dropped)
  L->passes = (bits + kDigitBits - 1) / kDigitBits;
  L->digit = (bits + L->passes - 1) / L->passes;
  L->tiles = (int)((T + kSortTile - 1) / kSortTile);
  L->runs = (int)((T + kRun - 1) / kRun);
  L->ld_part = (d + kColumns - 1) / kColumns * kColumns;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~size_t(255);
    return o;
  };
  L->head = take(256);
  for (int i = 0; i < 2; ++i) {
    L->key[i] = take((size_t)T * 4);
    L->val[i] = take((size_t)T * 4);
  }
  L->hist = take((size_t)std::max(L->tiles + 1, kMaxCluster) * 4 << L->digit);
  L->sums = take(kMaxCluster * 16);
  L->bad = take((size_t)L->tiles * 4);
  L->heads = take((size_t)L->tiles * 4);
  L->rank = take((size_t)T * 4);
  L->seg_start = take(((size_t)T + 1) * 4);
  L->n_arrived = (int64_t)L->runs * (L->ld_part / kColumns);
  L->arrived = take((size_t)L->n_arrived * 4);
  L->part = take((size_t)L->runs * 2 * L->ld_part * 4);
  L->total = off;
  return true;
}

// Launches with programmatic stream serialization: the kernel may start while
// its predecessor runs and waits for it (griddepcontrol.wait) before touching
// anything.
template <typename... P, typename... A>
cudaError_t launch_dep(int id, void (*fn)(P...), dim3 grid, int threads, size_t smem,
                       cudaStream_t s, bool dep, A... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = dep ? 1 : 0;
  LaunchScope ls(id, s);
  return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

cudaError_t sort_tokens(const SortArgs& a, cudaStream_t s) {
  const int bins = 1 << a.digit;
  const size_t smem = (size_t)kSortWarps * bins * 2;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(k_sort_scatter), (int)smem);
  for (int p = 0; p < a.passes && e == cudaSuccess; ++p) {
    e = launch_dep(K_EMBED_SORT, k_sort_count, dim3(a.tiles), kSortThreads, 0, s, p > 0, a, p);
    if (e == cudaSuccess)
      e = launch_dep(K_EMBED_SORT, k_sort_scan, dim3((bins + 63) / 64), 64, 0, s, true, a, p);
    if (e == cudaSuccess)
      e = launch_dep(K_EMBED_SORT, k_sort_scatter, dim3(a.tiles), kSortThreads, smem, s, true, a, p);
  }
  if (e == cudaSuccess)
    e = launch_dep(K_EMBED_SORT, k_sort_heads, dim3(a.tiles), kSortThreads, 0, s, true, a);
  if (e == cudaSuccess)
    e = launch_dep(K_EMBED_SORT, k_sort_segments, dim3(a.tiles), kSortThreads, 0, s, true, a);
  return e;
}

// Blocks of the sort's cluster: a power of two with at least 1024 tokens each
// where there are so many (a block's pass costs about the same for 1 to 1024
// tokens).
int cluster_blocks(int64_t T) {
  int n = 1;
  while (n < kMaxCluster && (int64_t)n * kSortThreads < T) n *= 2;
  return n;
}

// The one-launch sort; *done = false if this device cannot run it.
cudaError_t sort_tokens_cluster(const SortArgs& a, const FillArgs& f, cudaStream_t s, bool* done) {
  const int nc = cluster_blocks(a.T), bins = 1 << a.digit;
  const int tile = ((a.T + nc - 1) / nc + 31) / 32 * 32;
  const size_t smem = cluster_smem(tile, bins);
  *done = false;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(k_embed_sort), (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)nc;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)nc);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int resident = clusters_resident(reinterpret_cast<const void*>(k_embed_sort), nc, cfg);
  if (resident == 0) return cudaSuccess;
  if (f.out || f.ask) {
    // clusters that clear and ask: 64 KB or more for each of their blocks, and no more than run at
    // once beside the sort (clusters of 16 lie within a GPC: one more than that waited for the
    // first to end, and the dense gradient of 65,536 x 512 took 67 us instead of 57)
    const int64_t bytes = (f.out ? f.rows * f.row_bytes : 0) + f.ask_bytes;
    const int64_t fill = std::min<int64_t>((bytes + 65535) / 65536 / nc + 1, resident - 1);
    cfg.gridDim.x = (unsigned)(nc * (1 + std::max<int64_t>(fill, 1)));
  }
  *done = true;
  LaunchScope ls(K_EMBED_SORT, s);
  return cudaLaunchKernelEx(&cfg, k_embed_sort, a, f, tile);
}

cudaError_t clear_rows(const FillArgs& f, cudaStream_t s) {
  return f.row_bytes == f.pitch
             ? cudaMemsetAsync(f.out, 0, (size_t)(f.rows * f.row_bytes), s)
             : cudaMemset2DAsync(f.out, (size_t)f.pitch, 0, (size_t)f.row_bytes, (size_t)f.rows, s);
}

template <int DT>
cudaError_t sum_rows(const SumArgs& a, int runs, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)runs, (unsigned)((a.d + kColumns - 1) / kColumns));
  const bool plain = a.out_dt == HSTU_FP32 && !a.accumulate;
  auto* fn = vec ? plain ? k_embed_sum<DT, true, true> : k_embed_sum<DT, true, false>
                 : plain ? k_embed_sum<DT, false, true> : k_embed_sum<DT, false, false>;
  return launch_dep(K_EMBED_SUM, fn, grid, kRunWarps * 32, 0, s, true, a);
}

hstu_status cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return HSTU_OK;
  note_cuda_error(e, where);
  return HSTU_ERR_CUDA;
}

hstu_status embed_bwd(int64_t T, const int64_t* ids, const void* dY, int32_t dy_dt, int64_t ld_dy,
                      int64_t R, int32_t d, int64_t pad, float scale, int accumulate, int compact,
                      int64_t* row_ids, int64_t* n_unique, void* out, int32_t out_dt,
                      int64_t ld_out, void* ws, size_t ws_bytes, cudaStream_t s) {
  BwdLayout L;
  if (!bwd_layout(T, R, d, &L)) return HSTU_ERR_INVALID_ARG;
  if (!dtype_ok(dy_dt) || !dtype_ok(out_dt) || ld_dy < d || ld_out < d || ld_dy > kMaxStride ||
      ld_out > kMaxStride)
    return HSTU_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return HSTU_ERR_INVALID_ARG;
  if (!(scale - scale == 0.f)) return HSTU_ERR_INVALID_ARG;  // NaN or infinite
  if (T > 0 && (!ids || !dY || !out)) return HSTU_ERR_INVALID_ARG;
  if (compact && (!n_unique || (T > 0 && !row_ids))) return HSTU_ERR_INVALID_ARG;
  if (!compact && !out) return HSTU_ERR_INVALID_ARG;
  if (!al16(ids) || !al16(dY) || !al16(out) || !al16(row_ids) || !al16(n_unique))
    return HSTU_ERR_INVALID_ARG;
  if (!ws || ws_bytes < L.total || !al256(ws)) return HSTU_ERR_WORKSPACE;
  auto at = [&](size_t o) { return static_cast<uint8_t*>(ws) + o; };
  int32_t* status = reinterpret_cast<int32_t*>(at(L.head));
  FillArgs f{};
  if (!compact && !accumulate) {
    f.out = static_cast<uint8_t*>(out);
    f.rows = R;
    f.unit = (int)dsize(out_dt);
    f.row_bytes = (int64_t)d * f.unit;
    f.pitch = ld_out * f.unit;
  }
  const int64_t dy_bytes = T > 0 ? ((T - 1) * ld_dy + d) * (int64_t)dsize(dy_dt) : 0;
  if (ld_dy < 2 * (int64_t)d && f.rows * f.row_bytes <= kAskFill) {
    f.ask = static_cast<const uint8_t*>(dY);
    f.ask_bytes = std::min(dy_bytes, kAskMost) / 16 * 16;
    if (f.ask_bytes < kAskLeast) f.ask = nullptr, f.ask_bytes = 0;
  }
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess && f.out) e = clear_rows(f, s);
    if (e == cudaSuccess && compact) e = cudaMemsetAsync(n_unique, 0, 8, s);
    return cuda_status(e, "embed_bwd: empty batch");
  }
  SortArgs q{};
  q.ids = ids;
  q.pad = pad;
  q.n_rows = (uint32_t)R;
  q.T = (int)T;
  q.tiles = L.tiles;
  q.passes = L.passes;
  q.digit = L.digit;
  for (int i = 0; i < 2; ++i) {
    q.key[i] = reinterpret_cast<uint32_t*>(at(L.key[i]));
    q.val[i] = reinterpret_cast<uint32_t*>(at(L.val[i]));
  }
  q.hist = reinterpret_cast<uint32_t*>(at(L.hist));
  q.bad = reinterpret_cast<int32_t*>(at(L.bad));
  q.heads = reinterpret_cast<int32_t*>(at(L.heads));
  q.sums = reinterpret_cast<int32_t*>(at(L.sums));
  q.rank = reinterpret_cast<uint32_t*>(at(L.rank));
  q.seg_start = reinterpret_cast<uint32_t*>(at(L.seg_start));
  q.row_ids = compact ? row_ids : nullptr;
  q.n_unique = compact ? n_unique : nullptr;
  q.status = status;
  q.arrived = reinterpret_cast<uint32_t*>(at(L.arrived));
  q.n_arrived = L.n_arrived;
  cudaError_t e = cudaSuccess;
  bool sorted = false;
  if (T <= kClusterTokens) e = sort_tokens_cluster(q, f, s, &sorted);
  if (e == cudaSuccess && !sorted) {
    if (f.out) e = clear_rows(f, s);
    if (e == cudaSuccess) e = sort_tokens(q, s);
  }
  if (e != cudaSuccess) return cuda_status(e, "embed_bwd: sort");
  SumArgs a{};
  a.T = (int)T;
  a.n_rows = (uint32_t)R;
  a.key = q.key[L.passes & 1];
  a.val = q.val[L.passes & 1];
  a.rank = q.rank;
  a.seg_start = q.seg_start;
  a.dY = dY;
  a.out = out;
  a.part = reinterpret_cast<float*>(at(L.part));
  a.arrived = q.arrived;
  a.ld_dy = ld_dy;
  a.ld_out = ld_out;
  a.scale = scale;
  a.d = d;
  a.ld_part = L.ld_part;
  a.out_dt = out_dt;
  a.compact = compact;
  a.accumulate = accumulate;
  const bool vec = d % 8 == 0 && ld_dy % 8 == 0 && ld_out % 8 == 0;
  e = dy_dt == HSTU_BF16   ? sum_rows<HSTU_BF16>(a, L.runs, vec, s)
      : dy_dt == HSTU_FP16 ? sum_rows<HSTU_FP16>(a, L.runs, vec, s)
                           : sum_rows<HSTU_FP32>(a, L.runs, vec, s);
  return cuda_status(e, "embed_bwd: sums");
}

template <int DT, int OUT>
cudaError_t lookup(const LookupArgs& a, bool vec, int threads, int grid, cudaStream_t s) {
  LaunchScope ls(K_EMBED_LOOKUP, s);
  if (vec)
    k_embed_lookup<DT, OUT, true><<<grid, threads, 0, s>>>(a);
  else
    k_embed_lookup<DT, OUT, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}
template <int DT>
cudaError_t lookup(const LookupArgs& a, int out, bool vec, int threads, int grid, cudaStream_t s) {
  return out == HSTU_BF16   ? lookup<DT, HSTU_BF16>(a, vec, threads, grid, s)
         : out == HSTU_FP16 ? lookup<DT, HSTU_FP16>(a, vec, threads, grid, s)
                            : lookup<DT, HSTU_FP32>(a, vec, threads, grid, s);
}

}  // namespace
}  // namespace hstu

// ---------------------------------------------------------------- C ABI
extern "C" {

size_t hstu_embed_workspace_size(void) { return 256; }

hstu_status hstu_embed_fwd(int64_t n_tokens, const int64_t* ids, const void* table,
                           int32_t table_dtype, int64_t n_rows, int32_t d, int64_t ld_table,
                           int64_t pad_id, float scale, void* out, int32_t out_dtype,
                           int64_t ld_out, void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_tokens < 0 || n_tokens > kMaxTokens || n_rows < 1 || n_rows > kMaxRows || d < 1 ||
      d > (1 << 20) || ld_table < d || ld_out < d || ld_table > kMaxStride || ld_out > kMaxStride ||
      !dtype_ok(table_dtype) || !dtype_ok(out_dtype))
    return HSTU_ERR_INVALID_ARG;
  if (!(scale - scale == 0.f)) return HSTU_ERR_INVALID_ARG;  // NaN or infinite
  if (n_tokens > 0 && (!ids || !table || !out)) return HSTU_ERR_INVALID_ARG;
  if (!al16(ids) || !al16(table) || !al16(out)) return HSTU_ERR_INVALID_ARG;
  if (!ws || ws_bytes < hstu_embed_workspace_size() || !al256(ws)) return HSTU_ERR_WORKSPACE;
  LookupArgs a{};
  a.ids = ids;
  a.table = table;
  a.out = out;
  a.status = static_cast<int*>(ws);
  a.T = n_tokens;
  a.R = n_rows;
  a.ldt = ld_table;
  a.ldo = ld_out;
  a.pad = pad_id;
  a.scale = scale;
  a.d = d;
  a.check = n_tokens <= kCheckMax;
  const bool vec = d % 8 == 0 && ld_table % 8 == 0 && ld_out % 8 == 0;
  const int n_cols = vec ? d / 8 : d;
  a.cols = n_cols <= 256 ? n_cols : 256;
  const int rows = std::max(1, 256 / a.cols);
  const int threads = a.cols * rows;
  const int64_t per = (int64_t)rows * kLookupUnroll;
  const int64_t blocks = std::min<int64_t>((n_tokens + per - 1) / per, (int64_t)num_sms() * 16);
  if (!a.check) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), s);
    if (e != cudaSuccess) return cuda_status(e, "hstu_embed_fwd");
  }
  const int grid = (int)blocks + a.check;
  const cudaError_t e =
      table_dtype == HSTU_BF16   ? lookup<HSTU_BF16>(a, out_dtype, vec, threads, grid, s)
      : table_dtype == HSTU_FP16 ? lookup<HSTU_FP16>(a, out_dtype, vec, threads, grid, s)
                                 : lookup<HSTU_FP32>(a, out_dtype, vec, threads, grid, s);
  return cuda_status(e, "hstu_embed_fwd");
}

size_t hstu_embed_bwd_workspace_size(int64_t n_tokens, int64_t n_rows, int32_t d) {
  hstu::BwdLayout L;
  return hstu::bwd_layout(n_tokens, n_rows, d, &L) ? L.total : 0;
}

hstu_status hstu_embed_bwd(int64_t n_tokens, const int64_t* ids, const void* dY, int32_t dy_dtype,
                           int64_t ld_dy, int64_t n_rows, int32_t d, int64_t pad_id, float scale,
                           int32_t accumulate, void* dE, int32_t de_dtype, int64_t ld_de, void* ws,
                           size_t ws_bytes, void* stream) {
  return hstu::embed_bwd(n_tokens, ids, dY, dy_dtype, ld_dy, n_rows, d, pad_id, scale, accumulate,
                         0, nullptr, nullptr, dE, de_dtype, ld_de, ws, ws_bytes,
                         static_cast<cudaStream_t>(stream));
}

hstu_status hstu_embed_bwd_rows(int64_t n_tokens, const int64_t* ids, const void* dY,
                                int32_t dy_dtype, int64_t ld_dy, int64_t n_rows, int32_t d,
                                int64_t pad_id, float scale, int64_t* row_ids, void* rows,
                                int32_t rows_dtype, int64_t ld_rows, int64_t* n_unique, void* ws,
                                size_t ws_bytes, void* stream) {
  return hstu::embed_bwd(n_tokens, ids, dY, dy_dtype, ld_dy, n_rows, d, pad_id, scale, 0, 1,
                         row_ids, n_unique, rows, rows_dtype, ld_rows, ws, ws_bytes,
                         static_cast<cudaStream_t>(stream));
}

}  // extern "C"
