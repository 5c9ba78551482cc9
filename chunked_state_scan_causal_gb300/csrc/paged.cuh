// What the decode kernels over a paged cache share, in the tensors' own type (paged.cu) and in 8 bits (paged8.cu): the
// work split, the CUDA-core kernel of fp32 queries, and the join of an item's pieces.
#pragma once
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace linattn {
namespace {

// ------------------------------------------------------------------ work split of the decode
// A key head's rows are its query heads, each with T new tokens (paged.cu: T = 1): row r is head r / T, token r % T.
// An item is one (sequence, key head, slice of up to 16 of its rows): nt = ceil(len / 128)
// tiles of 128 tokens.  All tiles, item after item, are cut into G equal ranges, one per CTA, so
// ragged lengths balance by themselves and few long sequences are split over every SM.  A CTA that
// holds a whole item writes its output; the pieces of the other items go to the workspace, at most
// two per CTA (its first and its last item), and paged_join_kernel joins them.
constexpr int kTile = 128;
// What is not a number in the cache or in q reaches the rows that read it, as in the formula.  Maxima are taken with
// fmaxf, which drops NaN, over scores of at least kLowest where a token is there and -inf where none is: so a maximum
// of -inf says that no token is there (o = 0), and from any other one a NaN score gets a NaN weight and a score of
// -inf a weight of zero (0 / 0, NaN, if every weight is).
constexpr float kLowest = -3.402823466e+38f;

__device__ __forceinline__ int seq_len(const PagedProblem &p, int b) {
  const int64_t cap = (int64_t)p.max_blocks * p.page;
  const int n = p.seq_lens[b];
  return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n;
}
__device__ __forceinline__ int seq_tiles(const PagedProblem &p, int b) { return (seq_len(p, b) + kTile - 1) / kTile; }
// the first tile of CTA g's range, and the CTA whose range holds tile x
__device__ __forceinline__ int64_t range_lo(int64_t total, int G, int g) { return total * g / G; }
__device__ __forceinline__ int range_of(int64_t total, int G, int64_t x) { return (int)(((x + 1) * G - 1) / total); }

// Block-wide scan of the sequences' tiles: returns their sum, and `lo` is the first tile of this thread's
// sequence b0 + tid (`mine` tiles).  `buf` holds a value per warp.
template <int NT>
__device__ int64_t scan_tiles(const PagedProblem &p, int items, int b0, int64_t *buf, int64_t &lo, int64_t &mine) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, b = b0 + tid;
  mine = b < p.B ? (int64_t)seq_tiles(p, b) * items : 0;
  int64_t s = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();  // the last scan's values have been read
  if (lane == 31) buf[warp] = s;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += buf[w];
    all += buf[w];
  }
  lo = before + s - mine;
  return all;
}

constexpr int kHeads = 16;     // rows of an item
constexpr int kMaxGrid = 512;  // CTAs of a decode that paged_join_kernel joins at most

struct PagedItem {
  int b, hk, h0, nh;  // sequence, key head, first row (counted over all key heads), rows
};
// rows of a key head
__device__ __forceinline__ int group_rows(const PagedProblem &p) { return p.Hq / p.Hkv * p.T; }
// The head of row r < 2^28: the quotient by T <= 16 as a product with p.over_t = ceil(2^32 / T).
__device__ __forceinline__ int row_head(const PagedProblem &p, int r) { return p.T == 1 ? r : (int)__umulhi(r, p.over_t); }
// Where row r of sequence b lies in q and o.  (Without a division, whose branches would keep the loads of a piece's rows
// from overlapping: 200 fp32 sequences of up to 300 tokens 35.3 us, with one 37.9.)
__device__ __forceinline__ int64_t row_at(const PagedProblem &p, int b, int r) {
  const int head = row_head(p, r);
  return b * p.qsb + head * p.qsh + (r - head * p.T) * p.qst;
}
__device__ __forceinline__ PagedItem item_of(const PagedProblem &p, int slices, int b, int i) {
  PagedItem it;
  const int rows = group_rows(p), s = i % slices;
  it.b = b;
  it.hk = i / slices;
  it.h0 = it.hk * rows + s * kHeads;
  it.nh = min(kHeads, rows - s * kHeads);
  return it;
}

// The pieces of a CTA's range, in order: next() gives the item and its tiles [t0, t1).
struct PagedWalk {
  int64_t x, end, first;
  int b, slices, items;
  PagedItem it;
  int t0, t1, nt, len;
  __device__ bool next(const PagedProblem &p) {
    if (x >= end) return false;
    while (true) {
      nt = seq_tiles(p, b);
      if (nt > 0 && x < first + (int64_t)nt * items) break;
      first += (int64_t)nt * items;
      ++b;
    }
    len = seq_len(p, b);
    it = item_of(p, slices, b, (int)((x - first) / nt));
    t0 = (int)((x - first) % nt);
    t1 = (int)min((int64_t)nt, t0 + end - x);
    x += t1 - t0;
    return true;
  }
};

// This CTA's walk; false when there is nothing for it.  Called by every thread of the block; `buf` holds
// 34 values.  Up to NT sequences take one scan; more are summed first and scanned again to the range's start.
template <int NT>
__device__ bool walk_start(const PagedProblem &p, int64_t *buf, PagedWalk &w) {
  w.slices = (group_rows(p) + kHeads - 1) / kHeads;
  w.items = p.Hkv * w.slices;
  int64_t lo, mine, total = 0, base = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) total += scan_tiles<NT>(p, w.items, b0, buf, lo, mine);
  const int G = (int)min((int64_t)gridDim.x, total);  // no empty range between two pieces of an item
  if ((int)blockIdx.x >= G) return false;
  w.x = range_lo(total, G, blockIdx.x);
  w.end = range_lo(total, G, blockIdx.x + 1);
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int64_t all = p.B > NT ? scan_tiles<NT>(p, w.items, b0, buf, lo, mine) : total;
    if (mine > 0 && w.x >= base + lo && w.x < base + lo + mine) {
      buf[32] = b0 + threadIdx.x;
      buf[33] = base + lo;
    }
    base += all;
    if (w.x < base) break;
  }
  __syncthreads();
  w.b = (int)buf[32];
  w.first = buf[33];
  return true;
}

// The work split of the 8-bit cache: again all items lie one after the other and are cut into equal ranges, one per CTA.  Positions are
// 32-bit (the host bounds them) and take one division.  An item of nt tiles takes (nt << extra) + extra positions: 2 nt + 1, a
// piece's own costs being about half a tile's (256 sequences of 125 to 500 tokens: a CTA's time by its number of pieces), or
// nt where ranges are shorter than 4 (each must hold a tile).  A position u of an item stands for tile u >> extra.
struct Walk8 {
  uint32_t x, end, first, each, over;  // the next position, the range's end, the sequence's first; total / G, total % G
  int b, extra, t0, t1, nt, len;
  PagedItem it;
  __device__ uint32_t lo(uint32_t g) const { return g * each + min(g, over); }
  __device__ uint32_t holder(uint32_t at) const {  // the CTA whose range has this position
    const uint32_t split = over * (each + 1);
    return at < split ? at / (each + 1) : over + (at - split) / each;
  }
  __device__ uint32_t cost(int tiles) const { return tiles ? (uint32_t)((tiles << extra) + extra) : 0; }
  // (token numbers are 32-bit here)
  static __device__ int len_of(const PagedProblem &p, int n) { return min(max(n, 0), p.max_blocks * p.page); }
  __device__ bool next(const PagedProblem &p) {
#pragma unroll 1
    while (x < end) {
      len = len_of(p, p.seq_lens[b]);
      nt = (len + kTile - 1) / kTile;
      const uint32_t one = cost(nt), n = one * p.items;
      if (x - first >= n) {
        first += n;
        ++b;
        continue;
      }
      const uint32_t i = (x - first) / one, begin = first + i * one;
      t0 = (x - begin) >> extra;
      t1 = end - begin >= one ? nt : (end - begin) >> extra;
      last = begin + (nt << extra) - 1;
      x = min(end, begin + one);
      if (t0 >= t1) continue;  // (the range begins or ends in what the item takes beside its tiles)
      const int s = p.slices == 1 ? 0 : i % p.slices;
      it.b = b;
      it.hk = p.slices == 1 ? i : i / p.slices;
      it.h0 = it.hk * p.group + s * kHeads;
      it.nh = min(kHeads, p.group - s * kHeads);
      return true;
    }
    return false;
  }
  uint32_t last;  // the last position that stands for the item's last tile
  // By the lanes of one warp together; false when this CTA has no range.  256 sequences at a time, 8 a lane.
  __device__ bool start(const PagedProblem &p) {
    const int lane = threadIdx.x % 32;
    // the range, from all tiles and the items that have any
    auto range = [&](uint32_t all, uint32_t some) {
      const uint32_t G = min(gridDim.x, all);  // no empty range
      if (blockIdx.x >= G) return false;
      extra = 2 * all + some >= 4 * G;
      const uint32_t total = (all << extra) + extra * some;
      each = total / G;
      over = total - each * G;
      x = lo(blockIdx.x);
      end = lo(blockIdx.x + 1);
      return true;
    };
    if (p.B <= 32) {  // a sequence a lane: a third of the code, whose first fetch is what the start costs
      const int n = lane < p.B ? (len_of(p, p.seq_lens[lane]) + kTile - 1) / kTile : 0;
      if (!range(__reduce_add_sync(0xffffffffu, n) * p.items, __popc(__ballot_sync(0xffffffffu, n > 0)) * p.items)) return false;
      const uint32_t mine = cost(n) * p.items;
      first = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, first, o);
        if (lane >= o) first += y;
      }
      first -= mine;
      b = __ffs(__ballot_sync(0xffffffffu, x >= first && x < first + mine)) - 1;
      first = __shfl_sync(0xffffffffu, first, b);
      return true;
    }
    int tiles[8];
    auto load = [&](int b0) {  // tiles of this lane's sequences
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = b0 + lane * 8 + j;
        tiles[j] = at < p.B ? p.seq_lens[at] : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) tiles[j] = (len_of(p, tiles[j]) + kTile - 1) / kTile;
    };
    uint32_t all = 0, some = 0;  // tiles, items that have any
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 256) {
      load(b0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        all += tiles[j];
        some += tiles[j] > 0;
      }
    }
    if (!range(__reduce_add_sync(0xffffffffu, all) * p.items, __reduce_add_sync(0xffffffffu, some) * p.items)) return false;
    uint32_t base = 0;  // positions of the chunks before
#pragma unroll 1
    for (int b0 = 0;; b0 += 256) {
      if (p.B > 256) load(b0);
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += cost(tiles[j]) * p.items;
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t chunk = __shfl_sync(0xffffffffu, sum, 31);
      if (x < base + chunk) {  // the sequence that holds x is in this chunk: one lane has it
        b = b0 + lane * 8;
        first = base + sum - mine;
        const uint32_t who = __ballot_sync(0xffffffffu, x >= first && x < base + sum);
#pragma unroll
        for (int j = 0; j < 7; ++j) {
          const uint32_t n = cost(tiles[j]) * p.items;
          if (x < first + n) break;
          first += n;
          ++b;
        }
        const int src = __ffs(who) - 1;
        b = __shfl_sync(0xffffffffu, b, src);
        first = __shfl_sync(0xffffffffu, first, src);
        return true;
      }
      base += chunk;
    }
  }
};

// What the join has to do for the item that begins with piece w, the k-th of this CTA: see PagedProblem.
__device__ __forceinline__ void record_piece(const PagedProblem &p, const Walk8 &w, int k) {
  if (w.t0 == 0 && (p.by_item || w.t1 < w.nt))
    p.rec[p.by_item ? w.b * p.items + w.it.hk * p.slices + (w.it.h0 - w.it.hk * p.group) / kHeads : blockIdx.x] =
        w.t1 < w.nt ? make_int4(w.b, w.it.h0, w.it.nh | (k > 0) << 8, blockIdx.x | (w.holder(w.last) - blockIdx.x) << 16)
                    : make_int4(-1, 0, 0, 0);
}

// token / page, both below 2^31: with 2^(s - 1) < page <= 2^s and mul = floor(2^(31 + s) / page) + 1 the quotient is
// floor(token mul / 2^(31 + s)), since token (mul - 2^(31 + s) / page) is below 2^(31 + s) / page.
__device__ __forceinline__ int block_of(const PagedProblem &p, int token) {
  return p.page_mul ? (int)(__umulhi(token, p.page_mul) >> p.page_shift) : token;
}

// Zero rows (and records of nothing to join) for the sequences without tokens, by one warp of every CTA.
template <int D, typename T>
__device__ __noinline__ void empty_rows(const PagedProblem &p, T *o, float *lse, int lane) {
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (seq_len(p, b) == 0) {
      if (p.by_item)
#pragma unroll 1
        for (int i = lane; i < p.items; i += 32) p.rec[b * p.items + i] = make_int4(-1, 0, 0, 0);
#pragma unroll 1
      for (int r = 0; r < p.Hq * p.T; ++r) {
        if (lane < D * (int)sizeof(T) / 16) reinterpret_cast<uint4 *>(o + row_at(p, b, r))[lane] = make_uint4(0, 0, 0, 0);
        if (lse && lane == 0) lse[(int64_t)b * p.Hq * p.T + r] = -INFINITY;
      }
    }
}

// ------------------------------------------------------------------ fp32 decode (CUDA cores)
// Q8: the cache holds e4m3 codes, a scale per 16 tokens for keys and one for values, which go into the score and into
// the weight; and query t of T sees the tokens before len - T + 1 + t.
// A token's row is spread over LPT lanes, so a warp takes 32 / LPT tokens a step; every lane keeps its
// dimensions of HN query heads and of their outputs in registers (64 + 64 values at D = 128, whatever HN:
// more heads, more lanes per token) and copies its own pieces of K and V through a ring of its own, 16 KiB
// per warp, so nothing in the loop waits for another lane but the sums of a score.  Those are added up while
// the heads are halved (HN - 1 exchanges instead of HN per step), which leaves every lane one head, its
// maximum, its sum and its weight; the weights then go round.  The warps' (and lanes') maxima, sums and
// outputs are joined at a piece's end.  Up to 4 query heads per key head it is bound by the cache (105 us at 16
// sequences of 8192, 4 key heads of 4 query heads, D = 128: 0.75 of copy bandwidth), with 16 by its sums (257 us); on
// codes by its sums, shuffles and latencies (up to 8192 of them: 47 us, 0.27 of copy bandwidth).
// Four warps on two CTAs an SM leave them 255 registers: six warps, at 168, take 1.15 times as long.
constexpr int kSimtWarps = 4, kSimtThreads = 32 * kSimtWarps, kSimtPerSm = 2;
template <int D, int HN, bool Q8>
struct SimtLayout {
  static constexpr int LPT = 2 * HN < D / 4 ? 2 * HN : D / 4, TPW = 32 / LPT, NP = D / 4 / LPT;
  static constexpr int depth = !Q8 ? 16 / NP : NP > 1 ? 64 / NP : 32;  // at most 32: a bit each says that the token is there
  static constexpr size_t ring = (size_t)kSimtWarps * depth * 2 * NP * 32 * (Q8 ? 4 : 16);
  static constexpr size_t smem = ring + (Q8 ? (size_t)kSimtWarps * depth * 32 * sizeof(float2) : 0);
  static_assert(smem >= (size_t)kSimtWarps * HN * D * sizeof(float), "the ring holds the warps' outputs at the end");
};

// 16 bytes, or zeros when !there (src is not read then)
__device__ __forceinline__ void cp_async16_zfill(void *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

// the same of 4 and 8 bytes too
template <typename T>
__device__ __forceinline__ void cp_async_zfill(T *dst, const void *src, bool there) {
  if constexpr (sizeof(T) == 16)
    cp_async16_zfill(dst, src, there);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? (int)sizeof(T) : 0), "n"(sizeof(T))
                 : "memory");
}
// two e4m3 codes (the low 16 bits) as two f16
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}
// four values of a row
__device__ __forceinline__ float4 four_of(float4 x) { return x; }
__device__ __forceinline__ float4 four_of(uint32_t c) {
  const uint32_t a = f16x2_of_e4m3x2(c), b = f16x2_of_e4m3x2(c >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a)), y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
  return make_float4(x.x, x.y, y.x, y.y);
}
template <bool Q8>
struct SimtPiece {
  using cache = float;
  using walk = PagedWalk;
};
template <>
struct SimtPiece<true> {
  using cache = uint8_t;
  using walk = Walk8;
};
// Q8: the codes of a lane's 4 NP dimensions, which lie side by side
template <int NP>
struct SimtCodes {
  using type = uint32_t;
};
template <>
struct SimtCodes<2> {
  using type = uint2;
};
template <>
struct SimtCodes<4> {
  using type = uint4;
};

// The sums over lanes of 2 N heads: lanes with bit X take over the upper N of them, and so on.
template <int N, int X>
__device__ __forceinline__ void halve_heads(float *s, int lane) {
  if constexpr (N > 0) {
    const bool up = lane & X;
#pragma unroll
    for (int h = 0; h < N; ++h)
      s[h] = (up ? s[h + N] : s[h]) + __shfl_xor_sync(0xffffffffu, up ? s[h] : s[h + N], X);
    halve_heads<N / 2, X / 2>(s, lane);
  }
}

template <int D, int HN, bool Q8>
__global__ void __launch_bounds__(kSimtThreads, kSimtPerSm)
    paged_decode_simt(PagedProblem p, const float *q, const typename SimtPiece<Q8>::cache *kc,
                      const typename SimtPiece<Q8>::cache *vc, float *o, float *lse, float *part, float *ml) {
  using L = SimtLayout<D, HN, Q8>;
  constexpr int LPT = L::LPT, NP = L::NP, S = L::depth, kStep = kSimtWarps * L::TPW;
  // steps committed together; steps computed together, whose sums and shuffles overlap (16 sequences of up to 8192 tokens,
  // 4 key heads of 4 query heads: one 55.8, two 51.4, four 48.9 us)
  constexpr int U = S >= 16 ? 4 : S / 4, P = Q8 ? 4 : 1;
  static_assert(S % U == 0 && U % P == 0 && S >= 4, "whole groups");
  extern __shared__ float4 smem4[];
  __shared__ int64_t buf[34];
  __shared__ float sm[kSimtWarps][HN], sl[kSimtWarps][HN];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, sub = lane / LPT, g = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  typename SimtPiece<Q8>::walk w;
  int *status = p.status, pieces = 0;
  if constexpr (Q8) {  // every warp walks for itself; a status word per CTA
    status = p.errors + blockIdx.x;
    if (tid == 0) {
      *status = 0;
      if (!p.by_item) p.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    if (warp == 0) empty_rows<D>(p, o, lse, lane);
    if (!w.start(p)) return;
  } else {
    if (!walk_start<kSimtThreads>(p, buf, w)) return;
  }
  const float c = p.scale * 1.4426950408889634f;
  const int mine = lane % LPT / (LPT / HN), home = lane & ~(LPT - 1);
  // [slot][k, v][piece of four values], Q8 [slot][k, v], a lane's own column
  using Codes = typename SimtCodes<NP>::type;
  float4 *ring = smem4 + warp * (S * 2 * NP * 32) + lane;
  Codes *cring = reinterpret_cast<Codes *>(smem4) + warp * (S * 2 * 32) + lane;
  // the lane's j-th four dimensions (in fours)
  auto four = [&](int j) { return Q8 ? lane % LPT * NP + j : j * LPT + lane % LPT; };
  float2 *sring = reinterpret_cast<float2 *>(reinterpret_cast<char *>(smem4) + L::ring) + warp * (S * 32) + lane;
  const int hop = block_of(p, kStep), rest = kStep - hop * p.page;  // of a step
  int slot = 0;
  while (w.next(p)) {
    const PagedItem it = w.it;
    if constexpr (Q8)
      if (tid == 0) record_piece(p, w, pieces);
    ++pieces;
    const int b = w.b, end = min(w.t1 * kTile, w.len), first = w.t0 * kTile + warp * L::TPW + sub;
    const int steps = ((end - w.t0 * kTile + kStep - 1) / kStep + P - 1) / P * P;
    const int *table = p.table + (int64_t)b * p.tstride;
    float4 qr[HN][NP], acc[HN][NP];
    float m = -INFINITY, l = 0.f;  // of head `mine`
#pragma unroll
    for (int h = 0; h < HN; ++h) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        acc[h][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        qr[h][j] = acc[h][j];
        if (h < it.nh) {
          const float4 x = *reinterpret_cast<const float4 *>(q + row_at(p, b, it.h0 + h) + 4 * four(j));
          qr[h][j] = make_float4(x.x * c, x.y * c, x.z * c, x.w * c);
        }
      }
    }
    // Q8: the first token that row `r` of the item does not see, and the first that not every row sees
    auto limit = [&](int r) { return w.len - p.T + 1 + it.h0 + r - row_head(p, it.h0 + r) * p.T; };
    const int my_limit = Q8 ? limit(mine) : 0, partly = w.len - p.T + 1;
    // acc[h] times the factor that head h's lane holds
    auto rescale = [&](float f) {
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        const float fh = __shfl_sync(0xffffffffu, f, home + h * (LPT / HN));
#pragma unroll
        for (int j = 0; j < NP; ++j)
          acc[h][j] = make_float4(acc[h][j].x * fh, acc[h][j].y * fh, acc[h][j].z * fh, acc[h][j].w * fh);
      }
    };
    // Step i: this lane's token is first + i kStep.  Of the next step to be copied: the token, its page's place in the
    // table, the slot, and the page's id, which is read a step before the copies that use it.  (By additions: the divisions of a
    // step, one after the other, took most of a short sequence's copies.)
    int next = first, block = block_of(p, first), at = first - block * p.page, id = next < end ? table[block] : 0;
    uint32_t ok = 0;  // bit per slot: the token is there
    auto copy = [&](int i) {
      if (i < steps) {
        const int z = i % S;
        bool there = next < end;
        if (there && (id < 0 || id >= p.pages)) {
          if (lane % LPT == 0) report_error(status, -1);
          there = false;
        }
        const int64_t from = there ? id * p.csb + it.hk * p.csh + at * p.cst + 4 * four(0) : 0;
        ok = there ? ok | (1u << z) : ok & ~(1u << z);
        if constexpr (Q8) {
          cp_async_zfill(cring + z * 2 * 32, kc + from, there);
          cp_async_zfill(cring + (z * 2 + 1) * 32, vc + from, there);
          cp_async_zfill(sring + z * 32,
                         p.scales + (there ? id * p.ssb + it.hk * p.ssh + at / kScaleTokens * 2 : 0), there);
        } else {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            cp_async_zfill(ring + ((z * 2) * NP + j) * 32, kc + from + 4 * LPT * j, there);
            cp_async_zfill(ring + ((z * 2 + 1) * NP + j) * 32, vc + from + 4 * LPT * j, there);
          }
        }
        next += kStep;
        block += hop;
        at += rest;
        if (at >= p.page) {
          at -= p.page;
          ++block;
        }
        id = next < end ? table[block] : 0;
      }
    };
    // the lane's dimensions of step i's key (0) or value (1)
    auto row_of = [&](int i, int kv, float4 (&x)[NP]) {
      if constexpr (Q8) {
        const Codes c = cring[(i % S * 2 + kv) * 32];
#pragma unroll
        for (int j = 0; j < NP; ++j) x[j] = four_of(reinterpret_cast<const uint32_t *>(&c)[j]);
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) x[j] = ring[((i % S * 2 + kv) * NP + j) * 32];
      }
    };
    // Copies are committed by groups of U steps (a commit is 140 cycles), 4 or more groups to the ring; when there are no
    // more to issue all are waited for (with groups of one step: the step's own, by empty groups behind it).
    auto copies = [&](int i0) {
#pragma unroll 1
      for (int i = i0; i < i0 + U; ++i) copy(i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < S - U && (U == 1 || i < steps); i += U) copies(i);
#pragma unroll 1
    for (int i = 0; i < steps; i += P) {
      if (i % U == 0) {
        if (U == 1 || i + S - U < steps) {
          copies(i + S - U);
          asm volatile("cp.async.wait_group %0;" ::"n"(S / U - 1) : "memory");
        } else {
          asm volatile("cp.async.wait_all;" ::: "memory");
        }
      }
      float s[P][HN];
#pragma unroll
      for (int y = 0; y < P; ++y) {
        float4 x[NP];
        row_of(i + y, 0, x);
#pragma unroll
        for (int h = 0; h < HN; ++h) s[y][h] = 0.f;
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int h = 0; h < HN; ++h)
            s[y][h] = fmaf(x[j].x, qr[h][j].x,
                           fmaf(x[j].y, qr[h][j].y, fmaf(x[j].z, qr[h][j].z, fmaf(x[j].w, qr[h][j].w, s[y][h]))));
      }
      float2 sc[P];
      float score[P], top = -INFINITY;
#pragma unroll
      for (int y = 0; y < P; ++y) {
        halve_heads<HN / 2, LPT / 2>(s[y], lane);
#pragma unroll
        for (int x = LPT / HN / 2; x; x /= 2) s[y][0] += __shfl_xor_sync(0xffffffffu, s[y][0], x);
        sc[y] = make_float2(1.f, 1.f);
        if constexpr (Q8) {
          sc[y] = sring[((i + y) % S) * 32];
          s[y][0] *= sc[y].x;
        }
        const bool there = ((ok >> ((i + y) % S)) & 1) && (!Q8 || first + (i + y) * kStep < my_limit);
        score[y] = there ? s[y][0] : -INFINITY;
        top = fmaxf(top, there ? fmaxf(score[y], kLowest) : -INFINITY);
      }
      if (__any_sync(0xffffffffu, top > m)) {  // rare once the first steps have passed
        const float mn = fmaxf(m, top), f = exp2f(m - (mn == -INFINITY ? 0.f : mn));
        m = mn;
        l *= f;
        rescale(f);
      }
#pragma unroll
      for (int y = 0; y < P; ++y) {
        const int n = first + (i + y) * kStep;
        const float weight = exp2f(score[y] - (m == -INFINITY ? 0.f : m));
        l += weight;
#pragma unroll
        for (int h = 0; h < HN; ++h) s[y][h] = __shfl_sync(0xffffffffu, weight, home + h * (LPT / HN)) * sc[y].y;
        float4 x[NP];
        row_of(i + y, 1, x);
        auto add = [&](int h) {
#pragma unroll
          for (int j = 0; j < NP; ++j)
            acc[h][j] = make_float4(fmaf(s[y][h], x[j].x, acc[h][j].x), fmaf(s[y][h], x[j].y, acc[h][j].y),
                                    fmaf(s[y][h], x[j].z, acc[h][j].z), fmaf(s[y][h], x[j].w, acc[h][j].w));
        };
        if (Q8 && n >= partly) {
          // a row that does not see this token takes nothing of it, NaN neither
#pragma unroll
          for (int h = 0; h < HN; ++h)
            if (n < limit(h)) add(h);
        } else {
#pragma unroll
          for (int h = 0; h < HN; ++h) add(h);
        }
      }
    }
    // the lanes of different tokens joined, then the warps
    float mn = m;
#pragma unroll
    for (int x = LPT; x < 32; x *= 2) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    const float f = exp2f(m - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l *= f;
    rescale(f);
#pragma unroll
    for (int x = LPT; x < 32; x *= 2) {
      l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
      for (int h = 0; h < HN; ++h)
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          acc[h][j].x += __shfl_xor_sync(0xffffffffu, acc[h][j].x, x);
          acc[h][j].y += __shfl_xor_sync(0xffffffffu, acc[h][j].y, x);
          acc[h][j].z += __shfl_xor_sync(0xffffffffu, acc[h][j].z, x);
          acc[h][j].w += __shfl_xor_sync(0xffffffffu, acc[h][j].w, x);
        }
    }
    __syncthreads();  // every warp has left its ring
    if (sub == 0) {
#pragma unroll
      for (int h = 0; h < HN; ++h)
#pragma unroll
        for (int j = 0; j < NP; ++j) smem4[(warp * HN + h) * (D / 4) + four(j)] = acc[h][j];
      sm[warp][mine] = m;
      sl[warp][mine] = l;
    }
    __syncthreads();
    const bool whole = w.t0 == 0 && w.t1 == w.nt;
    for (int e = tid; e < it.nh * D; e += kSimtThreads) {
      const int h = e / D, dim = e % D;
      float mx = -INFINITY, a = 0.f, sum = 0.f;
#pragma unroll
      for (int x = 0; x < kSimtWarps; ++x) mx = fmaxf(mx, sm[x][h]);
#pragma unroll
      for (int x = 0; x < kSimtWarps; ++x) {
        const float f = exp2f(sm[x][h] - (mx == -INFINITY ? 0.f : mx));
        a = fmaf(f, reinterpret_cast<const float *>(smem4)[(x * HN + h) * D + dim], a);
        sum = fmaf(f, sl[x][h], sum);
      }
      const int64_t piece = (int64_t)(2 * g + slot) * (Q8 ? HN : kHeads) + h;
      if (whole) {
        o[row_at(p, b, it.h0 + h) + dim] = mx == -INFINITY ? 0.f : a / sum;
        if (lse && dim == 0) lse[(int64_t)b * p.Hq * p.T + it.h0 + h] = (mx + log2f(sum)) * 0.6931471805599453f;
      } else {
        part[piece * D + dim] = a;
        if (dim == 0) {
          ml[piece * 2] = mx;
          ml[piece * 2 + 1] = sum;
        }
      }
    }
    slot = 1;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ join
// One CTA of D threads per (sequence, row): joins the pieces of an item that was cut,
// o = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i, and writes the rows of empty sequences
// (o = 0, lse = -inf).  A piece sits in its CTA's slot 1 when that CTA's range began in an earlier
// item, else in slot 0.  Bound by finding its item (7 us for 2048 rows, largely behind the decode's own end).
template <int D, typename T>
__global__ void __launch_bounds__(D) paged_join_kernel(PagedProblem p, int grid, T *o, float *lse, const float *part,
                                                       const float *ml) {
  __shared__ int64_t buf[2 * D / 32 + 2];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, tid = threadIdx.x;  // (T = 1)
  griddep_wait();
  const int group = p.Hq / p.Hkv, slices = (group + kHeads - 1) / kHeads, items = p.Hkv * slices;
  const int64_t orow = b * p.qsb + h * p.qsh + tid;
  const int nt = seq_tiles(p, b);
  if (nt == 0) {
    o[orow] = (T)0.f;
    if (lse && tid == 0) lse[(int64_t)b * p.Hq + h] = -INFINITY;
    return;
  }
  int64_t before = 0, all = 0;
  for (int i = tid; i < p.B; i += D) {
    const int64_t n = (int64_t)seq_tiles(p, i) * items;
    all += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int w = 16; w; w /= 2) {
    before += __shfl_xor_sync(0xffffffffu, before, w);
    all += __shfl_xor_sync(0xffffffffu, all, w);
  }
  if (tid % 32 == 0) {
    buf[tid / 32] = before;
    buf[D / 32 + tid / 32] = all;
  }
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < D / 32; ++w) {
    before += buf[w];
    all += buf[D / 32 + w];
  }
  const int G = (int)min((int64_t)grid, all);
  const int s = (h % group) / kHeads, hh = (h % group) % kHeads;
  const int64_t lo = before + (int64_t)((h / group) * slices + s) * nt, hi = lo + nt;
  const int g0 = range_of(all, G, lo), g1 = range_of(all, G, hi - 1);
  if (g0 == g1) return;  // one CTA held the whole item and has written it
  // the first piece may be the last of its CTA's range (slot 1); the others begin theirs (slot 0)
  const int first = range_lo(all, G, g0) < lo;
  auto at = [&](int g) { return (int64_t)(2 * g + (g == g0 ? first : 0)) * kHeads + hh; };
  __shared__ float s_f[2 * kMaxGrid], s_w[D / 32];
  float m = -INFINITY;
  for (int g = g0 + tid; g <= g1; g += D) {
    const float2 v = *reinterpret_cast<const float2 *>(ml + at(g) * 2);
    s_f[2 * (g - g0)] = v.x;
    s_f[2 * (g - g0) + 1] = v.y;
    m = fmaxf(m, v.x);
  }
#pragma unroll
  for (int w = 16; w; w /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  if (tid % 32 == 0) s_w[tid / 32] = m;
  __syncthreads();
  for (int w = 0; w < D / 32; ++w) m = fmaxf(m, s_w[w]);
  const float use = m == -INFINITY ? 0.f : m;
  float a = 0.f, l = 0.f;
#pragma unroll 8
  for (int g = g0; g <= g1; ++g) {
    const float f = exp2f(s_f[2 * (g - g0)] - use);
    a = fmaf(f, part[at(g) * D + tid], a);
    l = fmaf(f, s_f[2 * (g - g0) + 1], l);
  }
  o[orow] = (T)(m == -INFINITY ? 0.f : a / l);
  if (lse && tid == 0) lse[(int64_t)b * p.Hq + h] = (m + log2f(l)) * 0.6931471805599453f;
}

// CTAs: `per` on each SM, fewer when even the longest possible sequences have fewer tiles.
int paged_grid(const PagedProblem &p, int per) {
  const int64_t slices = (p.Hq / p.Hkv * p.T + kHeads - 1) / kHeads;
  const int64_t tiles = ((int64_t)p.max_blocks * p.page + kTile - 1) / kTile;
  const int64_t most = tiles * p.B * p.Hkv * slices, want = (int64_t)p.num_sms * per;
  return (int)(most < want ? most : want);
}

template <int D, typename T, typename Launch>
cudaError_t run_decode(Launch launch, int per, const PagedProblem &p, void *o, float *lse, void *ws, cudaStream_t s) {
  const int all = paged_grid(p, per), G = all < kMaxGrid ? all : kMaxGrid;
  float *part = static_cast<float *>(ws), *ml = part + (size_t)2 * (2 * p.num_sms) * kHeads * D;
  {
    TimedLaunch t(K_PAGED_DECODE, s);
    cudaError_t e = launch(G, part, ml);
    if (e != cudaSuccess) return e;
  }
  TimedLaunch t(K_PAGED_JOIN, s);
  return launch_overlapped(paged_join_kernel<D, T>, dim3(p.B * p.Hq), dim3(D), 0, s, p, G, (T *)o, lse,
                           (const float *)part, (const float *)ml);
}

}  // namespace
}  // namespace linattn
