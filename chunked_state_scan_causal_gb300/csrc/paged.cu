// Softmax attention over a paged key-value cache: the serving form of the hybrid's softmax layers.
//
// The cache is a set of pages of `page` tokens, [pages, Hkv, page, d] with any strides; sequence b's
// token n lives in page block_table[b][n / page], slot n % page.  paged_append copies new keys and
// values into their slots; paged_decode attends with one query per sequence,
//     o[b,h] = sum_n softmax_n(scale q[b,h] . k_n) v_n   over n < seq_lens[b],
// query head h reading key head h / (Hq / Hkv).
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace linattn {
namespace {

// ------------------------------------------------------------------ append
// One thread per 16 bytes of a row of k and of v: a copy, bound by its bytes (8 prompts of 4096 tokens, 8 key heads:
// 40.7 us, 0.97 of copy bandwidth; or, for one token per sequence, by the launch).  Rows past new_lens, outside the table or with a page id outside the
// cache are left unwritten; the latter two are recorded in the status word.
__global__ void __launch_bounds__(256) paged_append_kernel(PagedProblem p, const char *k, const char *v, char *kc,
                                                           char *vc, uint32_t T, const int *start, const int *new_lens,
                                                           int64_t sb, int64_t sh, int64_t st, int shift,
                                                           uint32_t rows, int *status) {
  const uint32_t row = blockIdx.x * (256u >> shift) + (threadIdx.x >> shift), c = threadIdx.x & ((1u << shift) - 1);
  if (row >= rows) return;
  const uint32_t r = row / T, t = row % T, b = r / (uint32_t)p.Hkv, h = r % (uint32_t)p.Hkv;
  if (new_lens && (int)t >= new_lens[b]) return;
  const int first = start[b];
  const int64_t pos = (int64_t)first + t;
  if (first < 0 || pos >= (int64_t)p.max_blocks * p.page) {
    report_error(status, -1);
    return;
  }
  const uint32_t block = (uint32_t)pos / (uint32_t)p.page, slot = (uint32_t)pos % (uint32_t)p.page;
  const int id = p.table[(int64_t)b * p.tstride + block];
  if (id < 0 || id >= p.pages) {
    report_error(status, -1);
    return;
  }
  const int64_t src = (b * sb + h * sh + t * st) * p.esz + 16 * c;
  const int64_t dst = (id * p.csb + h * p.csh + slot * p.cst) * p.esz + 16 * c;
  const uint4 x = *reinterpret_cast<const uint4 *>(k + src), y = *reinterpret_cast<const uint4 *>(v + src);
  *reinterpret_cast<uint4 *>(kc + dst) = x;
  *reinterpret_cast<uint4 *>(vc + dst) = y;
}

// ------------------------------------------------------------------ work split of the decode
// An item is one (sequence, key head, slice of up to 16 of its query heads): nt = ceil(len / 128)
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

constexpr int kHeads = 16;    // query heads of an item
constexpr int kMaxGrid = 512;  // CTAs of a decode at most

struct PagedItem {
  int b, hk, h0, nh;  // sequence, key head, first query head, query heads
};
__device__ __forceinline__ PagedItem item_of(const PagedProblem &p, int slices, int b, int i) {
  PagedItem it;
  const int group = p.Hq / p.Hkv, s = i % slices;
  it.b = b;
  it.hk = i / slices;
  it.h0 = it.hk * group + s * kHeads;
  it.nh = min(kHeads, group - s * kHeads);
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
  w.slices = (p.Hq / p.Hkv + kHeads - 1) / kHeads;
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

// ------------------------------------------------------------------ bf16 decode (tensor cores)
// Per tile of 128 tokens, with lane = token and column = query head,
//     S = K Q^T,   p = 2^(c S - m),   O^T += V^T p^T   (lane = value dimension, column = query head):
// K and V are the 128-row A operands straight from shared memory, and the (at most 16) query heads the
// narrow side, so a tile costs 16 small products whatever the number of heads (each bound by reading its
// 128-row operand), and the kernel is bound by reading the cache once.  The softmax threads' work does grow with the
// heads: 64 sequences of up to 16384 tokens run at 1.04 of copy bandwidth with 1 or 4 query heads a key head (8 key
// heads), 1.01 with 8, 0.88 with 16 (4 key heads); more than 16 read the cache once per 16.  p enters as two bf16 parts side by
// side (columns 0..15 and 16..31 of O), so the weights keep 16 bits at no extra product.  The reference maximum m
// moves only when a tile exceeds it by more than 8 (in log2): p stays below 2^8 and O is rescaled rarely.
// Even and odd tiles are two streams with an m, a sum and an O of their own, joined at the piece's end, so
// the softmax of one tile overlaps the products of the next.
// With many short sequences a piece's latencies count (about 4.5 us a piece of three tiles): the next piece's Q is
// loaded and its first scores are made while this one's output goes out (256 sequences of 125 to 500 tokens, 8 key
// heads: 101 -> 93 us, 93 to 95 by the card, 0.50 of copy bandwidth; long sequences run at it).
// Warps: 0..3 and 4..7 softmax and output of the even and odd tiles, 8 issues the products, 9..12 load.
// Pages of a multiple of 8 tokens are loaded by tensor-map copies of up to 128 rows (one lane per copy);
// other pages by 16-byte asynchronous copies of all four warps, which are slower (a warp moves 512 bytes an
// instruction: 1.1 ms instead of 0.37 at 64 sequences of 16K).  Either way the softmax threads clear the
// value rows of absent tokens: a slot past the length may hold NaN, and 0 x NaN is NaN.
constexpr int kTcThreads = 416, kLoadWarps = 4;
template <int D>
struct TcLayout {
  static constexpr int ring = D == 128 ? 6 : 12;
  static constexpr uint32_t tile = 128 * D * 2, q = ring * tile, p = q + kHeads * D * 2,  // P: two buffers of 32 rows (hi, lo)
      x = p + 2 * 2 * 4096, end = x + kHeads * D * 4;  // X: the odd stream's O on its way to the even one's threads
  static constexpr size_t smem = end + 1024;
};
// Barriers; S, P and O have one per buffer (even and odd tiles), since a role may run a tile ahead of another.
// The ring's full and empty barriers follow.
enum { T_Q = 0, T_OFREE, T_S, T_P = T_S + 2, T_O = T_P + 2, T_FULL = T_O + 2 };

__device__ __forceinline__ void st_shared_h(uint32_t addr, float x) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(__float2bfloat16_rn(x))) : "memory");
}
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

// box: rows of a tensor-map copy (0: none, the pages have another size).
// HN: query heads handled by the softmax threads (4, 8 or 16; the products are always 16 wide)
template <int D, int HN>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_decode_tc(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, int box,
                    PagedProblem p, const __nv_bfloat16 *q, const __nv_bfloat16 *kc, const __nv_bfloat16 *vc,
                    __nv_bfloat16 *o, float *lse, float *part, float *ml) {
  using L = TcLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t buf[34];
  constexpr int kRing = L::ring, T_EMPTY = T_FULL + kRing;
  __shared__ uint64_t bar[T_EMPTY + kRing];
  __shared__ uint32_t tslot;
  __shared__ int abort_flag;
  __shared__ __align__(16) float s_red[2][HN][4];
  __shared__ float s_m[HN], s_l[HN];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const uint32_t base = smem_u32(smem);
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar[T_FULL + i], box ? 1 : kLoadWarps * 32);
      mbar_init(&bar[T_EMPTY + i], 1);
    }
    mbar_init(&bar[T_Q], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[T_S + i], 1);
      mbar_init(&bar[T_P + i], 4);
      mbar_init(&bar[T_O + i], 1);
    }
    mbar_init(&bar[T_OFREE], 8);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&tslot, 128);
    tmem_relinquish();
  }
  // the P rows of heads that no thread writes
  for (int i = tid; i < 4 * 4096 / 16; i += kTcThreads) st_shared_v4(base + L::p + 16 * i, 0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tslot, 0);  // S of the even and odd tiles: columns 0, 16; their O^T: 32, 64
  griddep_wait();
  griddep_launch_dependents();
  PagedWalk w;
  const bool any = walk_start<kTcThreads>(p, buf, w);
  auto wait = [&](int i, int parity) {
    return __all_sync(0xffffffffu, mbar_wait(&bar[i], parity & 1, &abort_flag, p.status));
  };
  auto wait2 = [&](int which, int tile) { return wait(which + (tile & 1), tile >> 1); };
  if (!any) {
  } else if (warp >= 9) {
    // ------------------------------------------------------------ loads
    int n = 0;
    bool ok = true;
    if (box && warp == 9) {
      // lane x < 128 / box: rows x box .. of every tile
      const int boxes = kTile / box;
      while (ok && w.next(p)) {
        const int *row = p.table + (int64_t)w.b * p.tstride;
        auto fetch = [&](int t) {
          const int tok = t * kTile + lane * box;
          return lane < boxes && tok < w.len ? row[tok / p.page] : -1;
        };
        int next = fetch(w.t0);
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          const int id = next, tok = t * kTile + lane * box;
          const bool in = id >= 0 && id < p.pages;
          if (!in && lane < boxes && tok < w.len) report_error(p.status, -1);
          next = t + 1 < w.t1 ? fetch(t + 1) : -1;
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, in)) * box * D * 2;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int s = n % kRing;
            if (n >= kRing && !(ok = wait(T_EMPTY + s, n / kRing - 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar[T_FULL + s], bytes);
            __syncwarp();
            if (in)
#pragma unroll
              for (int x = 0; x < D / 64; ++x)
                tma_load_4d(kv ? &mv : &mk, &bar[T_FULL + s], smem + s * L::tile + x * 16384 + lane * box * 128, 64 * x,
                            tok % p.page, w.it.hk, id, kPolicyEvictFirst);
          }
        }
      }
      // what is in flight lands before the block ends (a wait with a limit, also after an abort)
      volatile int no_abort = 0;
      for (int s = 0; s < kRing; ++s) {
        const int uses = n > s ? (n - 1 - s) / kRing + 1 : 0;
        if (uses && lane == 0) mbar_wait(&bar[T_FULL + s], (uses - 1) & 1, &no_abort, p.status);
      }
      __syncwarp();
    } else if (!box) {
      const int lt = tid - 288, c = lt % (D / 8), r0 = lt / (D / 8);
      constexpr int kRows = kLoadWarps * 32 / (D / 8), kIter = kTile / kRows;
      while (ok && w.next(p)) {
        const int *row = p.table + (int64_t)w.b * p.tstride;
        const int64_t head = w.it.hk * p.csh + 8 * c;
        // the page ids of this thread's rows of a tile, fetched a tile ahead (-1: past the length)
        int ids[kIter];
        auto fetch = [&](int t) {
#pragma unroll
          for (int j = 0; j < kIter; ++j) {
            const int tok = t * kTile + r0 + j * kRows;
            ids[j] = tok < w.len ? row[tok / p.page] : -1;
          }
        };
        fetch(w.t0);
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          int64_t off[kIter];
#pragma unroll
          for (int j = 0; j < kIter; ++j) {
            const int tok = t * kTile + r0 + j * kRows, id = ids[j];
            const bool good = id >= 0 && id < p.pages;
            if (!good && tok < w.len) report_error(p.status, -1);
            off[j] = good ? id * p.csb + (tok % p.page) * p.cst + head : -1;
          }
          if (t + 1 < w.t1) fetch(t + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int s = n % kRing;
            if (n >= kRing && !(ok = wait(T_EMPTY + s, n / kRing - 1))) break;
            const uint32_t dst = base + s * L::tile + (c >> 3) * 16384;
            const __nv_bfloat16 *src = kv ? vc : kc;
#pragma unroll
            for (int j = 0; j < kIter; ++j)
              if (off[j] >= 0) cp_async16(dst + swz(r0 + j * kRows, c & 7), src + off[j]);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&bar[T_FULL + s])) : "memory");
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ products
    const uint32_t id_qk = idesc_bf16(128, 16, false, false), id_pv = idesc_bf16(128, 32, true, false);
    int i = 0, seg = 0;  // tiles whose S is issued; pieces
    bool ok = true;
    auto qk = [&](int t) {
      const int s = (2 * t) % kRing;
      if (!wait(T_FULL + s, 2 * t / kRing)) return false;
      if (!box) fence_proxy_async_smem();  // the tile came by ordinary (asynchronous) copies
      tc_fence_after();
#pragma unroll
      for (uint32_t ks = 0; ks < D / 16; ++ks)
        mma_ss_warp(tmem + (t & 1) * 16, desc_kmajor(base + s * L::tile, ks), desc_kmajor_h(base + L::q, ks, 2048), id_qk,
                    ks > 0);
      mma_commit_warp(&bar[T_S + (t & 1)]);
      mma_commit_warp(&bar[T_EMPTY + s]);
      return true;
    };
    for (; ok && w.next(p); ++seg) {
      if (!(ok = wait(T_Q, seg))) break;  // Q of this piece is in place (and S of the last one read)
      tc_fence_after();
      const int n = w.t1 - w.t0;
      if (!(ok = qk(i))) break;
      for (int t = 0; t < n && ok; ++t, ++i) {
        if (t + 1 < n && !(ok = qk(i + 1))) break;
        const int s = (2 * i + 1) % kRing;
        if (!(ok = wait(T_FULL + s, (2 * i + 1) / kRing) && wait2(T_P, i) && (t > 1 || seg == 0 || wait(T_OFREE, seg - 1))))
          break;
        if (!box) fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t P = base + L::p + (i & 1) * 8192;
#pragma unroll
        for (uint32_t ks = 0; ks < 8; ++ks)
          mma_ss_warp(tmem + 32 + (i & 1) * 32, desc_mnmajor(base + s * L::tile, ks), desc_kmajor_h(P, ks, 4096), id_pv,
                      t > 1 || ks > 0);
        mma_commit_warp(&bar[T_O + (i & 1)]);
        mma_commit_warp(&bar[T_EMPTY + s]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and output: lane = token, then
    // lane = value dimension
    const int gr = warp >> 2;  // stream: tiles i with i % 2 == gr
    const uint32_t lt = tid & 127, t4 = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = p.scale * 1.4426950408889634f;
    int i0 = 0, slot = 0;  // tiles of the pieces before
    bool ok = true;
    // the warp's reductions of HN values over its lanes: the heads are halved over the lanes, so a lane ends
    // with one head's value; then the four warps' values meet in s_red
    auto reduce = [&](float (&y)[HN], auto op) {
      int h0 = 0, off = 16;
#pragma unroll
      for (int z = HN / 2; z >= 1; z /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int h = 0; h < z; ++h) {
          const float send = up ? y[h] : y[h + z], keep = up ? y[h + z] : y[h];
          y[h] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
        h0 += up ? z : 0;
      }
      for (; off >= 1; off /= 2) y[0] = op(y[0], __shfl_xor_sync(0xffffffffu, y[0], off));
      if (lane % (32 / HN) == 0) s_red[gr][h0][warp & 3] = y[0];
    };
    PagedWalk ahead = w;  // the piece after this one
    bool more = ahead.next(p);
    auto load_q = [&] {
      for (int e = tid; e < kHeads * D / 8; e += 256) {
        const int h = e / (D / 8), x = e % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (h < ahead.it.nh)
          v = *reinterpret_cast<const uint4 *>(q + ahead.b * p.qsb + (ahead.it.h0 + h) * p.qsh + 8 * x);
        st_shared_v4(base + L::q + (x >> 3) * 2048 + swz(h, x & 7), v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[T_Q]);
    };
    if (more) load_q();
    while (ok && more) {
      w = ahead;
      float m[HN], l[HN];
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
      }
      const int n = w.t1 - w.t0;
      const int *row = p.table + (int64_t)w.b * p.tstride;
      // this lane's token of a tile: its page id, fetched a tile of the stream ahead (-1: past the length)
      auto fetch = [&](int t) {
        const int tok = (w.t0 + t) * kTile + lt;
        return t < n && tok < w.len ? row[tok / p.page] : -1;
      };
      const int tf = (gr ^ i0) & 1;  // the stream's first tile of the piece
      int id = fetch(tf), last = -1;
      for (int t = tf; t < n; t += 2) {
        const int i = i0 + t;
        const bool valid = id >= 0 && id < p.pages;
        id = fetch(t + 2);
        last = i;
        ok = wait2(T_S, i);
        // P of the stream's tile before has been read; its product into O is done
        if (i >= 2) ok = wait2(T_O, i - 2) && ok;
        // one verdict for the four warps: they share the barriers below
        if (!(ok = group_all(ok, 1 + gr, 128))) break;
        tc_fence_after();
        uint32_t r[16];
        tmem_ld16(t4 + gr * 16, r);
        tmem_ld_wait();
        tc_fence_before();
        float x[HN], y[HN];
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          x[h] = valid ? __uint_as_float(r[h]) * c : -INFINITY;
          y[h] = valid ? fmaxf(x[h], kLowest) : -INFINITY;
        }
        reduce(y, [](float u, float v) { return fmaxf(u, v); });
        named_bar_sync(1 + gr, 128);
        bool move = false;
        float f[HN];
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float4 v = *reinterpret_cast<const float4 *>(s_red[gr][h]);
          const float mx = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
          f[h] = 1.f;
          if (mx > m[h] + 8.f) {  // (also the first token: m is -inf)
            f[h] = ex2(m[h] - mx);
            m[h] = mx;
            move = true;
          }
        }
        if (move) {
          if (t > tf) {  // O (lane = value dimension) to the new references
            tc_fence_after();
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a[16];
              tmem_ld16(t4 + 32 + gr * 32 + 16 * y, a);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < HN; ++h) a[h] = __float_as_uint(__uint_as_float(a[h]) * f[h]);
              tmem_st16(t4 + 32 + gr * 32 + 16 * y, a);
            }
            tmem_st_wait();
            tc_fence_before();
          }
#pragma unroll
          for (int h = 0; h < HN; ++h) l[h] *= f[h];
        }
        const uint32_t P = base + L::p + gr * 8192 + (lt >> 6) * 4096 + (lt & 7) * 2;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float e = m[h] == -INFINITY ? 0.f : ex2(x[h] - m[h]);
          l[h] += e;
          const uint32_t at = P + swz(h, (lt & 63) >> 3);
          st_shared_h(at, e);
          st_shared_h(at + 2048, e - __bfloat162float(__float2bfloat16_rn(e)));
        }
        if (!__all_sync(0xffffffffu, valid)) {
          const int s = (2 * i + 1) % kRing;
          ok = wait(T_FULL + s, (2 * i + 1) / kRing) && ok;
          if (!valid)
#pragma unroll
            for (uint32_t x = 0; x < D / 8; ++x)
              st_shared_v4(base + s * L::tile + (x >> 3) * 16384 + lt * 128 + (x & 7) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[T_P + gr]);
      }
      i0 += n;
      if (ok && last >= 0) ok = wait2(T_O, last);
      if (!(ok = group_all(ok, 3, 256))) break;
      // every product with this piece's Q is done: the next one's takes its place, and its first scores are made
      // while this piece is put out
      if ((more = ahead.next(p))) load_q();
      uint32_t a[16];
      if (last >= 0) {
        uint32_t a1[16];
        tc_fence_after();
        tmem_ld16(t4 + 32 + gr * 32, a);
        tmem_ld16(t4 + 48 + gr * 32, a1);
        tmem_ld_wait();
        tc_fence_before();
#pragma unroll
        for (int h = 0; h < HN; ++h) a[h] = __float_as_uint(__uint_as_float(a[h]) + __uint_as_float(a1[h]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[T_OFREE]);
      // the stream's sums over all tokens of the piece; then the odd stream goes to the even one's threads
      reduce(l, [](float u, float v) { return u + v; });
      named_bar_sync(1 + gr, 128);
      float *X = reinterpret_cast<float *>(smem + L::x);
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        const float4 v = *reinterpret_cast<const float4 *>(s_red[gr][h]);
        l[h] = (v.x + v.y) + (v.z + v.w);
        if (gr == 1) {
          if ((int)lt < D) X[h * D + lt] = last >= 0 ? __uint_as_float(a[h]) : 0.f;
          if (lt == 0) {
            s_m[h] = m[h];
            s_l[h] = l[h];
          }
        }
      }
      named_bar_sync(3, 256);
      if (gr == 0) {
        const bool whole = w.t0 == 0 && w.t1 == w.nt;
        const int64_t at = (int64_t)(2 * blockIdx.x + slot) * kHeads;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          if (h >= w.it.nh) break;
          const float mx = fmaxf(m[h], s_m[h]), use = mx == -INFINITY ? 0.f : mx;
          const float f0 = ex2(m[h] - use), f1 = ex2(s_m[h] - use), sum = f0 * l[h] + f1 * s_l[h];
          const float acc = (last >= 0 ? f0 * __uint_as_float(a[h]) : 0.f) + ((int)lt < D ? f1 * X[h * D + lt] : 0.f);
          if (whole) {
            if ((int)lt < D)
              o[w.b * p.qsb + (w.it.h0 + h) * p.qsh + lt] = __float2bfloat16_rn(mx == -INFINITY ? 0.f : acc / sum);
            if (lse && lt == 0) lse[(int64_t)w.b * p.Hq + w.it.h0 + h] = (mx + log2f(sum)) * 0.6931471805599453f;
          } else {
            if ((int)lt < D) part[(at + h) * D + lt] = acc;
            if (lt == 0) {
              ml[(at + h) * 2] = mx;
              ml[(at + h) * 2 + 1] = sum;
            }
          }
        }
      }
      slot = 1;
      named_bar_sync(3, 256);  // s_red, X and the odd stream's values are rewritten by the next piece
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 128);
}

// ------------------------------------------------------------------ fp32 decode (CUDA cores)
// A token's row is spread over LPT lanes, so a warp takes 32 / LPT tokens a step; every lane keeps its
// dimensions of HN query heads and of their outputs in registers (64 + 64 values at D = 128, whatever HN:
// more heads, more lanes per token) and copies its own pieces of K and V through a ring of its own, 16 KiB
// per warp, so nothing in the loop waits for another lane but the sums of a score.  Those are added up while
// the heads are halved (HN - 1 exchanges instead of HN per step), which leaves every lane one head, its
// maximum, its sum and its weight; the weights then go round.  The warps' (and lanes') maxima, sums and
// outputs are joined at a piece's end.  Up to 4 query heads per key head it is bound by the cache (72 us at 16
// sequences of 8192, 4 key heads of 4 query heads, D = 128: 0.71 of copy bandwidth), with 16 by its sums (216 us).
// Four warps on two CTAs an SM leave them 255 registers: six warps, at 168, take 83 us.
constexpr int kSimtWarps = 4, kSimtThreads = 32 * kSimtWarps, kSimtPerSm = 2;
template <int D, int HN>
struct SimtLayout {
  static constexpr int LPT = 2 * HN < D / 4 ? 2 * HN : D / 4, TPW = 32 / LPT, NP = D / 4 / LPT, depth = 16 / NP;
  static constexpr size_t smem = (size_t)kSimtWarps * depth * 2 * NP * 32 * sizeof(float4);
  static_assert(smem >= (size_t)kSimtWarps * HN * D * sizeof(float), "the ring holds the warps' outputs at the end");
};

// 16 bytes, or zeros when !there (src is not read then)
__device__ __forceinline__ void cp_async16_zfill(void *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

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

template <int D, int HN>
__global__ void __launch_bounds__(kSimtThreads, kSimtPerSm)
    paged_decode_simt(PagedProblem p, const float *q, const float *kc, const float *vc, float *o, float *lse, float *part,
                      float *ml) {
  using L = SimtLayout<D, HN>;
  constexpr int LPT = L::LPT, NP = L::NP, S = L::depth, kStep = kSimtWarps * L::TPW;
  extern __shared__ float4 smem4[];
  __shared__ int64_t buf[34];
  __shared__ float sm[kSimtWarps][HN], sl[kSimtWarps][HN];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, sub = lane / LPT, g = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  PagedWalk w;
  if (!walk_start<kSimtThreads>(p, buf, w)) return;
  const float c = p.scale * 1.4426950408889634f;
  const int mine = lane % LPT / (LPT / HN), home = lane & ~(LPT - 1);
  float4 *ring = smem4 + warp * (S * 2 * NP * 32) + lane;  // [slot][k, v][piece], a lane's own column
  int slot = 0;
  while (w.next(p)) {
    const PagedItem it = w.it;
    const int b = w.b, end = min(w.t1 * kTile, w.len), first = w.t0 * kTile + warp * L::TPW + sub;
    const int steps = (end - w.t0 * kTile + kStep - 1) / kStep;
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
          const float4 x = *reinterpret_cast<const float4 *>(q + b * p.qsb + (it.h0 + h) * p.qsh +
                                                             4 * (j * LPT + lane % LPT));
          qr[h][j] = make_float4(x.x * c, x.y * c, x.z * c, x.w * c);
        }
      }
    }
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
    // step i: this lane's token is first + i kStep; its page's id is read a step before the copies that use it
    uint32_t ok = 0;  // bit per slot: the token is there
    auto page_of = [&](int i) {
      const int n = first + i * kStep;
      return i < steps && n < end ? table[n / p.page] : 0;
    };
    auto copy = [&](int i, int id) {
      const int n = first + i * kStep, z = i % S;
      if (i < steps) {
        bool there = n < end;
        if (there && (id < 0 || id >= p.pages)) {
          if (lane % LPT == 0) report_error(p.status, -1);
          there = false;
        }
        const int64_t at = there ? id * p.csb + it.hk * p.csh + (int64_t)(n % p.page) * p.cst + 4 * (lane % LPT) : 0;
        ok = there ? ok | (1u << z) : ok & ~(1u << z);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          cp_async16_zfill(ring + ((z * 2) * NP + j) * 32, kc + at + 4 * LPT * j, there);
          cp_async16_zfill(ring + ((z * 2 + 1) * NP + j) * 32, vc + at + 4 * LPT * j, there);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int id = page_of(0);
    for (int i = 0; i < S - 1; ++i) {
      const int now = id;
      id = page_of(i + 1);
      copy(i, now);
    }
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int now = id;
      id = page_of(i + S);
      copy(i + S - 1, now);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      const float4 *kv = ring + (i % S) * 2 * NP * 32;
      float s[HN];
#pragma unroll
      for (int h = 0; h < HN; ++h) s[h] = 0.f;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float4 x = kv[j * 32];
#pragma unroll
        for (int h = 0; h < HN; ++h)
          s[h] = fmaf(x.x, qr[h][j].x, fmaf(x.y, qr[h][j].y, fmaf(x.z, qr[h][j].z, fmaf(x.w, qr[h][j].w, s[h]))));
      }
      halve_heads<HN / 2, LPT / 2>(s, lane);
#pragma unroll
      for (int x = LPT / HN / 2; x; x /= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], x);
      const bool there = (ok >> (i % S)) & 1;
      const float score = there ? s[0] : -INFINITY, top = there ? fmaxf(score, kLowest) : -INFINITY;
      if (__any_sync(0xffffffffu, top > m)) {  // rare once the first steps have passed
        const float mn = fmaxf(m, top), f = exp2f(m - (mn == -INFINITY ? 0.f : mn));
        m = mn;
        l *= f;
        rescale(f);
      }
      const float weight = exp2f(score - (m == -INFINITY ? 0.f : m));
      l += weight;
#pragma unroll
      for (int h = 0; h < HN; ++h) s[h] = __shfl_sync(0xffffffffu, weight, home + h * (LPT / HN));
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float4 x = kv[(NP + j) * 32];
#pragma unroll
        for (int h = 0; h < HN; ++h)
          acc[h][j] = make_float4(fmaf(s[h], x.x, acc[h][j].x), fmaf(s[h], x.y, acc[h][j].y),
                                  fmaf(s[h], x.z, acc[h][j].z), fmaf(s[h], x.w, acc[h][j].w));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
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
        for (int j = 0; j < NP; ++j) smem4[(warp * HN + h) * (D / 4) + j * LPT + lane] = acc[h][j];
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
      const int64_t piece = (int64_t)(2 * g + slot) * kHeads + h;
      if (whole) {
        o[b * p.qsb + (it.h0 + h) * p.qsh + dim] = mx == -INFINITY ? 0.f : a / sum;
        if (lse && dim == 0) lse[(int64_t)b * p.Hq + it.h0 + h] = (mx + log2f(sum)) * 0.6931471805599453f;
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
// One CTA of D threads per (sequence, query head): joins the pieces of an item that was cut,
// o = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i, and writes the rows of empty sequences
// (o = 0, lse = -inf).  A piece sits in its CTA's slot 1 when that CTA's range began in an earlier
// item, else in slot 0.  Bound by finding its item (7 us for 2048 rows, largely behind the decode's own end).
template <int D, typename T>
__global__ void __launch_bounds__(D) paged_join_kernel(PagedProblem p, int grid, T *o, float *lse, const float *part,
                                                       const float *ml) {
  __shared__ int64_t buf[2 * D / 32 + 2];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, tid = threadIdx.x;
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
  const int64_t slices = (p.Hq / p.Hkv + kHeads - 1) / kHeads;
  const int64_t tiles = ((int64_t)p.max_blocks * p.page + kTile - 1) / kTile;
  const int64_t most = tiles * p.B * p.Hkv * slices, want = (int64_t)(p.num_sms * per < kMaxGrid ? p.num_sms * per : kMaxGrid);
  return (int)(most < want ? most : want);
}

template <int D, typename T, typename Launch>
cudaError_t run_decode(Launch launch, int per, const PagedProblem &p, void *o, float *lse, void *ws, cudaStream_t s) {
  const int G = paged_grid(p, per);
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

template <int D>
cudaError_t run_dim(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse, void *ws,
                    cudaStream_t s) {
  const int group = p.Hq / p.Hkv;
  if (p.esz == 4) {
    auto kernel = group <= 4 ? paged_decode_simt<D, 4> : group <= 8 ? paged_decode_simt<D, 8> : paged_decode_simt<D, 16>;
    constexpr size_t smem = SimtLayout<D, 4>::smem;
    static_assert(smem == SimtLayout<D, 8>::smem && smem == SimtLayout<D, 16>::smem, "16 KiB per warp");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return run_decode<D, float>(
        [&](int G, float *part, float *ml) {
          return launch_overlapped(kernel, dim3(G), dim3(kSimtThreads), smem, s, p, (const float *)q, (const float *)kc,
                                   (const float *)vc, (float *)o, lse, part, ml);
        },
        kSimtPerSm, p, o, lse, ws, s);
  }
  using bf16 = __nv_bfloat16;
  // the rows of one copy: the largest power of two up to 128 that divides a page (a copy stays inside a page
  // and starts on the 8-row pattern of the tile)
  int box = p.page & -p.page;
  box = box > kTile ? kTile : box < 8 ? 0 : box;
  CUtensorMap mk{}, mv{};
  if (box) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.page, (uint64_t)p.Hkv, (uint64_t)p.pages};
    const uint64_t strides[3] = {(uint64_t)p.cst * 2, (uint64_t)p.csh * 2, (uint64_t)p.csb * 2};
    if (!make_tmap_bf16(&mk, kc, dims, strides, box) || !make_tmap_bf16(&mv, vc, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  auto kernel = group <= 4 ? paged_decode_tc<D, 4> : group <= 8 ? paged_decode_tc<D, 8> : paged_decode_tc<D, 16>;
  constexpr size_t smem = TcLayout<D>::smem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return run_decode<D, bf16>(
      [&](int G, float *part, float *ml) {
        return launch_overlapped(kernel, dim3(G), dim3(kTcThreads), smem, s, mk, mv, box, p, (const bf16 *)q,
                                 (const bf16 *)kc, (const bf16 *)vc, (bf16 *)o, lse, part, ml);
      },
      1, p, o, lse, ws, s);
}

}  // namespace

size_t paged_decode_ws_bytes(int d, int num_sms) {
  return align256((size_t)2 * (2 * num_sms) * kHeads * (d + 2) * sizeof(float));
}

cudaError_t paged_append(const PagedProblem &p, const void *k, const void *v, void *kc, void *vc, int T, int64_t sb,
                         int64_t sh, int64_t st, const int *start, const int *new_lens, int *status, cudaStream_t s) {
  TimedLaunch t(K_PAGED_APPEND, s);
  int shift = 0;  // log2 of the 16-byte pieces of a row (d = 64 or 128, 2 or 4 bytes: 8 to 32)
  while (16 << shift < p.d * p.esz) ++shift;
  const uint32_t rows = (uint32_t)p.B * p.Hkv * T, per = 256u >> shift;
  paged_append_kernel<<<(rows + per - 1) / per, 256, 0, s>>>(p, (const char *)k, (const char *)v, (char *)kc, (char *)vc,
                                                             (uint32_t)T, start, new_lens, sb, sh, st, shift, rows,
                                                             status);
  return cudaGetLastError();
}

cudaError_t paged_decode(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse,
                         void *ws, cudaStream_t s) {
  return p.d == 64 ? run_dim<64>(p, q, kc, vc, o, lse, ws, s) : run_dim<128>(p, q, kc, vc, o, lse, ws, s);
}

}  // namespace linattn
