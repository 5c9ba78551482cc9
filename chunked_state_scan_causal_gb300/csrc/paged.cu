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
// One thread per 16 bytes of a row of k and of v: a copy, bound by its bytes (or, for one token per
// sequence, by the launch).  Rows past new_lens, outside the table or with a page id outside the
// cache are left unwritten; the latter two are recorded in the status word.
__global__ void __launch_bounds__(256) paged_append_kernel(PagedProblem p, const char *k, const char *v, char *kc,
                                                           char *vc, int T, const int *start, const int *new_lens,
                                                           int64_t sb, int64_t sh, int64_t st, int row16,
                                                           int64_t n, int *status) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int c = (int)(i % row16);
  int64_t r = i / row16;
  const int t = (int)(r % T);
  r /= T;
  const int h = (int)(r % p.Hkv), b = (int)(r / p.Hkv);
  if (new_lens && t >= new_lens[b]) return;
  const int64_t pos = (int64_t)start[b] + t;
  const int64_t block = pos / p.page;
  if (start[b] < 0 || block >= p.max_blocks) {
    report_error(status, -1);
    return;
  }
  const int id = p.table[(int64_t)b * p.tstride + block];
  if (id < 0 || id >= p.pages) {
    report_error(status, -1);
    return;
  }
  const int64_t src = (b * sb + h * sh + t * st) * p.esz + 16 * c;
  const int64_t dst = (id * p.csb + h * p.csh + (pos - block * p.page) * p.cst) * p.esz + 16 * c;
  *reinterpret_cast<uint4 *>(kc + dst) = *reinterpret_cast<const uint4 *>(k + src);
  *reinterpret_cast<uint4 *>(vc + dst) = *reinterpret_cast<const uint4 *>(v + src);
}

// ------------------------------------------------------------------ work split of the decode
// An item is one (sequence, key head, slice of up to 16 of its query heads): nt = ceil(len / 128)
// tiles of 128 tokens.  All tiles, item after item, are cut into G equal ranges, one per CTA, so
// ragged lengths balance by themselves and few long sequences are split over every SM.  A CTA that
// holds a whole item writes its output; the pieces of the other items go to the workspace, at most
// two per CTA (its first and its last item), and paged_join_kernel joins them.
constexpr int kTile = 128;

__device__ __forceinline__ int seq_len(const PagedProblem &p, int b) {
  const int64_t cap = (int64_t)p.max_blocks * p.page;
  const int n = p.seq_lens[b];
  return n < 0 ? 0 : (int64_t)n > cap ? (int)cap : n;
}
__device__ __forceinline__ int seq_tiles(const PagedProblem &p, int b) { return (seq_len(p, b) + kTile - 1) / kTile; }
// the first tile of CTA g's range, and the CTA whose range holds tile x
__device__ __forceinline__ int64_t range_lo(int64_t total, int G, int g) { return total * g / G; }
__device__ __forceinline__ int range_of(int64_t total, int G, int64_t x) { return (int)(((x + 1) * G - 1) / total); }

// Sum over b < B of tiles, and the sequence holding tile x with its first tile (b = B when x is
// past the end; x = -1 only sums, the sequence index then limits the sum: tiles before sequence
// `upto`).  Called by every thread of the block; `buf` holds 34 values.
template <int NT>
__device__ int64_t locate(const PagedProblem &p, int items, int64_t x, int64_t *buf, int &b_out, int64_t &first) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int64_t base = 0;
  if (tid == 0) buf[32] = p.B;
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    const int64_t mine = b < p.B ? (int64_t)seq_tiles(p, b) * items : 0;
    int64_t s = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane == 31) buf[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += buf[w];
      all += buf[w];
    }
    const int64_t lo = base + before + s - mine;
    if (mine > 0 && x >= lo && x < lo + mine) {
      buf[32] = b;
      buf[33] = lo;
    }
    base += all;
    __syncthreads();
  }
  b_out = (int)buf[32];
  first = buf[33];
  __syncthreads();
  return base;
}

constexpr int kHeads = 16;  // query heads of an item

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

// ------------------------------------------------------------------ fp32 decode (CUDA cores)
constexpr int kSub = 64;       // tokens staged at a time
constexpr int kPagedThreads = 128;

template <int D>
constexpr size_t paged_simt_smem() {
  return (size_t)(2 * kSub * (D + 4) + kHeads * kSub + kHeads * D + 3 * kHeads) * 4;
}

template <int D, typename T>
__global__ void __launch_bounds__(kPagedThreads)
    paged_decode_simt(PagedProblem p, const T *q, const T *kc, const T *vc, T *o, float *lse, float *part, float *ml) {
  constexpr int LD = D + 4;
  constexpr int HT = kHeads * D / kPagedThreads;  // heads per thread in the value product
  extern __shared__ float4 smem4[];
  __shared__ int64_t buf[34];
  float *sk = reinterpret_cast<float *>(smem4), *sv = sk + kSub * LD, *sp = sv + kSub * LD, *sq = sp + kHeads * kSub;
  float *sm = sq + kHeads * D, *sl = sm + kHeads, *sc = sl + kHeads;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int slices = (p.Hq / p.Hkv + kHeads - 1) / kHeads, items = p.Hkv * slices;
  int b;
  int64_t first;
  const int64_t total = locate<kPagedThreads>(p, items, -1, buf, b, first);
  const int G = (int)min((int64_t)gridDim.x, total);  // no empty range between two pieces of an item
  if (g >= G) return;
  int64_t x = range_lo(total, G, g);
  const int64_t end = range_lo(total, G, g + 1);
  locate<kPagedThreads>(p, items, x, buf, b, first);
  const float c = p.scale * 1.4426950408889634f;
  const int dim = tid % D, hbase = (tid / D) * HT;
  int slot = 0;
  while (x < end) {
    const int nt = seq_tiles(p, b), len = seq_len(p, b);
    if (nt == 0 || x >= first + (int64_t)nt * items) {
      first += (int64_t)nt * items;
      ++b;
      continue;
    }
    const int i = (int)((x - first) / nt);
    const PagedItem it = item_of(p, slices, b, i);
    const int t0 = (int)((x - first) % nt), t1 = (int)min((int64_t)nt, t0 + end - x);
    for (int e = tid; e < kHeads * D; e += kPagedThreads) {
      const int h = e / D;
      sq[e] = h < it.nh ? (float)q[b * p.qsb + (it.h0 + h) * p.qsh + e % D] * c : 0.f;
    }
    if (tid < kHeads) {
      sm[tid] = -INFINITY;
      sl[tid] = 0.f;
    }
    float acc[HT];
#pragma unroll
    for (int h = 0; h < HT; ++h) acc[h] = 0.f;
    for (int n0 = t0 * kTile; n0 < min(t1 * kTile, len); n0 += kSub) {
      __syncthreads();
      for (int r = warp; r < kSub; r += kPagedThreads / 32) {
        const int n = n0 + r;
        int id = -1;
        if (n < len) {
          id = p.table[(int64_t)b * p.tstride + n / p.page];
          if (id < 0 || id >= p.pages) {
            if (lane == 0) report_error(p.status, -1);
            id = -1;
          }
        }
        const int64_t off = id * p.csb + it.hk * p.csh + (n % p.page) * p.cst;
        for (int e = lane; e < D; e += 32) {
          sk[r * LD + e] = id >= 0 ? (float)kc[off + e] : 0.f;
          sv[r * LD + e] = id >= 0 ? (float)vc[off + e] : 0.f;
        }
        if (lane < kHeads) sp[lane * kSub + r] = id >= 0 ? 0.f : -INFINITY;
      }
      __syncthreads();
      {
        const int n = tid % kSub;
        const float4 *kr = reinterpret_cast<const float4 *>(sk + n * LD);
        for (int h = tid / kSub; h < it.nh; h += kPagedThreads / kSub) {
          const float4 *qr = reinterpret_cast<const float4 *>(sq + h * D);
          float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll 8
          for (int e = 0; e < D / 4; ++e) {
            const float4 u = kr[e], w = qr[e];
            a0 = fmaf(u.x, w.x, a0);
            a1 = fmaf(u.y, w.y, a1);
            a2 = fmaf(u.z, w.z, a2);
            a3 = fmaf(u.w, w.w, a3);
          }
          if (sp[h * kSub + n] == 0.f) sp[h * kSub + n] = (a0 + a1) + (a2 + a3);
        }
      }
      __syncthreads();
      for (int h = warp; h < it.nh; h += kPagedThreads / 32) {
        const float s0 = sp[h * kSub + lane], s1 = sp[h * kSub + lane + 32];
        float m = fmaxf(s0, s1);
#pragma unroll
        for (int w = 16; w; w /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        const float old = sm[h], mn = fmaxf(old, m), use = mn == -INFINITY ? 0.f : mn;
        const float p0 = exp2f(s0 - use), p1 = exp2f(s1 - use);
        float l = p0 + p1;
#pragma unroll
        for (int w = 16; w; w /= 2) l += __shfl_xor_sync(0xffffffffu, l, w);
        sp[h * kSub + lane] = p0;
        sp[h * kSub + lane + 32] = p1;
        __syncwarp();
        if (lane == 0) {
          const float f = exp2f(old - use);
          sc[h] = f;
          sl[h] = sl[h] * f + l;
          sm[h] = mn;
        }
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < HT; ++h)
        if (hbase + h < it.nh) {
          float a = acc[h] * sc[hbase + h];
          const float *pr = sp + (hbase + h) * kSub;
#pragma unroll 8
          for (int r = 0; r < kSub; ++r) a = fmaf(pr[r], sv[r * LD + dim], a);
          acc[h] = a;
        }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
#pragma unroll
    for (int h = 0; h < HT; ++h)
      if (hbase + h < it.nh) {
        const int hh = hbase + h;
        if (whole)
          o[b * p.qsb + (it.h0 + hh) * p.qsh + dim] = (T)(sl[hh] > 0.f ? acc[h] / sl[hh] : 0.f);
        else
          part[((int64_t)(2 * g + slot) * kHeads + hh) * D + dim] = acc[h];
      }
    if (tid < it.nh) {
      if (whole) {
        if (lse) lse[(int64_t)b * p.Hq + it.h0 + tid] = (sm[tid] + log2f(sl[tid])) * 0.6931471805599453f;
      } else {
        ml[((int64_t)(2 * g + slot) * kHeads + tid) * 2] = sm[tid];
        ml[((int64_t)(2 * g + slot) * kHeads + tid) * 2 + 1] = sl[tid];
      }
    }
    slot = 1;
    x += t1 - t0;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ join
// One CTA of D threads per (sequence, query head): joins the pieces of an item that was cut,
// o = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i, and writes the rows of empty sequences
// (o = 0, lse = -inf).  A piece sits in its CTA's slot 1 when that CTA's range began in an earlier
// item, else in slot 0.
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
  float m = -INFINITY;
  for (int g = g0; g <= g1; ++g) {
    const int slot = range_lo(all, G, g) < lo;
    m = fmaxf(m, ml[((int64_t)(2 * g + slot) * kHeads + hh) * 2]);
  }
  const float use = m == -INFINITY ? 0.f : m;
  float a = 0.f, l = 0.f;
#pragma unroll 4
  for (int g = g0; g <= g1; ++g) {
    const int slot = range_lo(all, G, g) < lo;
    const int64_t at = (int64_t)(2 * g + slot) * kHeads + hh;
    const float f = exp2f(ml[at * 2] - use);
    a = fmaf(f, part[at * D + tid], a);
    l = fmaf(f, ml[at * 2 + 1], l);
  }
  o[orow] = (T)(l > 0.f ? a / l : 0.f);
  if (lse && tid == 0) lse[(int64_t)b * p.Hq + h] = (m + log2f(l)) * 0.6931471805599453f;
}

int paged_grid(const PagedProblem &p) {
  const int64_t slices = (p.Hq / p.Hkv + kHeads - 1) / kHeads;
  const int64_t tiles = ((int64_t)p.max_blocks * p.page + kTile - 1) / kTile;
  const int64_t most = tiles * p.B * p.Hkv * slices, want = (int64_t)p.num_sms * 2;
  return (int)(most < want ? most : want);
}

template <int D, typename T>
cudaError_t run_simt(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse,
                     void *ws, cudaStream_t s) {
  const int G = paged_grid(p);
  float *part = static_cast<float *>(ws), *ml = part + (size_t)2 * (2 * p.num_sms) * kHeads * D;
  constexpr size_t smem = paged_simt_smem<D>();
  cudaError_t e = cudaFuncSetAttribute(paged_decode_simt<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  {
    TimedLaunch t(K_PAGED_DECODE, s);
    e = launch_overlapped(paged_decode_simt<D, T>, dim3(G), dim3(kPagedThreads), smem, s, p, (const T *)q,
                          (const T *)kc, (const T *)vc, (T *)o, lse, part, ml);
    if (e != cudaSuccess) return e;
  }
  TimedLaunch t(K_PAGED_JOIN, s);
  return launch_overlapped(paged_join_kernel<D, T>, dim3(p.B * p.Hq), dim3(D), 0, s, p, G, (T *)o, lse,
                           (const float *)part, (const float *)ml);
}

}  // namespace

size_t paged_decode_ws_bytes(int d, int num_sms) {
  return align256((size_t)2 * (2 * num_sms) * kHeads * (d + 2) * sizeof(float));
}

cudaError_t paged_append(const PagedProblem &p, const void *k, const void *v, void *kc, void *vc, int T, int64_t sb,
                         int64_t sh, int64_t st, const int *start, const int *new_lens, int *status, cudaStream_t s) {
  TimedLaunch t(K_PAGED_APPEND, s);
  const int row16 = p.d * p.esz / 16;
  const int64_t n = (int64_t)p.B * p.Hkv * T * row16;
  paged_append_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, (const char *)k, (const char *)v, (char *)kc,
                                                                  (char *)vc, T, start, new_lens, sb, sh, st, row16,
                                                                  n, status);
  return cudaGetLastError();
}

cudaError_t paged_decode(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse,
                         void *ws, cudaStream_t s) {
  if (p.esz == 4)
    return p.d == 64 ? run_simt<64, float>(p, q, kc, vc, o, lse, ws, s) : run_simt<128, float>(p, q, kc, vc, o, lse, ws, s);
  return p.d == 64 ? run_simt<64, __nv_bfloat16>(p, q, kc, vc, o, lse, ws, s)
                   : run_simt<128, __nv_bfloat16>(p, q, kc, vc, o, lse, ws, s);
}

}  // namespace linattn
