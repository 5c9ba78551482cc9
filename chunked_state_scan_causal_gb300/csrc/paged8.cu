// The paged key-value cache in 8 bits: appending quantises, gathering reads back, decoding attends over the codes.
//
// The cache holds e4m3 codes, [pages, Hkv, page, d] with any strides (page a multiple of 16), and fp32 scales
// [pages, Hkv, page / 16, 2]: one for the keys and one for the values of every 16 tokens ("block") of a page and head; a
// cached value is code x scale.  Appending takes scale = 2^e with the smallest e >= -126 that keeps the block's
// largest finite magnitude within 448 2^e.  e4m3 is a floating-point format, so the scale only places its range:
// a power of two costs no relative precision, makes x / scale, the read-back and the change of a block's scale
// (an exponent shift, but for codes that become subnormal) exact, and the result is the same whatever the hardware.
// Decoding takes any positive finite scale.
#include <cuda_bf16.h>

#include <type_traits>

#include "paged.cuh"

namespace linattn {
namespace {

// two floats as e4m3 codes, to nearest (magnitudes above 448 and infinities give 448, NaN the code 0x7f)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t f16x2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
  return r;
}
// two f16 as e5m2 codes, to nearest
__device__ __forceinline__ uint32_t e5m2x2(uint32_t f16x2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(f16x2));
  return r;
}

// The exponent e of the scale of a block whose largest finite magnitude has these fp32 bits: with amax = m 2^E
// (1 <= m < 2) it is E - 8, or E - 7 where m > 1.75 (448 = 1.75 2^8).  Between -126 and 120.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return max(e, -126);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

// ------------------------------------------------------------------ append
// A warp per block of 16 slots, key head, and k or v: it owns the block, so nothing is shared with other warps.
// A lane takes 16 values of a row at a time, D / 16 lanes a row.  The rows stay in registers between the scan for
// the largest magnitude and the rounding.  Only the first block of a sequence's new tokens can hold older ones: where the
// new tokens need a larger scale, those are read, multiplied by old / new scale and rounded again.
// Slots without a new token keep their bytes.
// Bound by memory once the look for the largest magnitude takes few instructions (value by value: 30 us): 8 ragged prompts
// of up to 4096 tokens, 8 heads, bf16: 23.5 us, 0.85 of copy bandwidth; one token per sequence by its launch (2.1 us; which overlaps
// the end of the kernel before it: 4.1 -> 2.8 us call after call).
template <int D, typename T>
__global__ void __launch_bounds__(256)
    paged_append_q8_kernel(PagedProblem p, const T *k, const T *v, uint8_t *kc, uint8_t *vc, uint32_t tokens,
                           const int *start, const int *new_lens, int64_t sb, int64_t sh, int64_t st, uint32_t nblocks,
                           uint32_t warps) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSteps = kScaleTokens / kRows;  // lanes of a row, rows of a step
  constexpr int kWords = 16 * sizeof(T) / 16;                                         // 16-byte pieces of a lane
  griddep_wait();
  const uint32_t id = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (id >= warps) return;
  const uint32_t which = id & 1, r = id >> 1, j = r % nblocks, bh = r / nblocks, b = bh / (uint32_t)p.Hkv,
                 h = bh % (uint32_t)p.Hkv;
  const int first = start[b];
  const int64_t n = new_lens ? min(max(new_lens[b], 0), (int)tokens) : (int)tokens;
  const int off = first & (kScaleTokens - 1);                    // the first new token's slot in its block
  const int64_t t0 = (int64_t)j * kScaleTokens - off;            // the new token that slot 0 would hold
  if (n == 0 || t0 >= n) return;
  // the rows first: they travel while the page is looked up
  const int row = lane / kLanes, c = lane % kLanes, lo = (int)max((int64_t)0, -t0), hi = (int)min((int64_t)kScaleTokens, n - t0);
  const T *x = (which ? v : k) + b * sb + h * sh + (t0 + row) * st + c * 16;
  uint4 w[kSteps][kWords];
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int y = 0; y < kWords; ++y) {
      const int s = i * kRows + row;
      w[i][y] = s >= lo && s < hi ? reinterpret_cast<const uint4 *>(x + i * kRows * st)[y] : make_uint4(0, 0, 0, 0);
    }
  const int64_t pos = (int64_t)first + t0;                       // slot 0's position
  const bool inside = first >= 0 && pos < (int64_t)p.max_blocks * p.page;
  const int page = inside ? p.table[(int64_t)b * p.tstride + (uint32_t)pos / (uint32_t)p.page] : -1;
  if (page < 0 || page >= p.pages) {
    if (lane == 0) report_error(p.status, -1);
    return;
  }
  const int slot0 = (uint32_t)pos % (uint32_t)p.page;
  uint8_t *codes = (which ? vc : kc) + page * p.csb + h * p.csh + (slot0 + row) * p.cst + c * 16;
  float *scale = p.scales + page * p.ssb + h * p.ssh + slot0 / kScaleTokens * 2 + which;
  const float had = off && j == 0 ? *scale : 0.f;                // of the tokens that are there already
  // the largest magnitude: they order as integers (bf16 in pairs); what is not finite is left out, in a second look
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int y = 0; y < kWords; ++y)
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const uint32_t u = (&w[i][y].x)[z];
        top = sizeof(T) == 2 ? __vmaxu2(top, u & 0x7fff7fffu) : max(top, u & 0x7fffffffu);
      }
  if (sizeof(T) == 2) top = max(top & 0xffff0000u, top << 16);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool bad = top >= 0x7f800000u;
  if (bad) {
    top = 0;
#pragma unroll 1
    for (int i = 0; i < kSteps * kWords * 4; ++i) {
      uint32_t u = 0;
#pragma unroll
      for (int z = 0; z < kSteps * kWords * 4; ++z)
        if (z == i) u = (&w[z / 4 / kWords][z / 4 % kWords].x)[z % 4];
      const uint32_t a = sizeof(T) == 2 ? u & 0x7fff0000u : u & 0x7fffffffu, low = sizeof(T) == 2 ? u << 16 & 0x7fff0000u : 0;
      top = max(top, max(a >= 0x7f800000u ? 0u : a, low >= 0x7f800000u ? 0u : low));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const int e = scale_exponent(top);
  float now = exp2i(e), inv = exp2i(-e);
  if (had >= now) {  // the old scale does
    now = had;
    inv = 1.f / had;
  }
  if (off && j == 0 && had < now) {
    const float shift = had / now;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int s = i * kRows + row;
      if (s >= off) continue;
      uint4 *at = reinterpret_cast<uint4 *>(codes + i * kRows * p.cst);
      uint4 old = *at;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const uint32_t u = (&old.x)[z];
        const float4 f = four_of(u);
        (&old.x)[z] = e4m3x2(f.x * shift, f.y * shift) | e4m3x2(f.z * shift, f.w * shift) << 16;
      }
      *at = old;
    }
  }
  if (lane == 0 && now != had) *scale = now;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int s = i * kRows + row;
    if (s < lo || s >= hi) continue;
    uint4 out;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      float f[4];
      if constexpr (sizeof(T) == 2) {
        const uint32_t u0 = (&w[i][z / 2].x)[z % 2 * 2], u1 = (&w[i][z / 2].x)[z % 2 * 2 + 1];
        f[0] = bf16lo(u0), f[1] = bf16hi(u0), f[2] = bf16lo(u1), f[3] = bf16hi(u1);
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = __uint_as_float((&w[i][z].x)[y]);
      }
      if (bad)
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = fabsf(f[y]) <= 3.402823466e+38f ? f[y] : __uint_as_float(0x7fc00000u);
      (&out.x)[z] = e4m3x2(f[0] * inv, f[1] * inv) | e4m3x2(f[2] * inv, f[3] * inv) << 16;
    }
    *reinterpret_cast<uint4 *>(codes + i * kRows * p.cst) = out;
  }
}

// ------------------------------------------------------------------ gather
// A warp per block of 16 tokens, key head, and k or v: codes in by 16 bytes a lane, values out (16 a lane).  With
// `start` the tokens from start[b] on; the tokens of an output row block may then lie in two cache blocks, so every row
// looks its own page up.  Rows past the length, and rows on bad pages, are zero.
template <int D, typename T>
__global__ void __launch_bounds__(256, 5)
    paged_gather_q8_kernel(PagedProblem p, const uint8_t *kc, const uint8_t *vc, T *k, T *v, uint32_t tokens,
                           const int *start, int64_t sb, int64_t sh, int64_t st, uint32_t nblocks, uint32_t warps) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSteps = kScaleTokens / kRows;
  griddep_wait();
  const uint32_t id = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (id >= warps) return;
  const uint32_t which = id & 1, r = id >> 1, j = r % nblocks, bh = r / nblocks, b = bh / (uint32_t)p.Hkv,
                 h = bh % (uint32_t)p.Hkv, row = lane / kLanes, c = lane % kLanes;
  const int len = seq_len(p, b), first = start ? max(start[b], 0) : 0;
  const uint8_t *codes = (which ? vc : kc) + h * p.csh + c * 16;
  T *out = (which ? v : k) + b * sb + h * sh + c * 16;
  uint4 w[kSteps];
  float s[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t pos = (int64_t)first + (int64_t)j * kScaleTokens + i * kRows + row;
    int page = -1;
    const bool there = pos < len && j * kScaleTokens + i * kRows + row < tokens;
    if (there) {
      page = p.table[(int64_t)b * p.tstride + (uint32_t)pos / (uint32_t)p.page];
      if (page < 0 || page >= p.pages) {
        report_error(p.status, -1);
        page = -1;
      }
    }
    const uint32_t slot = (uint32_t)pos % (uint32_t)p.page;
    w[i] = page >= 0 ? *reinterpret_cast<const uint4 *>(codes + page * p.csb + slot * p.cst) : make_uint4(0, 0, 0, 0);
    s[i] = page >= 0 ? p.scales[page * p.ssb + h * p.ssh + slot / kScaleTokens * 2 + which] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t t = j * kScaleTokens + i * kRows + row;
    if (t >= tokens) continue;
    T *at = out + t * st;
    float4 f[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      f[z] = four_of((&w[i].x)[z]);
      f[z] = make_float4(f[z].x * s[i], f[z].y * s[i], f[z].z * s[i], f[z].w * s[i]);
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
        reinterpret_cast<uint4 *>(at)[z] =
            make_uint4(pack_bf16(f[2 * z].x, f[2 * z].y), pack_bf16(f[2 * z].z, f[2 * z].w),
                       pack_bf16(f[2 * z + 1].x, f[2 * z + 1].y), pack_bf16(f[2 * z + 1].z, f[2 * z + 1].w));
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z) reinterpret_cast<float4 *>(at)[z] = f[z];
    }
  }
}

// ------------------------------------------------------------------ bf16 decode (tensor cores)
// As in the bf16 cache's kernel (paged.cu), a tile is 128 tokens, the rows are the narrow side of the products, and
//     S = K Q^T  (lane = token, column = row),   O^T += V^T P^T  (lane = value dimension, column = row),
// here with the codes as the 128-row operands of 8-bit products, straight from shared memory: nothing of the cache is
// converted.  What is not in the cache is cut into 8-bit parts, a column of the product per part:
//   q / qs = q1 + q2 / 16 with qs a power of two, in e4m3 (4 significant bits): exact (a bf16 value has 8 bits) down to
//     2^-14 of the row's largest value, within 2^-21 of that value below;
//   the weight, an f16, w = p1 + p2 / 16 + p3 / 256 in e5m2: exact for every f16 up to 2^15, since a part (3 bits, rounded to
//     nearest) leaves at most 2^-3 of its power of two, 16 times which loses no bits above the smallest f16, 2^-24.
// (e4m3 parts, whose smallest step is 2^-9, would hold a weight to 2^-17 only, whatever its size, and many small
// weights beside a large one are what a softmax often consists of.)
// A key's scale goes into its score, a value's into its weight:
//   x = c ks qs (S1 + S2 / 16),   w = 2^(x - m) vs r <= 2^15,   o = (O1 + O2 / 16 + O3 / 256) / (r sum 2^(x - m)).
// Both references are a row's own and made of the tokens that it sees: r places the largest weight times value scale, so that
// large values at tokens of no weight leave the weights that count where they are.  m moves only when a score exceeds
// it by more than 8 (to that score), r only when a w exceeds 2^15 (that w to 2^11, where an f16 holds its 11 bits down to 2^-25 of
// it); both are asked for by one vote of the threads per tile, so that the reductions over the tile's tokens and the
// rescaling of O happen in the first tile and rarely after.
//
// Warps: four for the softmax (lane = token) and the output (lane = value dimension), eight with more than 8 rows, each
// four for half of them; then one that issues the products, one that walks the CTA's pieces, publishes them and
// loads tiles (tensor-map copies) and scales, one that cuts the queries of the next piece into parts.  A tile's chain
// (scores, softmax, product) takes longer than its loads, and a piece's ends add to it, so an SM holds as many
// CTAs as fit rather than deep rings: four up to 4 rows, three up to 8, two above.
// Bound by memory where sequences are long (64 of up to 16384 tokens, 8 key heads: 198 us, 0.99 of copy bandwidth, with
// up to 4 rows, 0.96 with 8, 0.88 with 16; d = 64, where a tile has half the bytes, 0.85); with 256 sequences of 125 to 500
// tokens by the pieces' ends (38 us with 4 rows, 47 with 8; the bytes alone 24).  The seven or eleven warps of a
// CTA run five different programs, so their instructions have to fit the caches: loops are not unrolled but over rows,
// waits are short, and a tile has one path.
template <int D, int HN>
struct Layout8 {
  static constexpr int G = HN > 8 ? 2 : 1, HG = HN / G;         // groups of four softmax warps; rows of a thread
  static constexpr int threads = 32 * (4 * G + 3), per_sm = HN == 4 ? 4 : HN == 8 ? 3 : 2;
  static constexpr int NS = HN < 8 ? 16 : 2 * HN;               // columns of S: part, row
  static constexpr int NO = HN < 8 ? 16 : HN == 8 ? 32 : 48;    // columns of O: (group,) part, row
  static constexpr int ring = D == 128 ? (HN == 4 ? 3 : HN == 8 ? 4 : 5) : (HN == 4 ? 6 : HN == 8 ? 8 : 11);
  static constexpr int pieces = 16, nsc = 8;                    // published pieces and tiles of scales kept: see the loads
  // two buffers for Q; those of 4 rows, which fill half of S, share the rows (and columns of S) of one
  static constexpr uint32_t qbuf = HN == 4 ? 8 * D : NS * D, scol = HN == 4 ? 8 : 0;
  static constexpr uint32_t tile = 128 * D, q = ring * tile, p = q + 2 * qbuf, sc = p + 128 * NO,
                            sq = sc + nsc * 64, desc = sq + pieces * HN * 4, red = desc + pieces * 32,
                            ref = red + G * HG * 32, sum = ref + G * HG * 8, nan = sum + HN * 16, bars = nan + D * 4;
  static constexpr int nbars = 2 * pieces + 2 * 2 + 2 + 2 + nsc + 2 * ring;
  static constexpr uint32_t end = bars + nbars * 8 + 16;  // (the tensor memory's address, two flags)
  // (at D = 64 the second half of a value tile's 128 lanes is whatever follows the tile)
  static constexpr size_t smem = D == 128 || end > q + tile ? end : q + tile;
  static_assert(per_sm * (smem + 1024) <= 233472, "what an SM holds");
  static constexpr uint32_t cols = HN > 8 ? 128 : 64;           // of tensor memory: S of even and odd tiles, O
};
// The reference of a row that no token has reached yet (NaN scores move none: their sum says that there are some); above it
// what a token's score counts as at least, -inf too, so that o is 0 only where no token is; and above that the least that
// a reference moves to, so that a score of -inf has a weight of zero even among its like (0 / 0).
constexpr float kNone = kLowest, kFirst = -3.2e38f, kFloor = -3e38f;
// A published piece.
struct Piece8 {
  int b, hk, h0, nh, t0, t1, nt, len;
};

// Instruction descriptor, kind::f8f6f4: e4m3 A, B of type b (0 e4m3, 1 e5m2), fp32 D (the fields of idesc_bf16).
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t b, uint32_t M, uint32_t N, bool a_mn, bool b_mn) {
  return (1u << 4) | (b << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Shared-memory descriptor with the layout field: 0 no swizzle, 2 128 bytes, 4 64 bytes.
__device__ __forceinline__ uint64_t sdesc(uint32_t start, uint32_t lbo, uint32_t sbo, uint64_t layout) {
  return (uint64_t)((start >> 4) & 0x3FFFu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         layout << 61;
}
// D[tmem] (+)= A[smem] B[smem], issued by one elected lane of the warp.
__device__ __forceinline__ void mma_codes_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Whether any of the group's threads says so.
__device__ __forceinline__ bool group_any(bool x, uint32_t id, uint32_t nthreads) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "barrier.cta.red.or.pred po, %2, %3, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}\n"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}
// The larger one, or NaN if there is one.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// The warp's largest value (NaN left out).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// The largest of three (NaN left out).
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// Two products, and two sums, an instruction.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(x)), "l"(reinterpret_cast<uint64_t &>(y)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(x)), "l"(reinterpret_cast<uint64_t &>(y)));
  return r;
}
// The larger ones (NaN left out).
__device__ __forceinline__ uint32_t max_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ float lg2(float x) {  // (to 2^-22 or so: it only places a reference)
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// What is left of two f16 values after their e4m3 part, times 16 (exact).
__device__ __forceinline__ uint32_t left16(uint32_t h, uint32_t part) {
  const uint32_t a = f16x2_of_e4m3x2(part);
  const __half2 m = __float2half2_rn(-16.f), n = __float2half2_rn(16.f);
  const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), m, __hmul2(*reinterpret_cast<__half2 *>(&h), n));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// The same after their e5m2 part, which is an f16's upper byte (up to 2^15: 16 h itself would not fit).
__device__ __forceinline__ uint32_t left16_e5m2(uint32_t h, uint32_t part) {
  const uint32_t a = __byte_perm(part, 0, 0x1404);
  const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&a)),
                            __float2half2_rn(16.f));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Byte offset of a row's 16-byte chunk in a tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
template <int D>
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile, uint32_t ks) {  // contraction over the D columns
  return D == 128 ? sdesc(tile + ks * 32, 16, 1024, 2) : sdesc(tile + ks * 32, 16, 512, 4);
}
template <int D>
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile, uint32_t ks) {  // contraction over the 128 rows
  return D == 128 ? sdesc(tile + ks * 4096, 16384, 1024, 2) : sdesc(tile + ks * 2048, 8192, 512, 4);
}

// what the scales of a token that is not there are
__device__ const float2 kAbsent = {0.f, -1.f};

// box: rows of a tensor-map copy, at most a page
template <int D, int HN>
__global__ void __launch_bounds__(Layout8<D, HN>::threads, Layout8<D, HN>::per_sm)
    paged_decode_q8_tc(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, int box,
                       const __grid_constant__ PagedProblem p, const __nv_bfloat16 *q, __nv_bfloat16 *o, float *lse,
                       float *part, float *ml) {
  using L = Layout8<D, HN>;
  constexpr int G = L::G, HG = L::HG, kRing = L::ring, kPieces = L::pieces;
  constexpr int B_D = 0, B_SQ = kPieces, B_QF = 2 * kPieces, B_QE = B_QF + 2, B_S = B_QE + 2, B_P = B_S + 2, B_O = B_P + 1,
                B_SC = B_O + 1, B_FULL = B_SC + L::nsc, B_EMPTY = B_FULL + kRing;
  static_assert(B_EMPTY + kRing == L::nbars, "the barriers");
  extern __shared__ __align__(1024) uint8_t smem[];  // the only shared memory: it begins on the swizzle's pattern
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::bars);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + L::nbars);
  int *abort_flag = reinterpret_cast<int *>(tslot + 1), *status = abort_flag + 1;
  float2(*s_red)[HG][4] = reinterpret_cast<float2(*)[HG][4]>(smem + L::red);
  float(*s_q)[HN] = reinterpret_cast<float(*)[HN]>(smem + L::sq);
  float2(*s_sc)[8] = reinterpret_cast<float2(*)[8]>(smem + L::sc);
  Piece8 *s_piece = reinterpret_cast<Piece8 *>(smem + L::desc);
  float(*s_ref)[2][HG] = reinterpret_cast<float(*)[2][HG]>(smem + L::ref);
  float(*s_sum)[4] = reinterpret_cast<float(*)[4]>(smem + L::sum);
  int *s_nan = reinterpret_cast<int *>(smem + L::nan);  // see the tail tiles
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const uint32_t base = smem_u32(smem);
  if (base & 1023) {
    if (tid == 0) p.errors[blockIdx.x] = -5;
    return;
  }
  if (tid == 0) *abort_flag = *status = 0;
  if (tid < L::nbars) {
    mbar_init(&bar[tid], tid == B_P ? 4 * G : tid >= B_SC && tid < B_FULL ? 32 : 1);
    fence_mbar_init();
  }
  if (warp == 4 * G) {
    tmem_alloc(tslot, L::cols);
    tmem_relinquish();
  }
  // columns that no thread writes
#pragma unroll 1
  for (uint32_t i = tid; i < (L::sc - L::q) / 16; i += L::threads) st_shared_v4(base + L::q + 16 * i, 0, 0, 0, 0);
  for (int i = tid; i < D; i += L::threads) s_nan[i] = 0x7fffffff;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);  // S of the even and odd tiles: 0, NS; O: 2 NS
  griddep_wait();
  auto wait = [&](int i, int parity) {
    return __all_sync(0xffffffffu, mbar_wait_short(&bar[i], parity & 1, abort_flag));
  };
  // the piece k, nh = 0: there are no more
  auto piece = [&](int k, Piece8 &x) {
    if (!wait(B_D + k % kPieces, k / kPieces)) return false;
    x = s_piece[k % kPieces];
    return true;
  };
  if (warp == 4 * G + 1) {
    // ------------------------------------------------------------ pieces, tiles and scales
    // Lane j < 8 has the tile's tokens 16 j ..: their page, and their scales; every box / 16 th such lane copies a box.
    // A published piece and a tile's scales are overwritten 16 pieces and 8 tiles later: a tile is loaded into a slot
    // that an earlier one's product has left, at most 6 tiles before, and that product came after the softmax of the tile
    // two before it; a piece is published before the tiles of the one before it are loaded.
    int n = 0, i = 0, k = 0;
    bool ok = true;
    Walk8 w;
    bool more = w.start(p);
    const uint64_t policy = p.slices > 1 ? kPolicyEvictNormal : kPolicyEvictFirst;  // more slices: read again
    const bool boxes = (lane * kScaleTokens & (box - 1)) == 0;  // (a power of two)
    const int step = block_of(p, kTile), rest = kTile - step * p.page;
    // this lane's tokens of a tile: the block of the sequence's table and the slot; the page's id is fetched a tile ahead
    struct Place {
      int tok, block, slot, id;
    };
    auto fetch = [&](const Walk8 &x, Place &a) {
      a.id = lane < 8 && a.tok < x.len ? p.table[(int64_t)x.b * p.tstride + a.block] : -1;
    };
    auto place = [&](const Walk8 &x) {
      Place a;
      a.tok = x.t0 * kTile + lane * kScaleTokens;
      a.block = block_of(p, a.tok);
      a.slot = a.tok - a.block * p.page;
      fetch(x, a);
      return a;
    };
    auto advance = [&](const Walk8 &x, Place &a) {
      a.tok += kTile;
      a.block += step;
      a.slot += rest;
      if (a.slot >= p.page) {
        a.slot -= p.page;
        ++a.block;
      }
      fetch(x, a);
    };
    if (lane == 0 && !p.by_item) p.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    // Tile t of piece w; behind its first tile's loads the piece after it is looked up and published, so that its queries
    // come early (the first piece before any).
    Place to{}, first{};
    Walk8 ahead = w;
    int t = 0;
    bool begun = false;
#pragma unroll 1
    while (ok) {
      if (begun) {
        const Place now = to;
        const bool in = now.id >= 0 && now.id < p.pages, copy = in && boxes;
        if (!in && lane < 8 && now.tok < w.len) report_error(status, -1);
        if (t + 1 < w.t1) advance(w, to);
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, copy)) * box * D;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int s = n % kRing;
          if (n >= kRing && !(ok = wait(B_EMPTY + s, n / kRing - 1))) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar[B_FULL + s], bytes);
          __syncwarp();
          if (copy)
            tma_load_4d(kv ? &mv : &mk, &bar[B_FULL + s], smem + s * L::tile + lane * kScaleTokens * D, 0, now.slot, w.it.hk,
                        now.id, policy);
          if (kv == 0) {
            if (lane < 8)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(&s_sc[i % L::nsc][lane])),
                           "l"(in ? reinterpret_cast<const float2 *>(p.scales + w.it.hk * p.ssh + now.id * p.ssb +
                                                                     now.slot / kScaleTokens * 2)
                                  : &kAbsent)
                           : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&bar[B_SC + i % L::nsc]))
                         : "memory");
          }
        }
        ++i;
      }
      if (!begun || t == w.t0) {
        if (begun) {
          if (lane == 0) record_piece(p, w, k - 1);
          ahead = w;
        }
        if ((more = more && ahead.next(p))) first = place(ahead);
        if (lane == 0) {
          s_piece[k % kPieces] = {ahead.b, ahead.it.hk, ahead.it.h0, more ? ahead.it.nh : 0, ahead.t0, ahead.t1, ahead.nt, ahead.len};
          mbar_arrive(&bar[B_D + k % kPieces]);
        }
        ++k;
      }
      if (begun && ++t < w.t1) continue;
      if (!more) break;
      begun = true;
      w = ahead;
      to = first;
      t = w.t0;
    }
    // what is in flight lands before the block ends (a wait with a limit, also after an abort)
    asm volatile("cp.async.wait_all;" ::: "memory");
    volatile int no_abort = 0;
#pragma unroll 1
    for (int s = 0; s < kRing; ++s) {
      const int uses = n > s ? (n - 1 - s) / kRing + 1 : 0;
      if (uses && lane == 0) mbar_wait(&bar[B_FULL + s], (uses - 1) & 1, &no_abort, status);
    }
    __syncwarp();
  } else if (warp == 4 * G + 2) {
    // ------------------------------------------------------------ queries: a lane cuts 8 values of a row into parts
    constexpr int kPer = D / 8, kIter = HN * kPer / 32;
    Piece8 x;
#pragma unroll 1
    for (int k = 0; piece(k, x) && x.nh; ++k) {
      uint4 v[kIter];
#pragma unroll
      for (int j = 0; j < kIter; ++j) {
        const int h = (j * 32 + lane) / kPer, c = lane % kPer;
        v[j] = make_uint4(0, 0, 0, 0);
        if (h < x.nh) {
          const int r = x.h0 + h, head = row_head(p, r);
          v[j] = *reinterpret_cast<const uint4 *>(q + (x.b * p.qsb + head * p.qsh + (r - head * p.T) * p.qst + 8 * c));
        }
      }
      if (k >= 2 && !wait(B_QE + (k & 1), (k >> 1) - 1)) break;
      const uint32_t Q = base + L::q + (k & 1) * L::qbuf;
      // with 16 rows two side by side, whose shuffles overlap (128 sequences of up to 1500, 16 rows: 31.4 -> 30.4 us; with 8 the
      // code costs more, 48.1 -> 48.9 at 256 of up to 500)
      constexpr int kPair = HN > 8 ? 2 : 1;
#pragma unroll 1
      for (int j = 0; j < kIter; j += kPair) {  // (one body: v moves down)
        const int c = lane % kPer;
        uint32_t top[kPair], one[kPair][2], two[kPair][2];
#pragma unroll
        for (int y = 0; y < kPair; ++y) {
          top[y] = 0;
#pragma unroll
          for (int z = 0; z < 4; ++z)
            top[y] = max(top[y], max((&v[y].x)[z] & 0x7fff0000u, (&v[y].x)[z] << 16 & 0x7fff0000u));
        }
#pragma unroll
        for (int x = kPer / 2; x; x /= 2)
#pragma unroll
          for (int y = 0; y < kPair; ++y) top[y] = max(top[y], __shfl_xor_sync(0xffffffffu, top[y], x));
#pragma unroll
        for (int y = 0; y < kPair; ++y) {
          const bool bad = top[y] >= 0x7f800000u;  // the row's scores are NaN then
          const int h = ((j + y) * 32 + lane) / kPer, e = scale_exponent(bad ? 0 : top[y]);
          const float inv = exp2i(-e);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t u0 = (&v[y].x)[2 * z], u1 = (&v[y].x)[2 * z + 1];
            const uint32_t a = f16x2(bf16lo(u0) * inv, bf16hi(u0) * inv), b = f16x2(bf16lo(u1) * inv, bf16hi(u1) * inv);
            const uint32_t a1 = e4m3x2(a), b1 = e4m3x2(b);
            one[y][z] = bad ? 0 : a1 | b1 << 16;
            two[y][z] = bad ? 0 : e4m3x2(left16(a, a1)) | e4m3x2(left16(b, b1)) << 16;
          }
          if (c == 0) s_q[k % kPieces][h] = bad ? __uint_as_float(0x7fc00000u) : exp2i(e) * (p.scale * 1.4426950408889634f);
        }
#pragma unroll
        for (int y = 0; y < kPair; ++y) {
          const int h = ((j + y) * 32 + lane) / kPer;
          st_shared_v2(Q + chunk_at<D>(h, c >> 1) + (c & 1) * 8, one[y][0], one[y][1]);
          st_shared_v2(Q + chunk_at<D>(HN + h, c >> 1) + (c & 1) * 8, two[y][0], two[y][1]);
        }
#pragma unroll
        for (int z = 0; z + kPair < kIter; ++z) v[z] = v[z + kPair];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar[B_QF + (k & 1)]);
        mbar_arrive(&bar[B_SQ + k % kPieces]);
      }
    }
    empty_rows<D>(p, o, lse, lane);
  } else if (warp == 4 * G) {
    // ------------------------------------------------------------ products
    const uint32_t id_qk = idesc_e4m3(0, 128, L::NS, false, false), id_pv = idesc_e4m3(1, 128, L::NO, true, true);
    // Scores run a tile ahead of the weighted sums, across pieces too.  i: the tile of the scores, of piece k, t behind
    // the tiles that are issued; first: whether it is a piece's first, and the tile's before
    bool more = true, first = false, before;
    int k = -1, t = 0, n = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
      before = first;
      if (t == n) {
        Piece8 x;
        if (!piece(++k, x)) break;
        more = x.nh;
        t = 0;
        n = x.t1 - x.t0;
      }
      if (more) {
        const int s = (2 * i) % kRing;
        first = t == 0;
        if (first && !wait(B_QF + (k & 1), k >> 1)) break;
        if (!wait(B_FULL + s, 2 * i / kRing)) break;
        tc_fence_after();
#pragma unroll
        for (uint32_t ks = 0; ks < D / 32; ++ks)
          mma_codes_warp(tmem + (i & 1) * L::NS, desc_rows<D>(base + s * L::tile, ks),
                        desc_rows<D>(base + L::q + (L::scol ? 0 : (k & 1) * L::qbuf), ks), id_qk, ks > 0);
        mma_commit_warp(&bar[B_S + (i & 1)]);
        mma_commit_warp(&bar[B_EMPTY + s]);
        if (++t == n) mma_commit_warp(&bar[B_QE + (k & 1)]);
      }
      if (i > 0) {
        const int j = i - 1, s = (2 * j + 1) % kRing;
        if (!wait(B_FULL + s, (2 * j + 1) / kRing) || !wait(B_P, j)) break;
        tc_fence_after();
#pragma unroll
        for (uint32_t ks = 0; ks < 4; ++ks)  // P: 16 columns (bytes) of a token side by side, 128 tokens; then the next 16
          mma_codes_warp(tmem + 2 * L::NS, desc_cols<D>(base + s * L::tile, ks), sdesc(base + L::p + ks * 512, 128, 2048, 0),
                        id_pv, !before || ks > 0);
        mma_commit_warp(&bar[B_O]);
        mma_commit_warp(&bar[B_EMPTY + s]);
      }
      if (!more) break;
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int gr = warp >> 2, h0 = gr * HG;  // group; its first row
    const uint32_t lt = tid & 127, t4 = tmem + ((uint32_t)((warp & 3) * 32) << 16), O = t4 + 2 * L::NS + gr * 24;
    bool dead = false;  // a wait gave up: a piece goes on without waiting, so that the barriers stay even
    auto await = [&](int i, int parity) {
      if (!dead) dead = !wait(i, parity);
    };
    int i = 0, slot = 0;  // tiles before
    Piece8 w;
#pragma unroll 1
    for (int k = 0;; ++k) {
      await(B_D + k % kPieces, k / kPieces);
      if (!dead) w = s_piece[k % kPieces];
      if (!dead && w.nh) await(B_SQ + k % kPieces, k / kPieces);
      if (!group_all(!dead, 3, 128 * G) || !w.nh) break;  // one verdict
      // in lane h row h's m (kNone before the first token) and log2 r; all rows' -m and r; this thread's sums
      float l[HG], my_mu = kNone, my_lr = 0.f;
      const float *refs = s_ref[gr][0];
#pragma unroll
      for (int h = 0; h < HG; ++h) l[h] = 0.f;
      const int partly = w.len - p.T + 1;  // the first token that not every row sees
      const int hr = row_head(p, w.h0 + h0), tr = w.h0 + h0 - hr * p.T;  // head and new token of the first row
      int tok = w.t0 * kTile + lt;
#pragma unroll 1
      for (int t = w.t0; t < w.t1; ++t, ++i, tok += kTile) {
        await(B_SC + i % L::nsc, i / L::nsc);
        await(B_S + (i & 1), i >> 1);
        tc_fence_after();
        const float2 sc = s_sc[i % L::nsc][lt / kScaleTokens];
        const bool valid = tok < w.len && !(sc.y < 0.f);
        const float ks = sc.x, vs = valid ? sc.y : 0.f;
        float x[HG];
        {
          constexpr int kPart = HG;
          uint32_t s[2 * kPart];
          if constexpr (HG == 4) {
            tmem_ld8(t4 + (i & 1) * L::NS + (k & 1) * L::scol, s);
          } else if constexpr (G == 1) {
            tmem_ld16(t4 + (i & 1) * L::NS, s);
          } else {
            tmem_ld8(t4 + (i & 1) * L::NS + h0, reinterpret_cast<uint32_t(&)[8]>(s));
            tmem_ld8(t4 + (i & 1) * L::NS + HN + h0, reinterpret_cast<uint32_t(&)[8]>(s[8]));
          }
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < HG; ++h)
            x[h] = max_nan(fmaf(__uint_as_float(s[kPart + h]), 0.0625f, __uint_as_float(s[h])) * ks * s_q[k % kPieces][h0 + h],
                           kFirst);
        }
        // from here on a score of -inf says that the row does not see the token
        const bool tail = p.T > 1 && (t + 1) * kTile > partly;
        if (tail) {
          int y = tr;
#pragma unroll
          for (int h = 0; h < HG; ++h) {
            if (tok >= partly + y) x[h] = -INFINITY;
            y = y + 1 == p.T ? 0 : y + 1;
          }
        }
#pragma unroll
        for (int h = 0; h < HG; ++h)
          if (!valid) x[h] = -INFINITY;
        // the exponentials and the weights, two rows a word; where they leave their range, and in the first tile, the references
        // move before
        float e[HG];
        uint32_t wt[HG / 2];
#pragma unroll 1
        for (bool move = t == w.t0;; move = true) {
          if (move) {
            // the warp's largest score, and the largest of score + log2 scale behind that score
            const float lv = lg2(vs);
#pragma unroll
            for (int h = 0; h < HG; ++h) {
              const float xw = warp_max(x[h]), jw = warp_max((x[h] - xw) + lv);
              if (lane == 0) s_red[gr][h][warp & 3] = make_float2(xw, jw);
            }
            named_bar_sync(1 + gr, 128);
            // lane h: row h
            const float4 v0 = *reinterpret_cast<const float4 *>(s_red[gr][lane % HG]),
                         v1 = *reinterpret_cast<const float4 *>(s_red[gr][lane % HG] + 2);
            const float xm = fmaxf(fmaxf(v0.x, v0.z), fmaxf(v1.x, v1.z));
            const float m = xm > my_mu + 8.f ? fmaxf(xm, kFloor) : my_mu;
            // (what is not there is -inf or NaN, which the maxima leave out)
            const float j = fmaxf(fmaxf(v0.y + (v0.x - m), v0.w + (v0.z - m)), fmaxf(v1.y + (v1.x - m), v1.w + (v1.z - m)));
            float lr = my_lr + (m - my_mu);  // (O as it is)
            if (j + lr > 15.f) lr = 11.f - j;
            lr = fminf(fmaxf(lr, -120.f), 120.f);
            const float f = ex2(my_mu - m), g = ex2((my_mu - m) + (lr - my_lr)), now = ex2(lr);  // (f 0 from kNone)
            my_mu = m;
            my_lr = lr;
            if (lane < HG) {  // (every warp the same values; the last reads of the ones before were before the barrier)
              s_ref[gr][0][lane] = -m;
              s_ref[gr][1][lane] = now;
            }
            __syncwarp();
            if (t > w.t0) {  // O (lane = value dimension) to the new references
              await(B_O, i - 1);
              tc_fence_after();
              float y[HG];
#pragma unroll
              for (int h = 0; h < HG; ++h) {
                l[h] *= __shfl_sync(0xffffffffu, f, h);
                y[h] = __shfl_sync(0xffffffffu, g, h);
              }
#pragma unroll 1
              for (int z = 0; z < 3; ++z) {
                if constexpr (HG == 4) {
                  uint32_t a[4];
                  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                               : "r"(O + 4 * z));
                  tmem_ld_wait();
#pragma unroll
                  for (int h = 0; h < 4; ++h) a[h] = __float_as_uint(__uint_as_float(a[h]) * y[h]);
                  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(O + 4 * z), "r"(a[0]),
                               "r"(a[1]), "r"(a[2]), "r"(a[3])
                               : "memory");
                } else {
                  uint32_t a[8];
                  tmem_ld8(O + 8 * z, a);
                  tmem_ld_wait();
#pragma unroll
                  for (int h = 0; h < 8; ++h) a[h] = __float_as_uint(__uint_as_float(a[h]) * y[h]);
                  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(O + 8 * z),
                               "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
                               : "memory");
                }
              }
              tmem_st_wait();
            }
          }
          float most = 0.f;
          uint32_t top = 0;
#pragma unroll
          for (int h = 0; h < HG; h += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(refs + h), r = *reinterpret_cast<const float4 *>(refs + HG + h);
            const float2 d0 = add2(make_float2(x[h], x[h + 1]), make_float2(m.x, m.y)),
                         d1 = add2(make_float2(x[h + 2], x[h + 3]), make_float2(m.z, m.w));
            e[h] = ex2(d0.x), e[h + 1] = ex2(d0.y), e[h + 2] = ex2(d1.x), e[h + 3] = ex2(d1.y);
            const float2 v = make_float2(vs, vs), w0 = mul2(mul2(make_float2(e[h], e[h + 1]), v), make_float2(r.x, r.y)),
                         w1 = mul2(mul2(make_float2(e[h + 2], e[h + 3]), v), make_float2(r.z, r.w));
            wt[h / 2] = f16x2(w0.x, w0.y);
            wt[h / 2 + 1] = f16x2(w1.x, w1.y);
            top = max_f16x2(top, max_f16x2(wt[h / 2], wt[h / 2 + 1]));
            most = max3(max3(most, e[h], e[h + 1]), e[h + 2], e[h + 3]);
          }
          // (the upper and the lower half against 2^15 = 0x7800: they are not negative)
          if (move || !group_any(most > 256.f || top >= 0x78010000u || (top & 0xffffu) > 0x7800u, 1 + gr, 128)) break;
        }
        // their parts: a word per part and four rows
        uint32_t pt[3][HG / 4];
#pragma unroll
        for (int h = 0; h < HG; ++h) l[h] += e[h];
#pragma unroll
        for (int h = 0; h < HG; h += 4) {
          const uint32_t a = wt[h / 2], b = wt[h / 2 + 1];
          const uint32_t a1 = e5m2x2(a), b1 = e5m2x2(b), ra = left16_e5m2(a, a1), rb = left16_e5m2(b, b1);
          const uint32_t a2 = e5m2x2(ra), b2 = e5m2x2(rb);
          pt[0][h / 4] = a1 | b1 << 16;
          pt[1][h / 4] = a2 | b2 << 16;
          pt[2][h / 4] = e5m2x2(left16_e5m2(ra, a2)) | e5m2x2(left16_e5m2(rb, b2)) << 16;
        }
        if (i >= 1) await(B_O, i - 1);  // P of the tile before has been read
        const uint32_t P = base + L::p + lt * 16;
        if constexpr (HG == 4) {
          st_shared_v4(P, pt[0][0], pt[1][0], pt[2][0], 0);
        } else if (gr == 0) {
          st_shared_v4(P, pt[0][0], pt[0][1], pt[1][0], pt[1][1]);
          st_shared_v2(P + 2048, pt[2][0], pt[2][1]);
        } else {
          st_shared_v2(P + 2048 + 8, pt[0][0], pt[0][1]);
          st_shared_v4(P + 4096, pt[1][0], pt[1][1], pt[2][0], pt[2][1]);
        }
        // Value rows that no weight may meet: 0 x NaN is NaN.  Those of absent tokens are cleared; NaN codes of tokens
        // that some rows see and some do not are cleared and kept in mind by their dimension, as the first such
        // token's distance behind `partly`: row t of T sees it when that is less than t.
        const bool some = tail && valid && tok >= partly;
        if (!__all_sync(0xffffffffu, valid && !some) && gr == 0) {
          const int s = (2 * i + 1) % kRing;
          await(B_FULL + s, (2 * i + 1) / kRing);
          const uint32_t V = base + s * L::tile;
          if (!valid) {
#pragma unroll
            for (uint32_t y = 0; y < D / 16; ++y) st_shared_v4(V + lt * D + y * 16, 0, 0, 0, 0);  // (the swizzle stays in a row)
          } else if (some) {
#pragma unroll 1
            for (uint32_t y = 0; y < D / 16; ++y) {
              const uint32_t at = V + chunk_at<D>(lt, y);
              uint32_t u[4], found = 0;
              ld_shared_v4(at, u[0], u[1], u[2], u[3]);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint32_t nan = __vcmpeq4(u[z] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                for (int byte = 0; nan && byte < 4; ++byte)
                  if (nan >> 8 * byte & 1) atomicMin(&s_nan[y * 16 + z * 4 + byte], tok - partly);
                u[z] &= ~nan;
                found |= nan;
              }
              if (found) st_shared_v4(at, u[0], u[1], u[2], u[3]);
            }
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_P]);
      }
      // the sums over all tokens of the piece: the rows are halved over the lanes
      halve_heads<HG / 2, 16>(l, lane);
#pragma unroll
      for (int y = 16 / HG; y; y /= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], y);
      if (lane % (32 / HG) == 0) s_sum[h0 + lane / (32 / HG)][warp & 3] = l[0];
      await(B_O, i - 1);
      named_bar_sync(3, 128 * G);
      tc_fence_after();
      uint32_t a[24];
      if constexpr (HG == 4) {
        tmem_ld16(O, reinterpret_cast<uint32_t(&)[16]>(a));
      } else {
        tmem_ld8(O, reinterpret_cast<uint32_t(&)[8]>(a));
        tmem_ld8(O + 8, reinterpret_cast<uint32_t(&)[8]>(a[8]));
        tmem_ld8(O + 16, reinterpret_cast<uint32_t(&)[8]>(a[16]));
      }
      tmem_ld_wait();
      tc_fence_before();
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      const uint32_t at = (2 * blockIdx.x + slot) * HN + h0;  // the row in part and ml
      // lane h of every warp: row h's sum, whether it has seen a token, and what its output is multiplied by
      const int row = lane < HG ? lane : 0;
      const float4 sums = *reinterpret_cast<const float4 *>(s_sum[h0 + row]);
      const float sum = (sums.x + sums.y) + (sums.z + sums.w), m = my_mu;
      const bool none = m == kNone && sum == 0.f;
      const float over_r = ex2(-my_lr), factor = whole ? __fdividef(over_r, sum) : over_r;
      const uint32_t nothing = __ballot_sync(0xffffffffu, none);
      if ((int)lt < HG && h0 + (int)lt < w.nh) {
        if (!whole) *reinterpret_cast<float2 *>(ml + (at + lt) * 2) = make_float2(none ? -INFINITY : m, sum);
        else if (lse)
          lse[(int64_t)w.b * p.Hq * p.T + w.h0 + h0 + lt] = none ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
      }
      const int bad_from = p.T > 1 && (int)lt < D ? s_nan[lt] : 0x7fffffff;
      __nv_bfloat16 *to = o + (w.b * p.qsb + hr * p.qsh + tr * p.qst + lt);
      float *to_part = part + at * D + lt;
      const int64_t next_token = p.qst, next_head = p.qsh - (p.T - 1) * p.qst;
      int y = tr;
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        float acc = fmaf(fmaf(__uint_as_float(a[2 * HG + h]), 0.0625f, __uint_as_float(a[HG + h])), 0.0625f,
                         __uint_as_float(a[h])) *
                    __shfl_sync(0xffffffffu, factor, h);
        if (bad_from < y) acc = __uint_as_float(0x7fc00000u);
        if (nothing >> h & 1) acc = 0.f;
        if ((int)lt < D && h0 + h < w.nh) {
          if (whole) *to = __float2bfloat16_rn(acc);
          else to_part[h * D] = acc;
        }
        to += y + 1 == p.T ? next_head : next_token;
        y = y + 1 == p.T ? 0 : y + 1;
      }
      slot = 1;
      if (p.T > 1) {
        named_bar_sync(3, 128 * G);
        for (int z = tid; z < D; z += 128 * G) s_nan[z] = 0x7fffffff;
      }
      // (s_sum and s_nan are written again behind the next piece's first barrier)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * G) tmem_dealloc(tmem, L::cols);
  if (tid == 0) p.errors[blockIdx.x] = *status;
}

// ------------------------------------------------------------------ join
// A CTA per record and kRows rows of its item: joins the item that one CTA of the decode began and others finished,
// o = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i.  A thread has four dimensions of a row and every
// kParts-th piece.  The pieces after the first are their CTAs' first (slot 0).  A CTA without work costs half as much as one
// with a few pieces, so there is one per item where items are fewer than the decode's CTAs.
template <int D, int HN, int kRows, typename T>
__global__ void __launch_bounds__(512, 1) paged_join_q8(PagedProblem p, T *o, float *lse, const float *part, const float *ml,
                                                        int ctas) {
  constexpr int kQuads = kRows * D / 4, kParts = 512 / kQuads;
  __shared__ float4 s_acc[kParts][kQuads];
  __shared__ float2 s_ml[kParts][kRows];
  griddep_wait();
  if (blockIdx.x == gridDim.x - 1) {  // one more than there are records: the status word
    if (blockIdx.y) return;
    int e = 0;
    for (int g = threadIdx.x; g < ctas; g += 512) e = e ? e : p.errors[g];
    const int any = __syncthreads_or(e);
    if (any ? e : threadIdx.x == 0) *p.status = e;  // (of several any)
    return;
  }
  // sequence, first row, rows + 256 times the slot of the first piece, its CTA + 2^16 times the pieces after it
  const int4 r = p.rec[blockIdx.x];
  const int r0 = kRows * blockIdx.y, rows = r.z & 255, from = r.w & 0xffff, more = r.w >> 16;
  if (r.x < 0 || r0 >= rows) return;
  // (a record that a block did not come to write, because a wait gave up, holds anything)
  if (r.x >= p.B || rows > HN || r.y < 0 || r.y > p.Hq * p.T - rows || more < 0 || from + more >= ctas) return;
  const int tid = threadIdx.x, y = tid / kQuads, e = tid % kQuads, h = e / (D / 4), c = e % (D / 4);
  auto at = [&](int g, int row) { return (2 * (from + g) + (g ? 0 : r.z >> 8 & 1)) * HN + r0 + row; };
  float m = -INFINITY, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float mz, float lz, float4 x) {
    const float mn = fmaxf(m, mz), use = mn == -INFINITY ? 0.f : mn, f0 = exp2f(m - use), f1 = exp2f(mz - use);
    a = make_float4(f0 * a.x + f1 * x.x, f0 * a.y + f1 * x.y, f0 * a.z + f1 * x.z, f0 * a.w + f1 * x.w);
    l = f0 * l + f1 * lz;
    m = mn;
  };
  if (r0 + h < rows)
#pragma unroll 1
    for (int g = y; g <= more; g += 4 * kParts) {
      float2 v[4];
      float4 x[4];
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (g + z * kParts <= more) {
          v[z] = *reinterpret_cast<const float2 *>(ml + at(g + z * kParts, h) * 2);
          x[z] = *reinterpret_cast<const float4 *>(part + at(g + z * kParts, h) * D + 4 * c);
        }
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (g + z * kParts <= more) add(v[z].x, v[z].y, x[z]);
    }
  s_acc[y][e] = a;
  if (c == 0) s_ml[y][h] = make_float2(m, l);
  __syncthreads();
  if (y || r0 + h >= rows) return;
#pragma unroll
  for (int z = 1; z < kParts; ++z) add(s_ml[z][h].x, s_ml[z][h].y, s_acc[z][e]);
  if (m == -INFINITY) l = 1.f;  // no piece had a token
  T *to = o + row_at(p, r.x, r.y + r0 + h) + 4 * c;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2 *>(to) =
        make_uint2(pack_bf16(__fdividef(a.x, l), __fdividef(a.y, l)), pack_bf16(__fdividef(a.z, l), __fdividef(a.w, l)));
  else
    *reinterpret_cast<float4 *>(to) = make_float4(a.x / l, a.y / l, a.z / l, a.w / l);
  if (lse && c == 0)
    lse[(int64_t)r.x * p.Hq * p.T + r.y + r0 + h] = m == -INFINITY ? m : (m + log2f(l)) * 0.6931471805599453f;
}

// The decode by `launch` (grid, pieces, maxima and sums) with up to per_sm CTAs an SM and HN rows of an item, and the join.
template <int D, int HN, typename T, typename Launch>
cudaError_t run_and_join(PagedProblem p, int per_sm, T *o, float *lse, void *ws, cudaStream_t s, Launch launch) {
  const int G = paged_grid(p, per_sm);
  p.group = p.Hq / p.Hkv * p.T;
  p.slices = (p.group + kHeads - 1) / kHeads;
  const int64_t items = (int64_t)p.B * p.Hkv * p.slices;
  // (the pieces of G CTAs, two of up to HN rows each, are within the rows that paged_decode_ws_bytes counts)
  float *part = static_cast<float *>(ws), *ml = part + (size_t)2 * (2 * p.num_sms) * kHeads * D;
  p.rec = reinterpret_cast<int4 *>(ml + (size_t)2 * (2 * p.num_sms) * kHeads * 2);
  p.errors = reinterpret_cast<int *>(p.rec + 4 * p.num_sms);
  p.by_item = items <= G;
  p.items = p.Hkv * p.slices;
  {
    TimedLaunch t(K_PAGED_DECODE8, s);
    cudaError_t e = launch(p, G, part, ml);
    if (e != cudaSuccess) return e;
  }
  TimedLaunch t(K_PAGED_JOIN, s);
  // Four rows a CTA, or where an item has many pieces, all of which a row's CTA reads, one: with 32 pieces an item 8.0 us instead of
  // 8.4 (B1 H16/4, 4000 tokens), with 304 17.2 instead of 25.0 (B1 H16/1, 100000), with 16 8.1 instead of 7.6 (B4 H16/4 2000).
  const bool single = G >= 32 * items;
  auto join = [&](auto k, int rows) {
    return launch_overlapped(k, dim3((p.by_item ? items : G) + 1, HN / rows), dim3(512), 0, s, p, o, lse, (const float *)part,
                             (const float *)ml, G);
  };
  return single ? join(paged_join_q8<D, HN, 1, T>, 1) : join(paged_join_q8<D, HN, 4, T>, 4);
}

template <int D, int HN>
cudaError_t run_q8_tc(const PagedProblem &p, const CUtensorMap &mk, const CUtensorMap &mv, int box, const void *q, void *o,
                      float *lse, void *ws, cudaStream_t s) {
  using L = Layout8<D, HN>;
  using bf16 = __nv_bfloat16;
  static_assert(L::per_sm * HN <= 2 * kHeads && L::per_sm <= 4, "an SM's pieces and records");
  auto kernel = paged_decode_q8_tc<D, HN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::smem);
  if (e != cudaSuccess) return e;
  return run_and_join<D, HN>(p, L::per_sm, (bf16 *)o, lse, ws, s, [&](const PagedProblem &p, int G, float *part, float *ml) {
    return launch_overlapped(kernel, dim3(G), dim3(L::threads), L::smem, s, mk, mv, box, p, (const bf16 *)q, (bf16 *)o, lse,
                             part, ml);
  });
}

template <int D, int HN>
cudaError_t run_q8_simt(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse, void *ws,
                        cudaStream_t s) {
  constexpr size_t smem = SimtLayout<D, HN, true>::smem;
  static_assert(kSimtPerSm * HN <= 2 * kHeads, "an SM's pieces");
  auto kernel = paged_decode_simt<D, HN, true>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return run_and_join<D, HN>(p, kSimtPerSm, (float *)o, lse, ws, s, [&](const PagedProblem &p, int G, float *part, float *ml) {
    return launch_overlapped(kernel, dim3(G), dim3(kSimtThreads), smem, s, p, (const float *)q, (const uint8_t *)kc,
                             (const uint8_t *)vc, (float *)o, lse, part, ml);
  });
}

template <int D>
cudaError_t run_q8(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse, void *ws,
                   cudaStream_t s) {
  const int rows = p.Hq / p.Hkv * p.T;
  if (p.esz == 4)
    return rows <= 4   ? run_q8_simt<D, 4>(p, q, kc, vc, o, lse, ws, s)
           : rows <= 8 ? run_q8_simt<D, 8>(p, q, kc, vc, o, lse, ws, s)
                       : run_q8_simt<D, 16>(p, q, kc, vc, o, lse, ws, s);
  // the rows of one copy: the largest power of two up to 128 that divides a page (a multiple of 16), so that a copy stays
  // inside a page and starts on the swizzle's pattern
  int box = p.page & -p.page;
  box = box > kTile ? kTile : box;
  CUtensorMap mk{}, mv{};
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.page, (uint64_t)p.Hkv, (uint64_t)p.pages};
  const uint64_t strides[3] = {(uint64_t)p.cst, (uint64_t)p.csh, (uint64_t)p.csb};
  if (!make_tmap_u8(&mk, kc, dims, strides, D, box) || !make_tmap_u8(&mv, vc, dims, strides, D, box))
    return cudaErrorInvalidValue;
  return rows <= 4   ? run_q8_tc<D, 4>(p, mk, mv, box, q, o, lse, ws, s)
         : rows <= 8 ? run_q8_tc<D, 8>(p, mk, mv, box, q, o, lse, ws, s)
                     : run_q8_tc<D, 16>(p, mk, mv, box, q, o, lse, ws, s);
}

}  // namespace

cudaError_t paged_append_q8(const PagedProblem &p, const void *k, const void *v, void *kc, void *vc, int T, int64_t sb,
                            int64_t sh, int64_t st, const int *start, const int *new_lens, cudaStream_t s) {
  TimedLaunch t(K_PAGED_APPEND8, s);
  // blocks that T tokens can touch
  const uint32_t nblocks = (uint32_t)(((int64_t)T + kScaleTokens - 2) / kScaleTokens + 1), warps = 2u * p.B * p.Hkv * nblocks;
  auto run = [&](auto kernel, auto *type) {
    using E = std::remove_pointer_t<decltype(type)>;
    return launch_overlapped(kernel, dim3((warps + 7) / 8), dim3(256), 0, s, p, (const E *)k, (const E *)v, (uint8_t *)kc,
                             (uint8_t *)vc, (uint32_t)T, start, new_lens, sb, sh, st, nblocks, warps);
  };
  using bf16 = __nv_bfloat16;
  if (p.esz == 2)
    return p.d == 64 ? run(paged_append_q8_kernel<64, bf16>, (bf16 *)0) : run(paged_append_q8_kernel<128, bf16>, (bf16 *)0);
  return p.d == 64 ? run(paged_append_q8_kernel<64, float>, (float *)0) : run(paged_append_q8_kernel<128, float>, (float *)0);
}

cudaError_t paged_gather_q8(const PagedProblem &p, const void *kc, const void *vc, void *k, void *v, int T, int64_t sb,
                            int64_t sh, int64_t st, const int *start, cudaStream_t s) {
  TimedLaunch t(K_PAGED_GATHER8, s);
  const uint32_t nblocks = (uint32_t)(((int64_t)T + kScaleTokens - 1) / kScaleTokens), warps = 2u * p.B * p.Hkv * nblocks;
  auto run = [&](auto kernel, auto *type) {
    using E = std::remove_pointer_t<decltype(type)>;
    return launch_overlapped(kernel, dim3((warps + 7) / 8), dim3(256), 0, s, p, (const uint8_t *)kc, (const uint8_t *)vc,
                             (E *)k, (E *)v, (uint32_t)T, start, sb, sh, st, nblocks, warps);
  };
  using bf16 = __nv_bfloat16;
  if (p.esz == 2)
    return p.d == 64 ? run(paged_gather_q8_kernel<64, bf16>, (bf16 *)0) : run(paged_gather_q8_kernel<128, bf16>, (bf16 *)0);
  return p.d == 64 ? run(paged_gather_q8_kernel<64, float>, (float *)0) : run(paged_gather_q8_kernel<128, float>, (float *)0);
}

cudaError_t paged_decode_q8(const PagedProblem &p, const void *q, const void *kc, const void *vc, void *o, float *lse,
                            void *ws, cudaStream_t s) {
  return p.d == 64 ? run_q8<64>(p, q, kc, vc, o, lse, ws, s) : run_q8<128>(p, q, kc, vc, o, lse, ws, s);
}

}  // namespace linattn
