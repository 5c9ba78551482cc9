// Gated delta rule on the tensor cores (bf16, d = 128; d = 64 as the zero-padded problem), by chunks
// of 64 tokens.  For one chunk, with g the cumulative log-gates inside it, Gam_ij = exp(g_i - g_j)
// (j <= i), b the write strengths, phi_j = exp(g_last - g_j) and S the state entering it:
//
//     Y  = T (V - diag(e^g) K S),   T = (I + tril(Gam * K K^T, -1) diag(b))^-1        (what each write
//     O  = diag(e^g) Q S + P diag(b) Y,   P = tril(Gam * Q K^T)                        corrects, y_t)
//     S' = e^(g_last) S + K^T diag(phi b) Y.
//
// T, W = -T diag(e^g) K and P do not involve the state, so one kernel forms them for all chunks at
// once (delta_prep); only Y = T V + W S and the update of S are a chain over the chunks, one CTA per
// (batch, head) and slice of value dimensions (delta_chain).  The backward runs the same chain in reverse time on R,
// the gradient at the state (delta_reverse), and then all gradients chunk by chunk (delta_grad):
//
//     dU  = P^T dO + diag(phi) K R,    Z = T^T diag(b) dU  (= dV),
//     R'  = e^(g_last) R + Q^T diag(e^g) dO + W^T diag(b) dU,
//     dQ  = diag(e^g) dO S^T + A K,      A_ij = b_j Gam_ij dO_i . y_j   (j <= i)
//     dK  = [ -diag(e^g) Z S^T + D K ] + [ diag(phi b) Y R^T + A^T Q + D^T K ],
//                                        D_ij = -b_j Gam_ij z_i . y_j   (j < i)
//     db_j = dU_j . y_j - sum_{i > j} Gam_ij (k_i . k_j) (z_i . y_j),
//     d(cumulative log-gate)_i = q_i . dq_i + k_i . [read part] - k_i . [write part].
//
// Precision: the state and every accumulator are fp32.  Operands of the chains that are not bf16 inputs
// (S, Y, W, T, P, R, dU) enter their products as two bf16 parts, hi + lo (16 significant bits): what a chain
// carries from chunk to chunk stays within about 2^-16 per step instead of 2^-8, so a final state is good for
// a decode that goes on for long (2.4e-6 to 4.4e-6 of exact at 777 to 8192 tokens, d_init_state alike; products
// of fp32 operands would leave 1.5e-7).  The gradient kernel's operands are single bf16 but for Y in dO Y^T and
// Y R^T and for A, which have two parts: its results are rounded to bf16 anyway, and gates' gradients that are
// returned in fp32 come from the same operands (0.3e-3 to 2.4e-3).
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace linattn {
namespace {

constexpr int kC = 64;                    // tokens of a chunk
constexpr uint32_t kSlot = 16384;         // a 64 x 128 (or 128 x 64) bf16 tile
// Warp numbers and tensor-memory addresses are taken by a shuffle from lane 0, which tells the compiler that they are
// the same in a whole warp: a role's products then find their operands in uniform registers, some 10 instructions
// each instead of 60 (B2 H16 T16384: chains 414 + 408 -> 388 + 384 us, gradients 366 -> 338).
// A chunk's record: W (64 x 128), T (64 x 64), P (64 x 64), each in two bf16 parts, as swizzled tiles
// ready for a plain bulk copy; then five fp32 rows of 64: e^g, phi, b, g and its low part (log2 units).
constexpr uint32_t kRecW = 0, kRecT = 32768, kRecP = 49152, kRecG = 65536, kGateBytes = 5 * 64 * 4;
constexpr size_t kRecBytes = 67584;
// P's parts are two tiles.  W and T are tiles of 128 rows: of every 16 tokens the hi rows, then the lo rows, so
// that one product of 128 rows takes both and their sums meet in one warp's lanes.
__device__ __forceinline__ uint32_t part_row(uint32_t token) { return 2 * (token & ~15u) + (token & 15u); }
constexpr uint32_t kPartLo = 16 * 128;  // from a hi row to its lo row
constexpr size_t kStateImg = 32768, kRowImg = 16384, kYImg = 2 * kRowImg;  // Y: hi, lo

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
// a and b as packed bf16 and what is left of them as packed bf16 (the difference of a pair in one
// packed instruction)
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(a, b);
  float x, y;
  asm("{\n\t.reg .b64 u, v, m;\n\t"
      "mov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 m, {%6, %6};\n\t"
      "fma.rn.f32x2 u, v, m, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(bf16lo(hi)), "f"(bf16hi(hi)), "f"(-1.f));
  lo = pack_bf16(x, y);
}
// offset of 16-byte piece c (0..7) of row r in a swizzled 64-column block
__device__ __forceinline__ uint32_t sw(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }
// Fragments of 16 rows x 16 columns (tmem_ld_frag): the place of lane l's address row for the four 8 x 8
// matrices, in a tile whose rows are the fragment's rows (columns 16 g .. of a 64-column block) ...
__device__ __forceinline__ uint32_t frag_at(uint32_t lane, uint32_t row0, uint32_t g) {
  return sw(row0 + (lane & 15u), 2 * g + (lane >> 4));
}
// ... and in one whose rows are the fragment's columns (row0 the first; its columns col0 .. + 15, blocks `half` apart)
__device__ __forceinline__ uint32_t frag_at_trans(uint32_t lane, uint32_t row0, uint32_t col0, uint32_t half) {
  const uint32_t c = (col0 >> 3) + ((lane >> 3) & 1u);
  return (c >> 3) * half + sw(row0 + (lane & 7u) + 8 * (lane >> 4), c & 7u);
}
// register i of a fragment belongs to the (i & 1) + (i & 4 ? 2 : 0)-th of the lane's four columns
__device__ __forceinline__ constexpr int frag_col(int i) { return (i & 1) | ((i >> 1) & 2); }
__device__ __forceinline__ uint32_t frag_token(uint32_t lane, int e) { return 2 * (lane & 3u) + (e & 1) + 8 * (e >> 1); }
__device__ __forceinline__ void frag_pack(const float (&x)[8], uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
}
// sum over the fragment's rows, for each of the lane's four columns (all lanes of equal l % 4 get it)
__device__ __forceinline__ void frag_col_sum(float (&x)[4]) {
#pragma unroll
  for (int o = 4; o < 32; o *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
}

// 8 packed words (16 columns) of row r, column group m of a swizzled block in global memory, as one 32-byte
// store: the swizzle moves pairs of pieces and, in odd rows, swaps a pair.
__device__ __forceinline__ uint32_t row8(uint32_t r, uint32_t m) { return r * 128u + ((m ^ ((r & 7u) >> 1)) << 5); }
__device__ __forceinline__ void store_row8(uint8_t *block, uint32_t r, uint32_t m, const uint32_t (&w)[8]) {
  const bool odd = r & 1u;
  uint8_t *dst = block + row8(r, m);
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = odd ? w[4 + e] : w[e];
    v[4 + e] = odd ? w[e] : w[4 + e];
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A sum of two fp32 parts, |lo| at most half a step of hi (sums by the error-free transformation of Knuth and
// Dekker's renormalisation).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)), __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s))};
}
__device__ __forceinline__ Two times_log2e(float x) {
  constexpr float c = 1.44269504f, d = 1.925963033e-8f;  // log2(e) as two fp32 parts
  const float hi = __fmul_rn(x, c);
  return {hi, __fmaf_rn(x, d, __fmaf_rn(x, c, -hi))};
}

struct DeltaTcParams {
  int H, T, N, d;          // N chunks; d = 64 or 128 (state rows and columns; the tiles are 128 wide)
  int f32;                 // type of the gates
  const void *lg, *beta;
  uint8_t *rec;            // [BH][N] records
  uint8_t *simg, *yimg;    // [BH][N] images of S entering the chunks, of Y in two parts (or null: not kept)
  uint8_t *rimg, *uimg;    // backward: [BH][N] images of R and of diag(b) dU
  float *dot;              // backward: [BH][N][64][8] parts of dU . y (16 value dimensions each)
  const float *in;         // initial state, or the final state's gradient (or null)
  float *out;              // final state, or the initial state's gradient (or null)
  float *anchor;           // backward: [BH][N] <R, S> at the chunks' ends
  float *gx;               // backward: [BH][T]
  void *dbeta;
  int *status;
};

__device__ __forceinline__ float load_gate(const void *p, int64_t i, int f32) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// ================================================================== prep
// One CTA per chunk: the stacked product [K; Q] K^T (lanes 0..63: K K^T, 64..127: Q K^T) on the tensor
// cores, the unit lower triangular inverse in fp32 on the CUDA cores (two 32 x 32 blocks, then the block
// below them; products in 4 x 4 tiles, since what bounds the kernel is what it reads from shared memory), and
// W^T = K^T (T diag(e^g))^T on the tensor cores.  Four CTAs fit an SM and hide each other's latencies: 192 us at
// B2 H16 T16384, 4.3 TB/s of what it reads and writes.
constexpr int kPrepThreads = 256;
constexpr int kLd = 68;  // row stride of the fp32 matrix T: 16-byte rows, spread over the banks
// The stacked tile [K; Q] (two blocks of 64 columns), then T.  A^T, later the parts of T diag(e^g), take the
// place of Q: rows 0..31 (the hi part) in the first block, the others in the second.
constexpr uint32_t kPrepA = 8192, kPrepT = 32768, kPrepEnd = kPrepT + kLd * 64 * 4;
constexpr size_t kPrepSmem = kPrepEnd + 1024;
static_assert(4 * (kPrepSmem + 2048) <= 232448, "four CTAs per SM (as the tensor memory has it)");

// A 4 x 4 tile of a product: one step of the contraction (a: four rows, u: four columns).
__device__ __forceinline__ void tile_fma(float4 (&acc)[4], const float4 &a, const float4 &u) {
  const float f[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    acc[e] = make_float4(fmaf(f[e], u.x, acc[e].x), fmaf(f[e], u.y, acc[e].y), fmaf(f[e], u.z, acc[e].z),
                         fmaf(f[e], u.w, acc[e].w));
}
// One halving step of a sum over lanes: lanes l and l ^ X keep N rows each of the sum of their 2 N rows.
template <int N, int X>
__device__ __forceinline__ void tile_halve(float4 (&acc)[4], int lane) {
  const bool up = lane & X;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float4 keep = up ? acc[e + N] : acc[e], send = up ? acc[e] : acc[e + N];
    acc[e] = make_float4(keep.x + __shfl_xor_sync(0xffffffffu, send.x, X), keep.y + __shfl_xor_sync(0xffffffffu, send.y, X),
                         keep.z + __shfl_xor_sync(0xffffffffu, send.z, X), keep.w + __shfl_xor_sync(0xffffffffu, send.w, X));
  }
}
// acc += A U and acc -= T U over 8 steps from m0: rows r0 .. + 3 of A (transposed, row stride 64) or T and
// columns c0 .. + 3 of U (both with row stride kLd).
__device__ __forceinline__ void tile_at(float4 (&acc)[4], const float *at, const float *u) {
#pragma unroll 1
  for (int m = 0; m < 8; m += 4, at += 4 * 64, u += 4 * kLd)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      tile_fma(acc, *reinterpret_cast<const float4 *>(at + e * 64), *reinterpret_cast<const float4 *>(u + e * kLd));
}
__device__ __forceinline__ void tile_minus(float4 (&acc)[4], const float *t, const float *u) {
#pragma unroll 1
  for (int m = 0; m < 8; m += 4, t += 4, u += 4 * kLd) {
    float4 r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = *reinterpret_cast<const float4 *>(t + e * kLd);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto at = [&](const float4 &x) { return e == 0 ? -x.x : e == 1 ? -x.y : e == 2 ? -x.z : -x.w; };
      tile_fma(acc, make_float4(at(r[0]), at(r[1]), at(r[2]), at(r[3])), *reinterpret_cast<const float4 *>(u + e * kLd));
    }
  }
}
// V (row stride kLd) = (I + A)^-1 for the strictly lower triangular 32 x 32 A, given transposed (row stride 64),
// by one warp: four 8 x 8 blocks by substitution, a column per lane, then twice the block below the diagonal,
// -T22 (A21 T11), with X = A21 T11 parked above the diagonal in between and zeroed after.
__device__ __forceinline__ void invert32(const float *A, float *V, int lane) {
  {
    const int o = lane & ~7, col = lane & 7;
    const float *a = A + o * 64 + o;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e == col ? 1.f : 0.f;
#pragma unroll
    for (int f = 0; f < 7; ++f) {
      const float4 x = *reinterpret_cast<const float4 *>(a + f * 64), y = *reinterpret_cast<const float4 *>(a + f * 64 + 4);
      const float c[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = f + 1; e < 8; ++e) v[e] = fmaf(-c[e], v[f], v[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) V[(o + e) * kLd + o + col] = v[e];
  }
  __syncwarp();
  {
    // 8 -> 16, both blocks at once: four outputs of a row per lane
    const int o = lane & 16, r = (lane & 15) >> 1, c0 = (lane & 1) * 4;
    float4 *X = reinterpret_cast<float4 *>(V + (o + r) * kLd + o + 8 + c0);
    const float *a = A + o * 64 + o + 8 + r, *u = V + o * kLd + o + c0, *t = V + (o + 8 + r) * kLd + o + 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float f = a[m * 64];
      const float4 y = *reinterpret_cast<const float4 *>(u + m * kLd);
      x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
    }
    *X = x;
    __syncwarp();
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float f = -t[m];
      const float4 y = *reinterpret_cast<const float4 *>(u + m * kLd + 8);
      x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
    }
    __syncwarp();
    *reinterpret_cast<float4 *>(V + (o + 8 + r) * kLd + o + c0) = x;
    *X = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncwarp();
  {
    // 16 -> 32: a 4 x 4 tile and half of the contraction per lane
    const int r0 = lane & 12, c0 = (lane & 3) * 4, m0 = (lane >> 4) * 8, row = r0 + 2 * (lane >> 4);
    float4 acc[4] = {};
    tile_at(acc, A + m0 * 64 + 16 + r0, V + m0 * kLd + c0);
    tile_halve<2, 16>(acc, lane);
    float4 *X = reinterpret_cast<float4 *>(V + row * kLd + 16 + c0);
    X[0] = acc[0];
    X[kLd / 4] = acc[1];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    tile_minus(acc, V + (16 + r0) * kLd + 16 + m0, V + m0 * kLd + 16 + c0);
    tile_halve<2, 16>(acc, lane);
    __syncwarp();
    float4 *Y = reinterpret_cast<float4 *>(V + (16 + row) * kLd + c0);
    Y[0] = acc[0];
    Y[kLd / 4] = acc[1];
    X[0] = X[kLd / 4] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

__global__ void __launch_bounds__(kPrepThreads, 4)
    delta_prep_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, DeltaTcParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  __shared__ uint64_t bar[3];
  __shared__ uint32_t tslot;
  __shared__ int abort_flag;
  __shared__ float2 s_g[kC];  // g and its low part
  __shared__ float s_b[kC], s_eg[kC];
  float *Ti = reinterpret_cast<float *>(smem + kPrepT);
  auto At = [&](int j) { return reinterpret_cast<float *>(smem + kPrepA + (j >> 5) * 16384) + (j & 31) * 64; };
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const int c = blockIdx.x % P.N, bh = blockIdx.x / P.N, b = bh / P.H, h = bh % P.H;
  uint8_t *rec = P.rec + ((int64_t)bh * P.N + c) * kRecBytes;

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tslot, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tslot, 0);
  griddep_wait();
  if (tid == 0) {
    mbar_arrive_expect_tx(&bar[0], 32768);
    for (int x = 0; x < 2; ++x) {
      tma_load_4d(&mk, &bar[0], smem + x * 16384, 64 * x, kC * c, h, b, kPolicyEvictNormal);
      tma_load_4d(&mq, &bar[0], smem + x * 16384 + 8192, 64 * x, kC * c, h, b, kPolicyEvictNormal);
    }
  }
  if (warp == 7) {
    // cumulative log2-gates as sums of two fp32 parts (differences of far sums must keep their low bits; in
    // 64-bit arithmetic, slow here, the scan alone took 1.5 us); a gate below 2^-1000 is zero either way
    const int t0 = kC * c + 2 * lane;
    const int64_t gi = (int64_t)bh * P.T + t0;
    Two l[2];
    float be[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool in = t0 + x < P.T;
      const float v = in && P.lg ? load_gate(P.lg, gi + x, P.f32) : 0.f;
      l[x] = v < -690.f ? Two{-1000.f, 0.f} : times_log2e(v);
      be[x] = in ? load_gate(P.beta, gi + x, P.f32) : 0.f;
    }
    Two s = l[0] + l[1];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const Two y{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
      if (lane >= o) s = s + y;
    }
    const Two last{__shfl_sync(0xffffffffu, s.hi, 31), __shfl_sync(0xffffffffu, s.lo, 31)};
    float *g = reinterpret_cast<float *>(rec + kRecG);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const Two gx = x ? s : s + Two{-l[1].hi, -l[1].lo};
      const int j = 2 * lane + x;
      const float eg = ex2(gx.hi) * ex2(gx.lo), phi = ex2((last.hi - gx.hi) + (last.lo - gx.lo));
      s_g[j] = make_float2(gx.hi, gx.lo);
      s_b[j] = be[x];
      s_eg[j] = eg;
      g[j] = eg;
      g[64 + j] = phi;
      g[128 + j] = be[x];
      g[192 + j] = gx.hi;
      g[256 + j] = gx.lo;
    }
  }
  bool ok = true;
  if (warp == 0) {
    ok = mbar_wait_w(&bar[0], 0, &abort_flag, P.status);
    if (ok) {
#pragma unroll
      for (uint32_t ks = 0; ks < 8; ++ks)
        mma_ss_warp(tmem, desc_kmajor(base, ks), desc_kmajor(base, ks), idesc_bf16(128, 64, false, false), ks > 0);
      mma_commit_warp(&bar[1]);
    }
  }
  __syncthreads();
  ok = ok && mbar_wait(&bar[1], 0, &abort_flag, P.status);
  if (__syncthreads_and(ok)) {
    tc_fence_after();
    // lanes 0..63: rows of K K^T, 64..127: of Q K^T; columns 32 x .. + 31
    const uint32_t quad = warp & 3, x = warp >> 2, lb = (quad * 32) << 16;
    const int i = (quad & 1) * 32 + lane;
    const float hi = s_g[i].x, lo = s_g[i].y;
    // (loops stay loops here: straight-line code, run once per CTA by a few warps, is bound by fetching it)
    if (quad < 2) {
      // A_ij = Gam_ij (k_i . k_j) b_j, j < i, transposed (the block above the diagonal is not used)
      if (x <= quad)
#pragma unroll 1
        for (int y = 0; y < 32; y += 8) {
          uint32_t r[8];
          tmem_ld8(tmem + lb + 32 * x + y, r);
          tmem_ld_wait();
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const int j = 32 * x + y + z;
            const float2 gj = s_g[j];
            const float e = ex2((hi - gj.x) + (lo - gj.y));
            At(j)[i] = j < i ? e * __uint_as_float(r[z]) * s_b[j] : 0.f;
          }
        }
      if (x == quad) {
        __syncwarp();
        invert32(At(quad * 32) + quad * 32, Ti + (quad * 32) * kLd + quad * 32, lane);
      }
    } else {
      // P_ij = Gam_ij (q_i . k_j), j <= i, straight to the record
#pragma unroll 1
      for (int y = 0; y < 2; ++y) {
        uint32_t r[16], ph[8], pl[8];
        tmem_ld16(tmem + lb + 32 * x + 16 * y, r);
        tmem_ld_wait();
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const int j = 32 * x + 16 * y + 2 * z;
          const float2 g0 = s_g[j], g1 = s_g[j + 1];
          const float p0 = ex2((hi - g0.x) + (lo - g0.y)) * __uint_as_float(r[2 * z]);
          const float p1 = ex2((hi - g1.x) + (lo - g1.y)) * __uint_as_float(r[2 * z + 1]);
          split2(j <= i ? p0 : 0.f, j + 1 <= i ? p1 : 0.f, ph[z], pl[z]);
        }
        store_row8(rec + kRecP, i, 2 * x + y, ph);
        store_row8(rec + kRecP + 8192, i, 2 * x + y, pl);
      }
    }
    __syncthreads();
    {
      // the off-diagonal block -T22 (A21 T11): X = A21 T11 parked in the upper right block, then zeroed
      const int r0 = 4 * warp, c0 = (lane & 7) * 4, m0 = (lane >> 3) * 8;
      float4 acc[4] = {};
      tile_at(acc, At(m0) + 32 + r0, Ti + m0 * kLd + c0);
      tile_halve<2, 16>(acc, lane);
      tile_halve<1, 8>(acc, lane);
      const int row = r0 + (lane >> 3);
      float4 *X = reinterpret_cast<float4 *>(Ti + row * kLd + 32 + c0);
      *X = acc[0];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      tile_minus(acc, Ti + (32 + r0) * kLd + 32 + m0, Ti + m0 * kLd + 32 + c0);
      tile_halve<2, 16>(acc, lane);
      tile_halve<1, 8>(acc, lane);
      __syncthreads();
      *reinterpret_cast<float4 *>(Ti + (32 + row) * kLd + c0) = acc[0];
      *X = make_float4(0.f, 0.f, 0.f, 0.f);
      __syncthreads();
    }
    {
      // T to the record; T diag(e^g), the operand of W, over A
      const int row = tid & 63, q = tid / 64;
      uint32_t th[8], tl[8];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t eh[4], el[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int j = 16 * q + 8 * y + 2 * z;
          const float2 u = *reinterpret_cast<const float2 *>(Ti + row * kLd + j);
          split2(u.x, u.y, th[4 * y + z], tl[4 * y + z]);
          split2(u.x * s_eg[j], u.y * s_eg[j + 1], eh[z], el[z]);
        }
        const uint32_t at = sw(row, 2 * q + y);
        st_shared_v4(base + kPrepA + at, eh[0], eh[1], eh[2], eh[3]);
        st_shared_v4(base + kPrepA + 16384 + at, el[0], el[1], el[2], el[3]);
      }
      store_row8(rec + kRecT, part_row(row), q, th);
      store_row8(rec + kRecT + kPartLo, part_row(row), q, tl);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
#pragma unroll
      for (uint32_t p = 0; p < 2; ++p)
#pragma unroll
        for (uint32_t ks = 0; ks < 4; ++ks)
          mma_ss_warp(tmem + 64, desc_mnmajor(base, ks), desc_kmajor(base + kPrepA + p * 16384, ks),
                      idesc_bf16(128, 64, true, false), p + ks > 0);
      mma_commit_warp(&bar[2]);
    }
    ok = mbar_wait(&bar[2], 0, &abort_flag, P.status);
    if (__syncthreads_and(ok)) {
      tc_fence_after();
      // W^T: lane = key dimension, column = token; negated, with tokens as rows over the K and Q tiles
#pragma unroll 1
      for (uint32_t y = 0; y < 4; ++y) {
        const uint32_t row0 = quad * 32 + 16 * (y & 1), tok0 = 32 * x + 16 * (y >> 1);
        float w[8];
        uint32_t h[4], l[4];
        tmem_ld_frag(tmem + (row0 << 16) + 64 + tok0, w);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(-w[2 * e], -w[2 * e + 1], h[e], l[e]);
        const uint32_t at = base + frag_at_trans(lane, part_row(tok0), row0, 16384);
        stmatrix4_trans(at, h);
        stmatrix4_trans(at + kPartLo, l);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        bulk_store(rec + kRecW, smem, 32768);
        bulk_commit();
        bulk_wait_all();
      }
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 128);
}

// ================================================================== chains
// One CTA per (batch, head, slice of VS value dimensions): the columns of S are independent given W, K and
// T, so slices spread a chain over several SMs.  Lanes are key dimensions (S: 128 rows) or tokens (O, dU: 64
// rows, lanes 16 q .. 16 q + 15 of every quarter; Y: the same for T's and W's hi parts and the other lanes for
// the lo parts), columns the slice.  What the threads make for the next product (S, Y, R, dU in two bf16 parts,
// side by side) goes to shared memory as its B operand, and both parts meet the same A tile in one product of
// 2 VS columns: a product costs what reading its operand rows costs (33 to 35 cycles per 16 of the contraction
// for 64 rows, 42 to 51 for 128, whatever the width up to 64), so few wide ones beat many narrow ones.
//
// A chunk's path is S -> (W S) -> Y -> (K^T Y) -> S: two products and two passes of the threads, each bounded
// by its latency: 1.52 us a chunk forward and 1.50 backward with slices of 32 (0.388 and 0.384 ms at B2 H16
// T16384, on 128 SMs; the other tensor work fits into the gaps).  Next comes what an SM takes in: 104 KB a chunk
// forward, 9 TB/s over all of them; with a slot less for W the rings run dry (0.49 ms).  Every role is a long
// loop of its own, so their instructions have to be few: with unrolled products and in-line waits two CTAs on
// neighbouring SMs took 1.5 times as long as one alone.  Warps: 1 issues the chain's products, 2 the output's, 0, 3
// and the last two load, 4 and on (4 VS/16) carry the chain (16 columns each: the threads' work is on the path, so
// it is spread thin), then 4 make the output (forward) or the scaled dO (backward).
constexpr int kGateRing = 4, kSideWarps = 4;
template <int VS>
struct Chain {
  static constexpr int warps = VS / 4, side = 4 + warps, threads = 32 * (side + kSideWarps + 2);  // side: first such warp
  // four rings of tiles in order of use: two of 8 KiB, then 16 KiB ones
  static constexpr int nx = VS == 32 ? 4 : 2, ny = 4, nz = 2, slots = 2 + nx + ny + nz;
  // operand tiles: rows of hi and lo parts side by side (VS = 32: one 128-byte row; 64: two blocks)
  static constexpr uint32_t state_lo = VS == 32 ? 64 : 16384, row_lo = VS == 32 ? 64 : 8192;
  static constexpr uint32_t op = (slots - 1) * kSlot, u0 = op + 128 * VS * 4, u1 = u0 + 64 * VS * 4,
                            gate = u1 + 64 * VS * 4, bar = gate + kGateRing * 2048;
  static constexpr size_t smem = bar + 512 + 1024;
};
static_assert(Chain<32>::smem <= 231000 && Chain<64>::smem <= 231000, "one CTA per SM");

enum { C_OP = 0,    // S (R) operand parts ready
       C_SCALED,    // backward: R's accumulator scaled by the chunk's decay
       C_ACC,       // its accumulator complete (next chunk)
       C_YFULL,     // Y (K R) accumulator complete
       C_YOP,       // the operand made from it for the update ready
       C_UOP,       // (C_YOP + 1) forward: its operand for the output ready; backward: the scaled dO
       C_QS, C_OFULL, C_OFREE,   // forward: Q S done; output complete, read
       C_GFULL, C_GEMPTY = C_GFULL + kGateRing, C_FULL = C_GEMPTY + kGateRing };

// A place in a ring (slots FIRST .. FIRST + CNT - 1): slot and the parity of its use.
template <int FIRST, int CNT>
struct RingPos {
  int s = FIRST;
  uint32_t ph = 0;
  __device__ void advance() {
    if (++s == FIRST + CNT) {
      s = FIRST;
      ph ^= 1;
    }
  }
  __device__ RingPos next() const {
    RingPos r = *this;
    r.advance();
    return r;
  }
};

// Descriptors are formed once per tile; a step of 16 along the contraction adds to the address field.
__device__ __forceinline__ uint64_t k_tile(uint32_t tile) { return sdesc_sw128(tile, 16u, 1024u); }
__device__ __forceinline__ uint64_t mn_tile(uint32_t tile, uint32_t block) { return sdesc_sw128(tile, block, 1024u); }
__device__ __forceinline__ constexpr uint64_t k_step(uint32_t ks) { return ks * 2u; }
__device__ __forceinline__ constexpr uint64_t mn_step(uint32_t ks) { return ks * 128u; }
// D (+)= A B over `n` times four steps, A K-major (AM = false) or MN-major, B MN-major; a_inc and b_inc lead
// to the next four (the next 64-column block of A, the next 64 rows of B, the other part of either).
// (A_ROWS: MN-major, the rows from one step of A to the next in units of 16)
template <bool AM, int A_ROWS = 1>
__device__ __forceinline__ void mma_four(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  mma_ss_warp(d, a, b, idesc, acc);
#pragma unroll
  for (uint32_t ks = 1; ks < 4; ++ks)
    mma_ss_warp(d, a + (AM ? mn_step(A_ROWS * ks) : k_step(ks)), b + mn_step(ks), idesc, 1);
}
// ROLL: as a loop (less code, a few cycles more): the forward, with more roles, gains from it, the backward
// only off its path
template <bool AM, bool ROLL, int N, int A_ROWS = 1>
__device__ __forceinline__ void mma_fours(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool fresh, uint32_t a_inc,
                                          uint32_t b_inc) {
  if (ROLL) {
    uint32_t acc = fresh ? 0 : 1;
#pragma unroll 1
    for (int i = 0; i < N; ++i, a += a_inc, b += b_inc, acc = 1) mma_four<AM, A_ROWS>(d, a, b, idesc, acc);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) mma_four<AM, A_ROWS>(d, a + i * a_inc, b + i * b_inc, idesc, i > 0 || !fresh);
  }
}
constexpr uint32_t kBlock = 8192 >> 4, kRows64 = 4 * 128;  // descriptor increments: 8 KiB; 64 rows

template <int VS>
struct ChainCtx {
  using L = Chain<VS>;
  static constexpr int empty0 = C_FULL + L::slots, count = empty0 + L::slots;
  uint8_t *smem;
  uint64_t *bar;
  volatile int *abort_flag;
  int *status;
  uint32_t base;
  __device__ bool wait(int idx, int parity) const {
    return mbar_wait_compact(&bar[idx], parity & 1, abort_flag, status);
  }
  __device__ bool wait_w(int idx, int parity) const { return __all_sync(0xffffffffu, wait(idx, parity)); }
  __device__ static uint32_t offset(int s) { return s < 2 ? s * 8192u : (s - 1) * kSlot; }
  template <typename Pos>
  __device__ uint32_t slot(Pos p) const { return base + offset(p.s); }
  template <typename Pos>
  __device__ bool full(Pos p) const { return wait_w(C_FULL + p.s, p.ph); }
  template <typename Pos>
  __device__ void release(Pos p) const { mma_commit_warp(&bar[empty0 + p.s]); }
  // Several barriers at once: their tests go out back to back (one wait costs some 150 cycles even when there
  // is nothing to wait for), and only if one is not yet there they are waited for one by one.
  template <int N>
  __device__ bool wait_all(const int (&idx)[N], const uint32_t (&parity)[N]) const {
    bool ready = true;
#pragma unroll
    for (int i = 0; i < N; ++i) ready &= mbar_test_wait(&bar[idx[i]], parity[i] & 1);
    if (__all_sync(0xffffffffu, ready)) return true;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!wait_w(idx[i], parity[i])) return false;
    return true;
  }
  __device__ bool gates_ready(int x) const { return wait_w(C_GFULL + x % kGateRing, x / kGateRing); }
  __device__ const float *gates(int x) const {
    return reinterpret_cast<const float *>(smem + L::gate + (x % kGateRing) * 2048);
  }
  // one arrival per warp, after the warp's accesses to tensor and shared memory
  __device__ void arrive(int idx, int lane) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[idx]);
  }
  __device__ void setup(uint32_t *tslot, int *abort, int warp, int uop) const {
    if (threadIdx.x == 0) {
      *abort = 0;
      for (int i = 0; i < count; ++i) {
        int n = 1;
        if (i >= C_GEMPTY && i < C_GEMPTY + kGateRing) n = L::warps + kSideWarps;
        if (i == C_OP || i == C_SCALED || i == C_YOP) n = L::warps;
        if (i == C_UOP) n = uop;  // the warps that make that operand
        if (i == C_OFREE) n = kSideWarps;
        mbar_init(&bar[i], n);
      }
      fence_mbar_init();
    }
    if (warp == 1) {
      tmem_alloc(tslot, 512);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
};

// A loading thread and its ring.  Four threads share every chunk's loads, since a single one spends most of a
// chunk's time on its waits; each has a ring of its own, since a slot's waits have to be in one thread's order;
// and all run the same code on what they are given, since code is what they have too much of.
struct ChainLoad {
  const CUtensorMap *map;  // a tile of a sequence tensor; or null: an image at `off` in the record
  uint32_t off, bytes;     // (bytes 8192: only the 64-column block of the tile that starts at column `off`)
};
template <int VS>
struct ChainLoader {
  const ChainCtx<VS> &k;
  int h, b, first, end;  // the ring's slots
  int s = first;
  uint32_t ph = 0;
  bool ok = true, lap = false;
  __device__ void load(const ChainLoad &l, int c, const uint8_t *rec) {
    // (a fresh barrier's wait for the parity before its first phase succeeds at once: no use precedes it)
    if (!ok || !(ok = k.wait(ChainCtx<VS>::empty0 + s, ph ^ 1))) return;
    uint8_t *dst = k.smem + k.offset(s);
    uint64_t *full = &k.bar[C_FULL + s];
    mbar_arrive_expect_tx(full, l.bytes);
    if (!l.map) {
      bulk_load(full, dst, rec + l.off, l.bytes);
    } else {
      tma_load_4d(l.map, full, dst, l.off, kC * c, h, b, kPolicyEvictNormal);
      if (l.bytes == kSlot) tma_load_4d(l.map, full, dst + 8192, 64, kC * c, h, b, kPolicyEvictNormal);
    }
    advance(s, ph);
    lap |= ph != 0;
  }
  __device__ void advance(int &at, uint32_t &parity) const {
    if (++at == end) {
      at = first;
      parity ^= 1;
    }
  }
  __device__ void gates(int x, const uint8_t *src) {
    const int g = x % kGateRing;
    if (!ok || (x >= kGateRing && !(ok = k.wait(C_GEMPTY + g, x / kGateRing - 1)))) return;
    mbar_arrive_expect_tx(&k.bar[C_GFULL + g], kGateBytes);
    bulk_load(&k.bar[C_GFULL + g], k.smem + Chain<VS>::gate + g * 2048, src, kGateBytes);
  }
  // One chunk after the other (step: 1 or -1), loads a then l (if it has bytes) of each, and the gates.
  __device__ void run(int n, int c, int step, const uint8_t *rec, const ChainLoad &a, const ChainLoad &l, bool with_gates) {
#pragma unroll 1
    for (int x = 0; x < n && ok; ++x, c += step, rec += step * (int64_t)kRecBytes) {
#pragma unroll 1
      for (int y = 0; y < 2; ++y)
        if (y == 0 || l.bytes) load(y ? l : a, c, rec);
      if (with_gates) gates(x, rec + kRecG);
    }
    // waits, each with its limit, for what is in flight before the block ends: the ring's last lap and the last gates
    volatile int no_abort = 0;
    int at = lap ? s : first;
    uint32_t parity = lap ? ph ^ 1 : 0;
    for (int left = lap ? end - first : s - first; left > 0; --left) {
      mbar_wait_compact(&k.bar[C_FULL + at], parity, &no_abort, k.status);
      advance(at, parity);
    }
    for (int x = with_gates && ok ? max(0, n - kGateRing) : n; x < n; ++x)
      mbar_wait_compact(&k.bar[C_GFULL + x % kGateRing], (x / kGateRing) & 1, &no_abort, k.status);
  }
};
// the ring of loading thread i: 0 (8 KiB slots), x, y, z
template <int VS>
__device__ __forceinline__ int ring_first(int i) {
  using L = Chain<VS>;
  return i == 0 ? 0 : i == 1 ? 2 : i == 2 ? 2 + L::nx : i == 3 ? 2 + L::nx + L::ny : L::slots;
}
// the loading thread that a warp is, or -1
template <int VS>
__device__ __forceinline__ int loader_of(int warp) {
  const int extra = warp - Chain<VS>::side - kSideWarps;
  return warp == 0 ? 0 : warp == 3 ? 1 : extra >= 0 ? 2 + extra : -1;
}

// 16 values of row r, columns 16 g .. + 15 of the slice, as hi and lo parts in an operand tile (`lo`: the
// offset of the lo parts); hi returns the former, packed
template <int VS>
__device__ __forceinline__ void put_split(uint32_t tile, uint32_t lo, uint32_t r, uint32_t g, const float (&x)[16],
                                          uint32_t (&hi)[8]) {
  uint32_t l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split2(x[2 * j], x[2 * j + 1], hi[j], l[j]);
  // VS = 32: the lo parts are pieces 4 .. 7 of the same 128-byte row
  const uint32_t row = tile + r * 128u, blk = VS == 32 ? row : row + lo, p = VS == 32 ? 4u : 0u;
  st_shared_v4(row + (((2 * g) ^ (r & 7u)) << 4), hi[0], hi[1], hi[2], hi[3]);
  st_shared_v4(row + (((2 * g + 1) ^ (r & 7u)) << 4), hi[4], hi[5], hi[6], hi[7]);
  st_shared_v4(blk + (((p + 2 * g) ^ (r & 7u)) << 4), l[0], l[1], l[2], l[3]);
  st_shared_v4(blk + (((p + 2 * g + 1) ^ (r & 7u)) << 4), l[4], l[5], l[6], l[7]);
}

// 8 values of row r, piece p of the slice, already split: words 0..3 are the hi parts, 4..7 the lo parts
template <int VS>
__device__ __forceinline__ void put_piece(uint32_t tile, uint32_t lo, uint32_t r, uint32_t p, const uint32_t (&w)[8]) {
  const uint32_t row = tile + r * 128u, blk = VS == 32 ? row : row + lo, pl = VS == 32 ? p + 4u : p;
  st_shared_v4(row + ((p ^ (r & 7u)) << 4), w[0], w[1], w[2], w[3]);
  st_shared_v4(blk + ((pl ^ (r & 7u)) << 4), w[4], w[5], w[6], w[7]);
}

// 16 columns of a state row in global memory (fp32, row and columns inside d)
__device__ __forceinline__ void load_state16(const float *p, float (&s)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = p ? reinterpret_cast<const float4 *>(p)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
    s[4 * j] = v.x;
    s[4 * j + 1] = v.y;
    s[4 * j + 2] = v.z;
    s[4 * j + 3] = v.w;
  }
}
__device__ __forceinline__ void store_state16(float *p, const float (&s)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<float4 *>(p)[j] = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
}
__device__ __forceinline__ void tmem_ldf(uint32_t addr, float (&x)[16]) {
  tmem_ld16(addr, *reinterpret_cast<uint32_t(*)[16]>(&x));
}
__device__ __forceinline__ void tmem_stf(uint32_t addr, const float (&x)[16]) {
  tmem_st16(addr, *reinterpret_cast<const uint32_t(*)[16]>(&x));
}

// Tensor memory of the forward chain (columns): S, Y, Q S and P Y, each as the products of both parts.
// Forward slices are always of 32: with 64, a chunk took 2.2 times as long (B2 H32 T4096, one turn of slices of 64
// against two of slices of 32: 247 us against 230, which are 203 now).
constexpr int kSlice = 32;
using kChain = Chain<kSlice>;
__global__ void __launch_bounds__(kChain::threads, 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, __nv_bfloat16 *o, int64_t osb, int64_t osh, int64_t ost,
                       DeltaTcParams P) {
  constexpr int VS = kSlice;
  using L = kChain;
  using RV = RingPos<0, 2>;
  using RX = RingPos<2, L::nx>;
  using RY = RingPos<2 + L::nx, L::ny>;
  using RZ = RingPos<2 + L::nx + L::ny, L::nz>;
  constexpr uint32_t kTS = 0, kTY = 2 * VS, kTQ = 4 * VS, kTP = 6 * VS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_flag;
  uint8_t *smem = align1024(smem_raw);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::bar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + ChainCtx<VS>::count);
  const ChainCtx<VS> k{smem, bar, &abort_flag, P.status, smem_u32(smem)};
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int ns = P.d / VS, bh = blockIdx.x / ns, b = bh / P.H, h = bh % P.H;
  const int x0 = (blockIdx.x % ns) * VS;  // the slice's first value dimension
  k.setup(tslot, &abort_flag, warp, L::warps);
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  griddep_wait();

  const int loader = loader_of<VS>(warp);
  if (loader >= 0) {
    // V, gates | T, K | W | Q, P
    if (lane == 0) {
      const ChainLoad a{loader == 0 ? &mv : loader == 3 ? &mq : nullptr,
                        loader == 0 ? x0 / 64 * 64u : loader == 1 ? kRecT : loader == 2 ? kRecW : 0u,
                        loader == 0 ? 8192u : kSlot};
      const ChainLoad l{loader == 1 ? &mk : nullptr, loader == 2 ? kRecW + kSlot : loader == 3 ? kRecP : 0u,
                        loader == 0 ? 0u : kSlot};
      ChainLoader<VS> ld{k, h, b, ring_first<VS>(loader), ring_first<VS>(loader + 1)};
      ld.run(P.N, 0, 1, P.rec + (int64_t)bh * P.N * kRecBytes, a, l, loader == 0);
    }
  } else if (warp == 1) {
    // the chain's own products, in the order of its dependences
    const uint32_t id_1 = idesc_bf16(128, VS, false, true), id_2 = idesc_bf16(128, 2 * VS, false, true),
                   id_k = idesc_bf16(128, 2 * VS, true, true);
    const uint64_t op = mn_tile(k.base + L::op, L::state_lo), ut = mn_tile(k.base + L::u0, L::row_lo);
    RV rv;  // V
    RX rx;  // T, K
    RY ry;  // W, in two blocks of 64 key dimensions
    auto landed = [&] { return k.full(rv) && k.full(rx) && k.full(ry) && k.full(ry.next()); };  // V, T, W
    auto vt = [&] {  // Y = T V
      tc_fence_after();
      const uint64_t v = mn_tile(k.slot(rv) + (x0 & 63) * 2, 8192), tt = k_tile(k.slot(rx));
      mma_fours<false, true, 1>(tmem + kTY, tt, v, id_1, true, 0, 0);
      k.release(rv);
      k.release(rx);
      rv.advance();
      rx.advance();
    };
    // The waits for the next chunk's tiles stand in the gap before Y's operand, not on the path behind it.
    bool ok = landed();
    if (ok) vt();
#pragma unroll 1
    for (int c = 0; c < P.N && ok; ++c) {
      // Y += W [S hi | S lo] (2 VS columns)
      const RY second = ry.next();
      if (!(ok = k.wait_w(C_OP, c))) break;
      tc_fence_after();
      mma_fours<false, true, 1>(tmem + kTY, k_tile(k.slot(ry)), op, id_2, false, 0, 0);
      mma_fours<false, true, 1>(tmem + kTY, k_tile(k.slot(second)), op + kRows64, id_2, false, 0, 0);
      mma_commit_warp(&bar[C_YFULL]);
      k.release(ry);
      k.release(second);
      ry = second.next();
      // S += K^T diag(phi b) Y
      const RX kt = rx;
      rx.advance();
      // (C_YOP: every thread has also written back its part of S, scaled)
      if (!(ok = k.full(kt) && (c + 1 == P.N || landed()) && k.wait_w(C_YOP, c))) break;
      tc_fence_after();
      mma_fours<true, true, 1>(tmem + kTS, mn_tile(k.slot(kt), 8192), ut, id_k, false, 0, 0);
      mma_commit_warp(&bar[C_ACC]);
      if (c + 1 < P.N) vt();
      k.release(kt);
    }
  } else if (warp == 2) {
    // the output's products, put into the gaps that the chain leaves the tensor cores: Q S while the
    // threads turn Y into operands, P Y while they turn S into operands
    const uint32_t id_1 = idesc_bf16(64, VS, false, true), id_2 = idesc_bf16(64, 2 * VS, false, true);
    const uint64_t op = mn_tile(k.base + L::op, L::state_lo), u = mn_tile(k.base + L::u1, L::row_lo);
    RZ rz;  // Q, P
    bool ok = true;
#pragma unroll 1
    for (int c = 0; c < P.N && ok; ++c) {
      if (!(ok = k.full(rz) && (c == 0 || k.wait_w(C_OFREE, c - 1)) && k.wait_w(C_YFULL, c))) break;
      tc_fence_after();
      mma_fours<false, true, 2>(tmem + kTQ, k_tile(k.slot(rz)), op, id_2, true, kBlock, kRows64);
      mma_commit_warp(&bar[C_QS]);
      k.release(rz);
      rz.advance();
      if (!(ok = k.full(rz) && k.wait_w(C_UOP, c) && k.wait_w(C_ACC, c))) break;
      tc_fence_after();
      const uint64_t pp = k_tile(k.slot(rz));
      mma_fours<false, true, 1>(tmem + kTP, pp, u, id_2, true, 0, 0);
      mma_fours<false, true, 1>(tmem + kTP, pp + kBlock, u, id_1, false, 0, 0);
      mma_commit_warp(&bar[C_OFULL]);
      k.release(rz);
      rz.advance();
    }
  } else if (warp < L::side) {
    // S: key dimension `row`, columns 16 cg .. + 15 of the slice; Y: token `tok`, the sums' parts from the hi
    // rows of T and W in lanes 0..15 and from the lo rows in 16..31, put together as 8 columns per lane
    const uint32_t quad = warp & 3, cg = (warp - 4) >> 2, row = quad * 32 + lane, tok = quad * 16 + (lane & 15);
    const uint32_t t = tmem + ((quad * 32) << 16) + 16 * cg;
    const uint32_t gcol = x0 + 16 * cg;  // the columns' value dimension
    const int64_t at = ((int64_t)bh * P.d + row) * P.d + gcol;
    const bool in = (int)row < P.d;
    const float zero[16] = {};
    tmem_stf(t + kTY + VS, zero);
    tmem_st_wait();
    bool ok = true;
    for (int c = 0; c <= P.N && ok; ++c) {
      float s[16];
      if (c == 0) {
        load_state16(P.in && in ? P.in + at : nullptr, s);
      } else {
        // (Q S of the last chunk has read the operand that is rewritten here)
        if (!(ok = k.wait_w(C_QS, c - 1) && k.wait_w(C_ACC, c - 1))) break;
        tc_fence_after();
        float s2[16];
        tmem_ldf(t + kTS, s);
        tmem_ldf(t + kTS + VS, s2);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j] += s2[j];
      }
      if (c == P.N) {
        if (P.out && in) store_state16(P.out + at, s);
        break;
      }
      uint32_t hi[8];
      put_split<VS>(k.base + L::op, L::state_lo, row, cg, s, hi);
      fence_proxy_async_smem();
      k.arrive(C_OP, lane);
      if (!(ok = k.gates_ready(c))) break;
      const float *g = k.gates(c);
      const float f = g[63], phi = g[64 + tok], be = g[128 + tok];
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] *= f;
      tmem_stf(t + kTS, s);
      tmem_stf(t + kTS + VS, zero);
      if (P.simg) store_row8(P.simg + ((int64_t)bh * P.N + c) * kStateImg + (gcol >> 6) * 16384, row, (gcol & 63) >> 4, hi);
      // The last chunk's output product is done: it has read the operand that is rewritten below, and its
      // issuer has seen that chunk's C_ACC, which the arrival at C_YOP may lead to complete again.
      if (!(ok = (c == 0 || k.wait_w(C_OFULL, c - 1)) && k.wait_w(C_YFULL, c))) break;
      tc_fence_after();
      float y[16], z[16];
      tmem_ldf(t + kTY, y);
      tmem_ldf(t + kTY + VS, z);
      tmem_ld_wait();
      tmem_stf(t + kTY + VS, zero);
#pragma unroll
      for (int j = 0; j < 16; ++j) y[j] += z[j];
      const bool up = lane & 16;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = (up ? y[j + 8] : y[j]) + __shfl_xor_sync(0xffffffffu, up ? y[j] : y[j + 8], 16);
      tmem_st_wait();
      const uint32_t piece = 2 * cg + (lane >> 4);
      float w = phi * be;  // the update's factor, then the output's
#pragma unroll 1
      for (int e = 0; e < 2; ++e, w = be) {
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(w * y[2 * j], w * y[2 * j + 1], hi[j], hi[4 + j]);
        put_piece<VS>(k.base + L::u0 + e * (L::u1 - L::u0), L::row_lo, tok, piece, hi);
        fence_proxy_async_smem();
        k.arrive(C_YOP + e, lane);
      }
      if (lane == 0) mbar_arrive(&bar[C_GEMPTY + c % kGateRing]);
      if (P.yimg) {
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(y[2 * j], y[2 * j + 1], hi[j], hi[4 + j]);
        uint8_t *img = P.yimg + ((int64_t)bh * P.N + c) * kYImg + (gcol >> 6) * 8192 +
                       sw(tok, ((gcol & 63) >> 3) + (lane >> 4));
        *reinterpret_cast<uint4 *>(img) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(img + kRowImg) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      }
    }
  } else {
    // O = diag(e^g) Q S + P diag(b) Y, a token per lane (lanes 0..15)
    const uint32_t quad = warp & 3, tok = quad * 16 + (lane & 15), t = tmem + ((quad * 32) << 16);
    __nv_bfloat16 *dst = o + b * osb + h * osh + x0;
    bool ok = true;
    for (int c = 0; c < P.N && ok; ++c) {
      if (!(ok = k.gates_ready(c) && k.wait_w(C_QS, c) && k.wait_w(C_OFULL, c))) break;
      tc_fence_after();
      const float eg = k.gates(c)[tok];
      const bool in = lane < 16 && kC * c + (int)tok < P.T;
#pragma unroll 1
      for (int x = 0; x < VS / 16; ++x) {
        float q[2][16], p[2][16];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          tmem_ldf(t + kTQ + y * VS + 16 * x, q[y]);
          tmem_ldf(t + kTP + y * VS + 16 * x, p[y]);
        }
        tmem_ld_wait();
        if (x + 1 == VS / 16) k.arrive(C_OFREE, lane);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = pack_bf16(fmaf(eg, q[0][2 * j] + q[1][2 * j], p[0][2 * j] + p[1][2 * j]),
                           fmaf(eg, q[0][2 * j + 1] + q[1][2 * j + 1], p[0][2 * j + 1] + p[1][2 * j + 1]));
        if (in) {
          uint4 *to = reinterpret_cast<uint4 *>(dst + (int64_t)(kC * c + tok) * ost + 16 * x);
          to[0] = make_uint4(w[0], w[1], w[2], w[3]);
          to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (lane == 0) mbar_arrive(&bar[C_GEMPTY + c % kGateRing]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Tensor memory of the reverse chain: R (both parts' products); P^T dO; K R (both).
template <int VS>
__global__ void __launch_bounds__(Chain<VS>::threads, 1)
    delta_reverse_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mdo, DeltaTcParams P) {
  using L = Chain<VS>;
  using RV = RingPos<0, 2>;
  using RX = RingPos<2, L::nx>;
  using RY = RingPos<2 + L::nx, L::ny>;
  using RZ = RingPos<2 + L::nx + L::ny, L::nz>;
  constexpr uint32_t kTR = 0, kT1 = 2 * VS, kT2 = 3 * VS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_flag;
  uint8_t *smem = align1024(smem_raw);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::bar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + ChainCtx<VS>::count);
  const ChainCtx<VS> k{smem, bar, &abort_flag, P.status, smem_u32(smem)};
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int ns = P.d / VS, bh = blockIdx.x / ns, b = bh / P.H, h = bh % P.H, x0 = (blockIdx.x % ns) * VS;
  k.setup(tslot, &abort_flag, warp, kSideWarps);
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  griddep_wait();

  // step x of the walk is chunk N - 1 - x
  const int loader = loader_of<VS>(warp);
  if (loader >= 0) {
    // dO, gates | P, K | W | Q
    if (lane == 0) {
      const ChainLoad a{loader == 0 ? &mdo : loader == 3 ? &mq : nullptr,
                        loader == 0 ? x0 / 64 * 64u : loader == 1 ? kRecP : loader == 2 ? kRecW : 0u,
                        loader == 0 ? 8192u : kSlot};
      const ChainLoad l{loader == 1 ? &mk : nullptr, loader == 2 ? kRecW + kSlot : 0u,
                        loader == 0 || loader == 3 ? 0u : kSlot};
      ChainLoader<VS> ld{k, h, b, ring_first<VS>(loader), ring_first<VS>(loader + 1)};
      ld.run(P.N, P.N - 1, -1, P.rec + ((int64_t)bh * P.N + P.N - 1) * kRecBytes, a, l, loader == 0);
    }
  } else if (warp == 1) {
    const uint32_t id_p = idesc_bf16(64, VS, true, true), id_2 = idesc_bf16(64, 2 * VS, false, true),
                   id_k = idesc_bf16(128, VS, true, true), id_k2 = idesc_bf16(128, 2 * VS, true, true);
    const uint64_t op = mn_tile(k.base + L::op, L::state_lo), ut = mn_tile(k.base + L::u0, L::row_lo),
                   dos = mn_tile(k.base + L::u1, L::row_lo);
    RV rv;  // dO
    RX rx;  // P, K
    RY ry;  // W, in two blocks of 64 key dimensions (neighbours in a ring of an even number)
    static_assert(L::ny % 2 == 0, "");
    RZ rz;  // Q
    auto pd = [&](RV d) {  // P^T dO
      tc_fence_after();
      mma_fours<true, true, 2>(tmem + kT1, mn_tile(k.slot(rx), 8192), mn_tile(k.slot(d) + (x0 & 63) * 2, 8192), id_p, true,
                               kBlock, 0);
      k.release(rx);
      rx.advance();
    };
    bool ok = k.full(rv) && k.full(rx);
    if (ok) pd(rv);
#pragma unroll 1
    for (int x = 0; x < P.N && ok; ++x) {
      if (!(ok = k.full(rx) && k.wait_w(C_OP, x))) break;
      tc_fence_after();
      mma_fours<false, false, 2>(tmem + kT2, k_tile(k.slot(rx)), op, id_2, true, kBlock, kRows64);  // K R
      mma_commit_warp(&bar[C_YFULL]);
      k.release(rx);
      rx.advance();
      // R += Q^T diag(e^g) dO
      {
        const int idx[3] = {C_FULL + rz.s, C_SCALED, C_UOP};
        const uint32_t parity[3] = {rz.ph, (uint32_t)x, (uint32_t)x};
        if (!(ok = k.wait_all(idx, parity))) break;
      }
      tc_fence_after();
      mma_fours<true, false, 1>(tmem + kTR, mn_tile(k.slot(rz), 8192), dos, id_k2, false, 0, 0);
      k.release(rz);
      rz.advance();
      k.release(rv);  // the scaled dO is ready: every reader of this tile is done
      rv.advance();
      // R += W^T diag(b) dU: hi hi, hi lo, lo hi (after the waits for the next step's dO and P)
      const RY second = ry.next();
      if (x + 1 < P.N) {
        const int idx[4] = {C_FULL + ry.s, C_FULL + second.s, C_FULL + rv.s, C_FULL + rx.s};
        const uint32_t parity[4] = {ry.ph, second.ph, rv.ph, rx.ph};
        ok = k.wait_all(idx, parity);
      } else {
        ok = k.full(ry) && k.full(second);
      }
      if (!(ok = ok && k.wait_w(C_YOP, x))) break;
      tc_fence_after();
      const uint64_t wt = mn_tile(k.slot(ry), kSlot);
      mma_fours<true, false, 1, 2>(tmem + kTR, wt, ut, id_k2, false, 0, 0);
      mma_fours<true, false, 1, 2>(tmem + kTR, wt + (kPartLo >> 4), ut, id_k, false, 0, 0);
      mma_commit_warp(&bar[C_ACC]);
      if (x + 1 < P.N) pd(rv);
      k.release(ry);
      k.release(second);
      ry = second.next();
    }
  } else if (warp == 2) {
    // (the forward's output products)
  } else if (warp < L::side) {
    const uint32_t quad = warp & 3, cg = (warp - 4) >> 2, row = quad * 32 + lane, tok = quad * 16 + (lane & 15);
    const uint32_t t = tmem + ((quad * 32) << 16) + 16 * cg;
    const uint32_t gcol = x0 + 16 * cg;
    const int64_t at = ((int64_t)bh * P.d + row) * P.d + gcol;
    const bool in = (int)row < P.d;
    const float zero[16] = {};
    bool ok = true;
    for (int x = 0; x <= P.N && ok; ++x) {
      const int64_t ci = (int64_t)bh * P.N + P.N - 1 - x;
      float s[16];
      if (x == 0) {
        load_state16(P.in && in ? P.in + at : nullptr, s);
      } else {
        if (!(ok = k.wait_w(C_ACC, x - 1))) break;
        tc_fence_after();
        float s2[16];
        tmem_ldf(t + kTR, s);
        tmem_ldf(t + kTR + VS, s2);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j] += s2[j];
      }
      if (x == P.N) {
        if (P.out && in) store_state16(P.out + at, s);
        break;
      }
      uint32_t hi[8];
      put_split<VS>(k.base + L::op, L::state_lo, row, cg, s, hi);
      fence_proxy_async_smem();
      k.arrive(C_OP, lane);
      if (!(ok = k.gates_ready(x))) break;
      const float *g = k.gates(x);
      const float f = g[63], phi = g[64 + tok], be = g[128 + tok];
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] *= f;
      tmem_stf(t + kTR, s);
      tmem_stf(t + kTR + VS, zero);
      tmem_st_wait();
      k.arrive(C_SCALED, lane);
      store_row8(P.rimg + ci * kStateImg + (gcol >> 6) * 16384, row, (gcol & 63) >> 4, hi);
      const int64_t img = ci * kYImg + (gcol >> 6) * 8192 + sw(tok, ((gcol & 63) >> 3) + (lane >> 4));
      prefetch_l1(P.yimg + img);
      prefetch_l1(P.yimg + img + kRowImg);
      if (!(ok = k.wait_w(C_YFULL, x))) break;
      tc_fence_after();
      float u[16], v[16], w[16];
      tmem_ldf(t + kT1, u);
      tmem_ldf(t + kT2, v);
      tmem_ldf(t + kT2 + VS, w);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) u[j] = fmaf(phi, v[j] + w[j], u[j]);
      // lanes 16..31 take over the last 8 columns of lanes 0..15
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = __shfl_sync(0xffffffffu, u[j + 8], lane & 15);
        if (lane & 16) u[j] = y;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) split2(be * u[2 * j], be * u[2 * j + 1], hi[j], hi[4 + j]);
      put_piece<VS>(k.base + L::u0, L::row_lo, tok, 2 * cg + (lane >> 4), hi);
      fence_proxy_async_smem();
      k.arrive(C_YOP, lane);
      if (lane == 0) mbar_arrive(&bar[C_GEMPTY + x % kGateRing]);
      // (hi: diag(b) dU)
      *reinterpret_cast<uint4 *>(P.uimg + img - ci * kRowImg) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 y = *reinterpret_cast<const uint4 *>(P.yimg + img + e * kRowImg);
        const uint32_t t[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(u[2 * j], bf16lo(t[j]), fmaf(u[2 * j + 1], bf16hi(t[j]), dot));
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 16);
      if (lane < 16) P.dot[(ci * kC + tok) * 8 + (gcol >> 4)] = dot;
    }
  } else {
    // diag(e^g) dO in two parts: 16 columns of a token at a time
    const uint32_t th = threadIdx.x - 32 * L::side, tok = th & 63;
    bool ok = true;
    RV n;
#pragma unroll 1
    for (int x = 0; x < P.N && ok; ++x, n.advance()) {
      if (!(ok = k.gates_ready(x) && k.full(n) && (x == 0 || k.wait_w(C_ACC, x - 1)))) break;
      const float eg = k.gates(x)[tok];
      const uint32_t src = k.slot(n) + tok * 128;
#pragma unroll
      for (uint32_t cg = th >> 6; cg < VS / 16; cg += 2) {
        uint32_t r[8], hi[8];
        const uint32_t p = (x0 & 63) / 8 + 2 * cg;
        ld_shared_v4(src + ((p ^ (tok & 7u)) << 4), r[0], r[1], r[2], r[3]);
        ld_shared_v4(src + (((p + 1) ^ (tok & 7u)) << 4), r[4], r[5], r[6], r[7]);
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[2 * j] = eg * bf16lo(r[j]);
          v[2 * j + 1] = eg * bf16hi(r[j]);
        }
        put_split<VS>(k.base + L::u1, L::row_lo, tok, cg, v, hi);
      }
      fence_proxy_async_smem();
      k.arrive(C_UOP, lane);
      if (lane == 0) mbar_arrive(&bar[C_GEMPTY + x % kGateRing]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ================================================================== gradients of a chunk
// Chunk after chunk, independent of each other, on one CTA per SM.  Products of the form [dimension x token]
// have lane = dimension; the 64 x 64 ones come from 128-row operands whose other rows are unused: [K; dO]
// stacked gives K K^T in lanes 0..63 and dO Y^T in lanes 64..127.  Warps 0..15 turn products into operands and
// results (16 columns each), warp 16 issues the products, warp 17 loads and stores: the next chunk's tiles arrive
// and its first product runs while the threads are in this one's last step.  Bound by its 224 KB a chunk (0.338 ms
// at B2 H16 T16384: 5.4 TB/s, 0.80 of copy bandwidth) and the latencies between the five steps: the tiles of one
// chunk fill shared memory, so the loads overlap only the last step.
//
// Single bf16 operands except Y in dO Y^T and Y R^T and the matrix A, which have two parts: with one the
// gradients' errors come to 2.9e-3 of their size, 1.75 times the rounding of the results themselves, 1.65e-3 (now
// 1.7e-3 to 2.7e-3; Z, D and the images of S and R would cost another 40 products for at most 0.5e-3).
constexpr int kGradThreads = 576, kGradWarps = 16;
constexpr uint32_t kGrKD = 0, kGrQ = 32768, kGrS = 49152, kGrR = 81920, kGrY = 114688, kGrU = 147456, kGrZ = 163840,
                   kGrA = 180224,           // A hi, A lo, D (8 KiB each); T lives over the last two before them
                   kGrX = 204800, kGrG = 221184, kGrEnd = kGrG + 2 * 1536;
constexpr uint32_t kGrT = kGrA + 8192, kGrD = kGrA + 16384;
constexpr size_t kGradSmem = kGrEnd + 1024;
static_assert(kGradSmem + 4096 <= 232448, "one CTA per SM");
constexpr uint32_t kGZ = 0, kGKK = 64, kGdP = 128, kGGY = 192, kGdq = 256, kGdr = 320, kGdw = 384;
enum { G_UT = 0, G_SR, G_KQ,      // loads: diag(b) dU, T, Y, gates; S, R; K, dO, Q
       G_Z, G_64, G_ALL,          // products: Z; the 64 x 64 ones; all
       G_ZT, G_AD, G_END,         // the threads: Z tile and dv ready; A and D; the chunk's results in place
       G_STORED,                  // dq and dk have left shared memory
       G_COUNT };

__global__ void __launch_bounds__(kGradThreads, 1)
    delta_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mdo, const __grid_constant__ CUtensorMap mdq,
                      const __grid_constant__ CUtensorMap mdk, const __grid_constant__ CUtensorMap mdv,
                      DeltaTcParams P, int items) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  __shared__ uint64_t bar[G_COUNT];
  __shared__ uint32_t tslot;
  __shared__ int abort_flag;
  // (s_rs twice, by the chunk's parity: the next chunk's sums may be written while one thread still adds these up.
  // The others are written behind products that wait for every warp's arrival in the next chunk.)
  __shared__ float s_col[2][kC], s_x[4][kC], s_rs[2][kGradWarps], s_kw[kGradWarps], s_last;
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < G_COUNT; ++i) mbar_init(&bar[i], i == G_ZT || i == G_AD || i == G_END ? kGradWarps : 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tslot, 0);
  griddep_wait();
  auto wait = [&](int i, int parity) {
    return __all_sync(0xffffffffu, mbar_wait_compact(&bar[i], parity & 1, &abort_flag, P.status));
  };
  auto arrive = [&](int i) {
    tc_fence_before();
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[i]);
  };
  const uint32_t KD = base + kGrKD, dO = KD + 8192, Y = base + kGrY, Z = base + kGrZ, S = base + kGrS, R = base + kGrR;
  bool ok = true;

  if (warp == kGradWarps) {
    // contractions over value dimensions: d = 64 has no others (the images hold nothing there)
    const int kd = P.d / 64;
    const uint32_t id_mm = idesc_bf16(128, 64, true, true), id_mk = idesc_bf16(128, 64, true, false),
                   id_km = idesc_bf16(128, 64, false, true), id_kk = idesc_bf16(128, 64, false, false);
    // D (+)= A B over n times four steps of 16; a_step and b_step within four, a_inc and b_inc to the next four
    auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool fresh, int n, uint32_t a_step, uint32_t a_inc,
                   uint32_t b_step, uint32_t b_inc) {
      uint32_t acc = fresh ? 0 : 1;
#pragma unroll 1
      for (int i = 0; i < n; ++i, a += a_inc, b += b_inc) {
#pragma unroll
        for (uint32_t ks = 0; ks < 4; ++ks, acc = 1) mma_ss_warp(tmem + d, a + ks * a_step, b + ks * b_step, id, acc);
      }
    };
    constexpr uint32_t kK = 2, kM = 128, k8 = 8192 >> 4, k16 = 16384 >> 4;  // K-major and MN-major steps; blocks
    int x = 0;
#pragma unroll 1
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++x) {
      const uint64_t y = k_tile(Y), ylo = k_tile(Y + 16384), zm = mn_tile(Z, 16384), sk = k_tile(S), rk = k_tile(R),
                     km = mn_tile(KD, 16384), kk = k_tile(KD), am = mn_tile(base + kGrA, 8192), ak = k_tile(base + kGrA),
                     dm = mn_tile(base + kGrD, 8192), dk = k_tile(base + kGrD), qm = mn_tile(base + kGrQ, 8192);
      if (!(ok = wait(G_UT, x))) break;
      tc_fence_after();
      // Z^T = (diag(b) dU)^T T
      mma(kGZ, mn_tile(base + kGrU, 8192), mn_tile(base + kGrT, 8192), id_mm, true, 2, kM, 0, 2 * kM, kM);
      mma_commit_warp(&bar[G_Z]);
      // (the accumulators that follow are read in the last chunk's last step)
      if (!(ok = wait(G_KQ, x) && (x == 0 || wait(G_END, x - 1)))) break;
      tc_fence_after();
      mma(kGKK, kk, kk, id_kk, true, 2, kK, k16, kK, k16);                 // K K^T (lanes 0..63)
      mma(kGdP, kk, y, id_kk, true, kd, kK, k16, kK, k8);                  // dO Y^T (lanes 64..127)
      mma(kGdP, kk, ylo, id_kk, false, kd, kK, k16, kK, k8);
      if (!(ok = wait(G_ZT, x))) break;
      tc_fence_after();
      mma(kGGY, zm, y, id_mk, true, kd, kM, 4 * kM, kK, k8);               // Z Y^T (lanes 0..63)
      mma_commit_warp(&bar[G_64]);
      if (!(ok = wait(G_SR, x))) break;
      tc_fence_after();
      mma(kGdr, sk, zm, id_km, true, kd, kK, k16, kM, 4 * kM);             // (Z S^T)^T
      mma(kGdq, sk, k_tile(dO), id_kk, true, kd, kK, k16, kK, k16);        // (dO S^T)^T
      mma(kGdw, rk, y, id_kk, true, kd, kK, k16, kK, k8);                  // (Y R^T)^T
      mma(kGdw, rk, ylo, id_kk, false, kd, kK, k16, kK, k8);
      if (!(ok = wait(G_AD, x))) break;
      tc_fence_after();
      mma(kGKK, km, ak, id_mk, true, 2, kM, 0, kK, k8);                    // (A K)^T
      mma(kGdP, km, dk, id_mk, true, 1, kM, 0, kK, 0);                     // (D K)^T
      mma(kGGY, qm, am, id_mm, true, 2, kM, 0, kM, k8);                    // (A^T Q + D^T K)^T
      mma(kGGY, km, dm, id_mm, false, 1, kM, 0, kM, 0);
      mma_commit_warp(&bar[G_ALL]);
    }
  } else if (warp > kGradWarps) {
    if (lane == 0) {
      auto await = [&](int i, int x) { return mbar_wait_compact(&bar[i], x & 1, &abort_flag, P.status); };
      auto load = [&](int item, int g) {
        const int c = item % P.N, bh = item / P.N, b = bh / P.H, h = bh % P.H;
        const uint8_t *rec = P.rec + (int64_t)item * kRecBytes;
        mbar_arrive_expect_tx(&bar[G_UT], 16384 + kGateBytes + 16384 + 32768);
        bulk_load(&bar[G_UT], smem + kGrU, P.uimg + (int64_t)item * kRowImg, 16384);
        bulk_load(&bar[G_UT], smem + kGrT, rec + kRecT, 16384);
        bulk_load(&bar[G_UT], smem + kGrG + g * 1536, rec + kRecG, kGateBytes);
        bulk_load(&bar[G_UT], smem + kGrY, P.yimg + (int64_t)item * kYImg, 32768);
        mbar_arrive_expect_tx(&bar[G_KQ], 49152);
        for (int x = 0; x < 2; ++x) {
          tma_load_4d(&mk, &bar[G_KQ], smem + kGrKD + x * 16384, 64 * x, kC * c, h, b, kPolicyEvictFirst);
          tma_load_4d(&mdo, &bar[G_KQ], smem + kGrKD + x * 16384 + 8192, 64 * x, kC * c, h, b, kPolicyEvictFirst);
          tma_load_4d(&mq, &bar[G_KQ], smem + kGrQ + x * 8192, 64 * x, kC * c, h, b, kPolicyEvictFirst);
        }
        mbar_arrive_expect_tx(&bar[G_SR], 65536);
        bulk_load(&bar[G_SR], smem + kGrS, P.simg + (int64_t)item * kStateImg, 32768);
        bulk_load(&bar[G_SR], smem + kGrR, P.rimg + (int64_t)item * kStateImg, 32768);
      };
      auto store = [&](const CUtensorMap *m, uint32_t from, int item) {
        const int c = item % P.N, bh = item / P.N, b = bh / P.H, h = bh % P.H;
        for (int y = 0; y < P.d / 64; ++y) tma_store_4d(m, smem + from + y * 8192, 64 * y, kC * c, h, b);
        bulk_commit();
      };
      int x = 0, loaded = 0;
      if ((int)blockIdx.x < items) load(blockIdx.x, 0);
#pragma unroll 1
      for (int item = blockIdx.x; item < items; item += gridDim.x, ++x) {
        if (!(ok = await(G_ZT, x))) break;
        store(&mdv, kGrU, item);
        if (!(ok = await(G_ALL, x))) break;
        bulk_wait_read_all();  // dv has left the place that the next chunk's diag(b) dU takes
        if (item + (int)gridDim.x < items) {
          load(item + gridDim.x, (x + 1) & 1);
          ++loaded;
        }
        if (!(ok = await(G_END, x))) break;
        store(&mdq, kGrZ, item);
        store(&mdk, kGrX, item);
        bulk_wait_read_all();
        mbar_arrive(&bar[G_STORED]);
      }
      bulk_wait_all();
      if (!ok) {  // after an abort, with limits: what is in flight lands before the block ends
        volatile int no_abort = 0;
        for (int i = G_UT; i <= G_KQ; ++i) mbar_wait_compact(&bar[i], loaded & 1, &no_abort, P.status);
      }
    }
    __syncwarp();
  } else {
    // 32 lanes (dimensions, or rows of a 64 x 64 product) and 16 columns of every product, as two fragments
    const uint32_t quad = warp & 3, cg = warp >> 2, t = tmem + ((quad * 32) << 16) + 16 * cg;
    auto frag = [&](uint32_t col, uint32_t hh, float (&f)[8]) { tmem_ld_frag(t + col + (hh << 20), f); };
    // the threads' part of the x-th chunk; false when a wait gave up
    auto step = [&](int x) {
      const float *g = reinterpret_cast<const float *>(smem + kGrG + (x & 1) * 1536);
      // Z: an operand tile (row = value dimension), where dq was, and dv, where dU was
      if (!(wait(G_Z, x) && (x == 0 || wait(G_STORED, x - 1)))) return false;
      tc_fence_after();
#pragma unroll 1
      for (uint32_t hh = 0; hh < 2; ++hh) {
        float z[8];
        uint32_t p[4];
        frag(kGZ, hh, z);
        tmem_ld_wait();
        frag_pack(z, p);
        stmatrix4(Z + frag_at(lane, quad * 32 + 16 * hh, cg), p);
        stmatrix4_trans(base + kGrU + frag_at_trans(lane, 16 * cg, quad * 32 + 16 * hh, 8192), p);
      }
      arrive(G_ZT);
      // <R, S> of the chunk's two states (its end's needs the tokens' writes added: below)
      if (!wait(G_SR, x)) return false;
      {
        float dot = 0.f;
        const uint32_t at = (cg >> 1) * 16384;
#pragma unroll
        for (uint32_t p = 0; p < 4; ++p) {
          uint32_t u[4], v[4];
          const uint32_t o = at + sw(quad * 32 + lane, 4 * (cg & 1) + p);
          ld_shared_v4(S + o, u[0], u[1], u[2], u[3]);
          ld_shared_v4(R + o, v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = fmaf(bf16lo(u[e]), bf16lo(v[e]), fmaf(bf16hi(u[e]), bf16hi(v[e]), dot));
        }
#pragma unroll
        for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) s_rs[x & 1][warp] = 32 * (int)cg < P.d ? dot : 0.f;
      }
      // this lane's four columns
      float be[4], jh[4], jl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * cg + frag_token(lane, e);
        be[e] = g[128 + j];
        jh[e] = g[192 + j];
        jl[e] = g[256 + j];
      }
      // q and k of the last step, so that their tiles are free before it
      uint32_t qf[2][4], kf[2][4];
      if (!wait(G_KQ, x)) return false;
#pragma unroll
      for (uint32_t hh = 0; hh < 2; ++hh) {
        ldmatrix4_trans(base + kGrQ + frag_at_trans(lane, 16 * cg, quad * 32 + 16 * hh, 8192), qf[hh]);
        ldmatrix4_trans(KD + frag_at_trans(lane, 16 * cg, quad * 32 + 16 * hh, 16384), kf[hh]);
      }
      if (!wait(G_64, x)) return false;
      tc_fence_after();
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (uint32_t hh = 0; hh < 2; ++hh) {
        const uint32_t row0 = (quad & 1) * 32 + 16 * hh;
        float a[8], zy[8];
        frag(quad < 2 ? kGKK : kGdP, hh, a);
        if (quad < 2) frag(kGGY, hh, zy);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = frag_col(i), r = row0 + lane / 4 + (i & 2 ? 8 : 0), j = 16 * cg + frag_token(lane, e);
          const float gam = ex2((g[192 + r] - jh[e]) + (g[256 + r] - jl[e]));
          if (quad < 2) {
            // D_ij = -b_j Gam_ij z_i . y_j, and the parts of sum_i Gam_ij (k_i . k_j) (z_i . y_j)
            const float v = j < r ? gam * zy[i] : 0.f;
            sum[e] += j < r ? v * a[i] : 0.f;
            a[i] = -be[e] * v;
          } else {
            a[i] = j <= r ? gam * be[e] * a[i] : 0.f;  // A_ij = b_j Gam_ij dO_i . y_j
          }
        }
        uint32_t p[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2(a[2 * i], a[2 * i + 1], p[i], l[i]);
        const uint32_t at = base + (quad < 2 ? kGrD : kGrA) + frag_at(lane, row0, cg);
        stmatrix4(at, p);
        if (quad >= 2) stmatrix4(at + 8192, l);
      }
      arrive(G_AD);
      if (quad < 2) {
        frag_col_sum(sum);
        if (lane < 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) s_col[quad][16 * cg + frag_token(lane, e)] = sum[e];
      }
      float eg[4], pb[4], w[4] = {0.f, 0.f, 0.f, 0.f}, kw = 0.f;  // kw: sum of phi b k^T R y
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * cg + frag_token(lane, e);
        eg[e] = g[j];
        pb[e] = g[64 + j] * be[e];
      }
      if (!wait(G_ALL, x)) return false;
      tc_fence_after();
      // lane = key dimension; w gathers q . dq + k . (read - write part)
#pragma unroll
      for (uint32_t hh = 0; hh < 2; ++hh) {
        const uint32_t row0 = quad * 32 + 16 * hh, at = frag_at_trans(lane, 16 * cg, row0, 8192);
        float a[8], b[8];
        uint32_t p[4];
        frag(kGdq, hh, a);
        frag(kGKK, hh, b);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = fmaf(eg[frag_col(i)], a[i], b[i]);
          w[frag_col(i)] = fmaf(a[i], i & 1 ? bf16hi(qf[hh][i / 2]) : bf16lo(qf[hh][i / 2]), w[frag_col(i)]);
        }
        frag_pack(a, p);
        stmatrix4_trans(Z + at, p);
        float f[8], u[8];
        frag(kGdr, hh, a);
        frag(kGdP, hh, b);
        frag(kGdw, hh, f);
        frag(kGGY, hh, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = frag_col(i);
          const float kv = i & 1 ? bf16hi(kf[hh][i / 2]) : bf16lo(kf[hh][i / 2]), r = pb[e] * f[i];
          const float read = fmaf(-eg[e], a[i], b[i]), write = r + u[i];
          kw = fmaf(kv, r, kw);
          w[e] = fmaf(read - write, kv, w[e]);
          a[i] = read + write;
        }
        frag_pack(a, p);
        stmatrix4_trans(base + kGrX + at, p);
      }
#pragma unroll
      for (int o = 16; o; o /= 2) kw += __shfl_xor_sync(0xffffffffu, kw, o);
      if (lane == 0) s_kw[warp] = kw;
      frag_col_sum(w);
      if (lane < 4)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_x[quad][16 * cg + frag_token(lane, e)] = w[e];
      if (tid == kC) s_last = g[63];
      arrive(G_END);
      return true;
    };
    int x = 0;
#pragma unroll 1
    for (int item = blockIdx.x; item < items; item += gridDim.x, ++x) {
      // one verdict for all warps: none is left alone in the barrier
      if (!(ok = group_all(step(x), 1, 32 * kGradWarps))) break;
      const int c = item % P.N, bh = item / P.N;
      if (tid < kC) {
        const int j = tid;
        const int64_t ci = (int64_t)bh * P.N + c, at = (int64_t)bh * P.T + kC * c + j;
        if (kC * c + j < P.T) {
          P.gx[at] = (s_x[0][j] + s_x[1][j]) + (s_x[2][j] + s_x[3][j]);
          float db = -(s_col[0][j] + s_col[1][j]);
          const float *dot = P.dot + (ci * kC + j) * 8;
          for (int y = 0; y < P.d / 16; ++y) db += dot[y];
          if (P.f32)
            static_cast<float *>(P.dbeta)[at] = db;
          else
            static_cast<__nv_bfloat16 *>(P.dbeta)[at] = __float2bfloat16_rn(db);
        }
      } else if (tid == kC) {
        float rs = 0.f, kws = 0.f;
        for (int y = 0; y < kGradWarps; ++y) {
          rs += s_rs[x & 1][y];
          kws += s_kw[y];
        }
        P.anchor[(int64_t)bh * P.N + c] = fmaf(s_last, rs, kws);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

bool seq64_tmap(const Problem &p, const void *x, CUtensorMap *m) {
  // d = 64: the box of columns 64..127 lies past the rows' end; loads fill zeros there
  const uint64_t dims[4] = {(uint64_t)p.d, (uint64_t)p.T, (uint64_t)p.H, (uint64_t)p.B};
  const uint64_t strides[3] = {(uint64_t)p.st * 2, (uint64_t)p.sh * 2, (uint64_t)p.sb * 2};
  return make_tmap_bf16(m, x, dims, strides, 64);
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// The reverse chain's slices: of 32 value dimensions while all the chains run at once with one CTA per SM, else
// of 64 (a chunk takes 1.5 times as long: 153 us at B2 H32 T4096, where slices of 32 would take two turns of 102).
bool narrow_slices(const Problem &p) { return (int64_t)p.B * p.H * (p.d / 32) <= p.num_sms; }
int chunks(const Problem &p) { return (p.T + kC - 1) / kC; }
size_t bhs(const Problem &p) { return (size_t)p.B * p.H; }
size_t rec_bytes(const Problem &p) { return bhs(p) * chunks(p) * kRecBytes; }

DeltaTcParams params(const Problem &p, const DeltaGates &g, int *status) {
  DeltaTcParams P{};
  P.H = p.H;
  P.T = p.T;
  P.N = chunks(p);
  P.d = p.d;
  P.f32 = g.f32;
  P.lg = g.lg;
  P.beta = g.beta;
  P.status = status;
  return P;
}

}  // namespace

bool delta_tc_supported(const Problem &p) { return p.dtype == 0; }
size_t delta_tc_fwd_ws_bytes(const Problem &p) { return align256(rec_bytes(p)); }
size_t delta_tc_ckpt_bytes(const Problem &p) {
  if (p.T == 0) return 0;
  return align256(rec_bytes(p) + bhs(p) * chunks(p) * (kStateImg + kYImg));
}
size_t delta_tc_bwd_ws_bytes(const Problem &p) {
  const size_t n = bhs(p) * chunks(p);
  return align256(n * (kStateImg + kRowImg + (8 * kC + 1) * sizeof(float)) + bhs(p) * p.T * sizeof(float));
}

cudaError_t delta_tc_fwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v, void *o,
                         const float *init, float *fin, void *ckpt, void *ws, int *status, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  if (!seq64_tmap(p, q, &mq) || !seq64_tmap(p, k, &mk) || !seq64_tmap(p, v, &mv)) return cudaErrorInvalidValue;
  DeltaTcParams P = params(p, g, status);
  P.rec = static_cast<uint8_t *>(ckpt ? ckpt : ws);
  if (ckpt) {
    P.simg = P.rec + rec_bytes(p);
    P.yimg = P.simg + bhs(p) * (size_t)P.N * kStateImg;
  }
  P.in = init;
  P.out = fin;
  cudaError_t e = allow_smem(delta_prep_kernel, kPrepSmem);
  if (e != cudaSuccess) return e;
  {
    TimedLaunch t(K_DELTA_PREP, s);
    e = launch_overlapped(delta_prep_kernel, dim3((unsigned)(bhs(p) * P.N)), dim3(kPrepThreads), kPrepSmem, s, mq, mk, P);
    if (e != cudaSuccess) return e;
  }
  if ((e = allow_smem(delta_chain_kernel, kChain::smem)) != cudaSuccess) return e;
  TimedLaunch t(K_DELTA_CHAIN, s);
  return launch_overlapped(delta_chain_kernel, dim3((unsigned)(bhs(p) * (p.d / kSlice))), dim3(kChain::threads),
                           kChain::smem, s, mq, mk, mv, static_cast<__nv_bfloat16 *>(o), p.sb, p.sh, p.st, P);
}

cudaError_t delta_tc_bwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *dO,
                         const float *d_final, const void *ckpt, void *dq, void *dk, void *dv, void *dlg, void *dbeta,
                         float *dinit, void *ws, int *status, cudaStream_t s) {
  CUtensorMap mq, mk, mdo, mdq, mdk, mdv;
  if (!seq64_tmap(p, q, &mq) || !seq64_tmap(p, k, &mk) || !seq64_tmap(p, dO, &mdo) || !seq64_tmap(p, dq, &mdq) ||
      !seq64_tmap(p, dk, &mdk) || !seq64_tmap(p, dv, &mdv))
    return cudaErrorInvalidValue;
  DeltaTcParams P = params(p, g, status);
  const size_t n = bhs(p) * P.N;
  P.rec = const_cast<uint8_t *>(static_cast<const uint8_t *>(ckpt));
  P.simg = P.rec + rec_bytes(p);
  P.yimg = P.simg + bhs(p) * (size_t)P.N * kStateImg;
  P.rimg = static_cast<uint8_t *>(ws);
  P.uimg = P.rimg + n * kStateImg;
  P.dot = reinterpret_cast<float *>(P.uimg + n * kRowImg);
  P.anchor = P.dot + n * kC * 8;
  P.gx = P.anchor + n;
  P.dbeta = dbeta;
  P.in = d_final;
  P.out = dinit;
  cudaError_t e = allow_smem(delta_grad_kernel, kGradSmem);
  if (e != cudaSuccess) return e;
  auto reverse = [&](auto kernel, int slice, int threads, size_t smem) {
    cudaError_t err = allow_smem(kernel, smem);
    if (err != cudaSuccess) return err;
    TimedLaunch t(K_DELTA_REVERSE, s);
    return launch_overlapped(kernel, dim3((unsigned)(bhs(p) * (p.d / slice))), dim3(threads), smem, s, mq, mk, mdo, P);
  };
  e = narrow_slices(p) ? reverse(delta_reverse_kernel<32>, 32, Chain<32>::threads, Chain<32>::smem)
                       : reverse(delta_reverse_kernel<64>, 64, Chain<64>::threads, Chain<64>::smem);
  if (e != cudaSuccess) return e;
  {
    TimedLaunch t(K_DELTA_GRAD, s);
    const int items = (int)n, grid = items < p.num_sms ? items : p.num_sms;
    e = launch_overlapped(delta_grad_kernel, dim3(grid), dim3(kGradThreads), kGradSmem, s, mq, mk, mdo,
                          mdq, mdk, mdv, P, items);
    if (e != cudaSuccess) return e;
  }
  return dlg ? delta_gate_sums(p, P.gx, P.anchor, dlg, g.f32, s) : cudaSuccess;
}

}  // namespace linattn
