// Gated delta rule on the CUDA cores: the fp32 path (and the recurrent decode, fp32 or bf16).
//
//     S'_t = a_t S_{t-1},   y_t = v_t - S'_t^T k_t,   S_t = S'_t + k_t (b_t y_t)^T,   o_t = S_t^T q_t
//
// (a_t = exp(log_gate_t), b_t the write strength; S is d_k x d_v, fp32).  Backward, with R the
// gradient arriving at S_t from later tokens (d_final_state at the end):
//
//     R += q_t dO_t^T;  du = R^T k_t;  dy = b_t du;  dv_t = dy;  db_t = du . y_t;
//     dk_t = R (b_t y_t) - S'_t dy;  dq_t = S_t dO_t;  R <- a_t (R - k_t dy^T).
//
// The log-gates enter only as the factor of the state between two tokens, so with
// G_t = q_t . dq_t + k_t . (the read part of dk_t) - k_t . (its write part), the gradient of the
// cumulative log-gate at t, and <R, S> at a chunk's end, the sum of G over all later tokens:
//     d_log_gate_t = sum of G from t to the chunk's end + <R, S> there.
// (Anchoring at every chunk keeps the sums short: a sum over the whole rest of the sequence would
// gather the rounding of every later token.)
//
// Four walks over the tokens, none of which waits for another warp: a warp owns four columns of S (or, once
// y and dy are known, four rows), eight lanes each, so the sums over a column (row) are three shuffles.
//     outputs:  forward over the columns of S     o, y, and S where every chunk begins
//     reverse:  backward over the columns of R    dv, dy, parts of db, R and <R, S> where every chunk ends
//     writes:   backward over the rows of R       the write part of dk, all chunks at once
//     reads:    forward over the rows of S        dq, dk, all chunks at once
// A CTA of four warps stages blocks of 8 tokens in shared memory while it walks the block before.  D/16
// CTAs per (batch, head), and per chunk in the last two; bound by the latency of a token's sums.  A training
// step of 257 tokens (B1 H2 d64) takes 167 us; with one CTA per (batch, head), the matrix in its registers
// and three block barriers a token it took 625 us, and with the last two walks uncut 254 us.
#include <cuda_bf16.h>
#include "internal.h"
#include "ptx.cuh"

namespace linattn {
namespace {

constexpr int kWalkThreads = 128, kBlockT = 8, kVecs = 16;  // tokens staged at a time; rows or columns of a CTA

__device__ __forceinline__ float ld_gate(const void *p, int64_t i, int f32) {
  return f32 ? static_cast<const float *>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void st_gate(void *p, int64_t i, int f32, float x) {
  if (f32)
    static_cast<float *>(p)[i] = x;
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}
__device__ __forceinline__ float ld_val(const float *p) { return *p; }
__device__ __forceinline__ float ld_val(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_val(float *p, float x) { *p = x; }
__device__ __forceinline__ void st_val(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

enum { W_OUTPUTS = 0, W_REVERSE, W_WRITES, W_READS };

// What a walk reads per token: up to three rows of D values and up to three pieces of kVecs (its own columns
// or rows), each with its row stride; pointers already at the (batch, head).
struct WalkRows {
  const float *row[3], *vec[3];
  int64_t row_st[3], vec_st[3];
};
struct WalkArgs {
  const float *q, *k, *v, *dO;      // user tensors
  float *o, *dq, *dk, *dv;          // (strides of the Problem)
  float *y, *dy, *dkw;              // [BH][T][D]
  float *states, *grads;            // [BH][N + 1][D][D] S, or null; [BH][N][D][D] R
  const float *in;                  // initial state, or the final state's gradient, or null
  float *out;                       // final state, or the initial state's gradient, or null
  float *xpart, *dbpart, *apart;    // [BH][T][D/4], [BH][T][D/4], [BH][N][D/4]: one value per warp
};

// sum over the eight lanes of a column (row)
__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int o = 1; o < 8; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// ... and over the warp's four of them
__device__ __forceinline__ float sum4(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kWalkThreads) delta_walk(Problem p, DeltaGates g, WalkArgs w) {
  constexpr bool kForward = MODE == W_OUTPUTS || MODE == W_READS, kColumns = MODE == W_OUTPUTS || MODE == W_REVERSE;
  constexpr int NV = MODE == W_OUTPUTS ? 1 : MODE == W_READS ? 3 : 2, NRW = kColumns ? 2 : 3, NE = D / 32;  // float4s
  __shared__ float4 rows[2][NRW][kBlockT][D / 4];
  __shared__ float4 vecs[2][NV][kBlockT][kVecs / 4];
  __shared__ float gates[2][2][kBlockT];
  constexpr int slices = D / kVecs;
  const int N = (p.T + 63) / 64, seq = blockIdx.x / slices, bh = kColumns ? seq : seq / N, chunk = kColumns ? 0 : seq % N;
  const int b = bh / p.H, h = bh % p.H, x0 = (blockIdx.x % slices) * kVecs;
  const int begin = chunk * 64, end = kColumns ? p.T : min(p.T, begin + 64);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, x = x0 + 4 * warp + (lane >> 3), e0 = (lane & 7) * 4;
  const int64_t user = (int64_t)b * p.sb + (int64_t)h * p.sh, own = (int64_t)bh * p.T * D, gb = (int64_t)bh * p.T;
  const int part = x0 / 4 + warp;
  WalkRows in;
  auto row = [&](int i, const float *t, bool is_user) {
    in.row[i] = t + (is_user ? user : own);
    in.row_st[i] = is_user ? p.st : D;
  };
  auto vec = [&](int i, const float *t, bool is_user) {
    in.vec[i] = t + (is_user ? user : own) + x0;
    in.vec_st[i] = is_user ? p.st : D;
  };
  if (kColumns) {
    row(0, w.k, true);
    row(1, w.q, true);
    vec(0, MODE == W_OUTPUTS ? w.v : w.dO, true);
    if (MODE == W_REVERSE) vec(1, w.y, false);
  } else {
    row(0, w.dO, true);
    row(1, w.dy, false);
    row(2, w.y, false);
    vec(0, w.q, true);
    vec(1, w.k, true);
    if (MODE == W_READS) vec(2, w.dkw, false);
  }
  // block i of the walk: tokens t0 .. (in time order inside)
  const int blocks = (end - begin + kBlockT - 1) / kBlockT;
  auto first = [&](int i) { return begin + (kForward ? i : blocks - 1 - i) * kBlockT; };
  auto stage = [&](int i) {
    const int t0 = first(i), n = min(kBlockT, end - t0), s = i & 1;
#pragma unroll
    for (int a = 0; a < NRW; ++a)
#pragma unroll
      for (int e = tid; e < kBlockT * (D / 4); e += kWalkThreads) {
        const int c = e % (D / 4), t = e / (D / 4);
        if (t < n) cp_async16(smem_u32(&rows[s][a][t][c]), in.row[a] + (t0 + t) * in.row_st[a] + 4 * c);
      }
    static_assert(kBlockT * (kVecs / 4) == 32, "one warp stages one array's pieces");
#pragma unroll
    for (int a = 0; a < NV; ++a)
      if (warp == a && lane / 4 < n)
        cp_async16(smem_u32(&vecs[s][a][lane / 4][lane % 4]),
                   in.vec[a] + (t0 + lane / 4) * in.vec_st[a] + 4 * (lane % 4));
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < n) {
      gates[s][0][tid] = g.lg ? expf(ld_gate(g.lg, gb + t0 + tid, g.f32)) : 1.f;
      gates[s][1][tid] = ld_gate(g.beta, gb + t0 + tid, g.f32);
    }
  };
  // element 4 m + c of this lane's part of its column (row) is entry e0 + 32 m + c
  auto at = [&](const float *m, int i, int c) {
    const int e = e0 + 32 * i + c;
    return m + (kColumns ? (int64_t)e * D + x : (int64_t)x * D + e);
  };
  float4 s[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float *m = MODE == W_READS    ? w.states + ((int64_t)bh * (N + 1) + chunk) * D * D
                     : MODE == W_WRITES ? w.grads + ((int64_t)bh * N + chunk) * D * D
                     : w.in             ? w.in + (int64_t)bh * D * D
                                        : nullptr;
    s[i] = m ? make_float4(*at(m, i, 0), *at(m, i, 1), *at(m, i, 2), *at(m, i, 3)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto store = [&](float *m) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      *const_cast<float *>(at(m, i, 0)) = s[i].x;
      *const_cast<float *>(at(m, i, 1)) = s[i].y;
      *const_cast<float *>(at(m, i, 2)) = s[i].z;
      *const_cast<float *>(at(m, i, 3)) = s[i].w;
    }
  };
  auto dot = [](float4 a, float4 b, float c) { return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c)))); };
  auto axpy = [](float f, float4 a, float4 b) {  // f a + b
    return make_float4(fmaf(f, a.x, b.x), fmaf(f, a.y, b.y), fmaf(f, a.z, b.z), fmaf(f, a.w, b.w));
  };
  auto scale = [](float f, float4 a) { return make_float4(f * a.x, f * a.y, f * a.z, f * a.w); };
  stage(0);
#pragma unroll 1
  for (int i = 0; i < blocks; ++i) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // block i is in place, and block i - 1's place is free
    if (i + 1 < blocks) stage(i + 1);
    const int t0 = first(i), n = min(kBlockT, end - t0), z = i & 1;
#pragma unroll 1
    for (int u = 0; u < n; ++u) {
      const int tt = kForward ? u : n - 1 - u, t = t0 + tt;
      const float a = gates[z][0][tt], be = gates[z][1][tt];
      float4 r[NRW][NE];
#pragma unroll
      for (int m = 0; m < NRW; ++m)
#pragma unroll
        for (int e = 0; e < NE; ++e) r[m][e] = rows[z][m][tt][(lane & 7) + 8 * e];
      float c[NV];
#pragma unroll
      for (int m = 0; m < NV; ++m) c[m] = reinterpret_cast<const float *>(vecs[z][m][tt])[x - x0];
      const bool lead = (lane & 7) == 0;
      const int64_t mine = own + (int64_t)t * D + x, theirs = user + (int64_t)t * p.st + x;
      if (MODE == W_OUTPUTS) {
        // rows k, q; c: v_j
        if (w.states && t % 64 == 0) store(w.states + ((int64_t)bh * (N + 1) + t / 64) * D * D);
        float sk = 0.f, sq = 0.f, kq = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          sk = dot(s[e], r[0][e], sk);
          sq = dot(s[e], r[1][e], sq);
          kq = dot(r[0][e], r[1][e], kq);
        }
        sk = sum8(sk);
        sq = sum8(sq);
        kq = sum8(kq);
        const float y = fmaf(-a, sk, c[0]), uj = be * y;
#pragma unroll
        for (int e = 0; e < NE; ++e) s[e] = axpy(uj, r[0][e], scale(a, s[e]));
        if (lead) {
          w.o[theirs] = fmaf(kq, uj, a * sq);
          if (w.y) w.y[mine] = y;
        }
      } else if (MODE == W_REVERSE) {
        // rows k, q; c: dO_j, y_j
        if (t == p.T - 1 || t % 64 == 63) {
          const float *S = w.states + ((int64_t)bh * (N + 1) + t / 64 + 1) * D * D;
          store(w.grads + ((int64_t)bh * N + t / 64) * D * D);
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < NE; ++e)
            d = dot(s[e], make_float4(*at(S, e, 0), *at(S, e, 1), *at(S, e, 2), *at(S, e, 3)), d);
          d = sum4(sum8(d));
          if (lane == 0) w.apart[((int64_t)bh * N + t / 64) * (D / 4) + part] = d;
        }
        float du = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          s[e] = axpy(c[0], r[1][e], s[e]);
          du = dot(s[e], r[0][e], du);
        }
        du = sum8(du);
        const float dy = be * du, db = sum4(du * c[1]);
#pragma unroll
        for (int e = 0; e < NE; ++e) s[e] = scale(a, axpy(-dy, r[0][e], s[e]));
        if (lead) {
          w.dv[theirs] = dy;
          w.dy[mine] = dy;
        }
        if (lane == 0) w.dbpart[(gb + t) * (D / 4) + part] = db;
      } else {
        // rows dO, dy, y; c: q_i, k_i (and dkw_i)
        float d0 = 0.f, d1 = 0.f;
        if (MODE == W_WRITES) {
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            s[e] = axpy(c[0], r[0][e], s[e]);
            d0 = dot(s[e], r[2][e], d0);
            s[e] = scale(a, axpy(-c[1], r[1][e], s[e]));
          }
          d0 = be * sum8(d0);
          d1 = sum4(-c[1] * d0);
          if (lead) w.dkw[mine] = d0;
        } else {
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            s[e] = scale(a, s[e]);
            d0 = dot(s[e], r[1][e], d0);
            s[e] = axpy(be * c[1], r[2][e], s[e]);
            d1 = dot(s[e], r[0][e], d1);
          }
          d0 = -sum8(d0);
          d1 = sum8(d1);
          if (lead) {
            w.dq[theirs] = d1;
            w.dk[theirs] = d0 + c[NV - 1];
          }
          d1 = sum4(fmaf(c[0], d1, c[1] * d0));
        }
        if (lane == 0) w.xpart[(gb + t) * (D / 4) + part] = d1;
      }
    }
  }
  if (kColumns && w.out) store(w.out + (int64_t)bh * D * D);
  if (MODE == W_OUTPUTS && w.states) store(w.states + ((int64_t)bh * (N + 1) + N) * D * D);
}

// The warps' parts added up, in order: G (its two walks' parts), db and the anchors.  One thread each.
__global__ void __launch_bounds__(256) delta_walk_sums(int64_t tokens, int64_t chunks, int parts, const float *x0,
                                                       const float *x1, const float *dbpart, const float *apart,
                                                       float *gx, void *dbeta, int f32, float *anchor) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < tokens) {
    float x = 0.f, d = 0.f;
    for (int j = 0; j < parts; ++j) {
      x += x0[i * parts + j] + x1[i * parts + j];
      d += dbpart[i * parts + j];
    }
    gx[i] = x;
    st_gate(dbeta, i, f32, d);
  } else if (i - tokens < chunks) {
    float d = 0.f;
    for (int j = 0; j < parts; ++j) d += apart[(i - tokens) * parts + j];
    anchor[i - tokens] = d;
  }
}

// d_log_gate: the sums of G from every token to its chunk's end, plus the chunk's anchor.  One warp per chunk
// of 64 tokens; bound by its launch (4 us at B2 H16 T4096).
__global__ void delta_gate_grad(int64_t BH, int T, int N, const float *gx, const float *anchor, void *dlg, int f32) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x % 32;
  if (w >= BH * N) return;
  const int64_t bh = w / N;
  const int c = (int)(w % N), t0 = c * 64 + 2 * lane;
  const float x0 = t0 < T ? gx[bh * T + t0] : 0.f, x1 = t0 + 1 < T ? gx[bh * T + t0 + 1] : 0.f;
  float s = x0 + x1;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const float y = __shfl_down_sync(0xffffffffu, s, o);
    if (lane + o < 32) s += y;
  }
  s += anchor[w];
  if (t0 < T) st_gate(dlg, bh * T + t0, f32, s);
  if (t0 + 1 < T) st_gate(dlg, bh * T + t0 + 1, f32, s - x0);
}

// ------------------------------------------------------------------ recurrent decode
// As the library's linear decode: CS CTAs of 8 warps per sequence, each owning D/CS columns of the
// state in registers.  Both column reductions run on the state before the update,
//     y = v - a S^T k,   u = b y,   o = a S^T q + (q . k) u,   S <- a S + k u^T,
// so a token takes one reduction across the warps.  Bound by the state's read and write (2 x 64 KiB per head at
// d = 128): 157 us at B512 H16, 1.01 of copy bandwidth, with 8-byte accesses marked as passing through (168 us with
// single floats, 163 without the marks).
constexpr int kDecThreads = 256;

template <int D, int CS, typename T>
__global__ void __launch_bounds__(kDecThreads) delta_decode_kernel(Problem p, DeltaGates g, const T *q, const T *k,
                                                                   const T *v, T *o, float *state) {
  constexpr int W = D / CS, NC = W / 32, NR = D / 8;
  static_assert(NC == 2, "a lane's columns are one float2");
  __shared__ float kk[D], qq[D], pk[8][W], pq[8][W], uu[W], dots[8];
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * W;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t off = (int64_t)b * p.sb + (int64_t)h * p.sh, gb = (int64_t)bh * p.T;
  float *base = state + (int64_t)bh * D * D + c0 + NC * lane;
  float s[NR][NC];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const float2 x = __ldcs(reinterpret_cast<const float2 *>(base + (warp + 8 * i) * D));
    s[i][0] = x.x;
    s[i][1] = x.y;
  }
  for (int t = 0; t < p.T; ++t) {
    const int64_t row = off + (int64_t)t * p.st;
    const float a = g.lg ? expf(ld_gate(g.lg, gb + t, g.f32)) : 1.f, be = ld_gate(g.beta, gb + t, g.f32);
    float x = 0.f;
    if (tid < D) {
      kk[tid] = ld_val(k + row + tid);
      qq[tid] = ld_val(q + row + tid);
      x = kk[tid] * qq[tid];
    }
    const float vj = tid < W ? ld_val(v + row + c0 + tid) : 0.f;
#pragma unroll
    for (int m = 16; m; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lane == 0) dots[warp] = x;
    __syncthreads();
    float ak[NC], aq[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) ak[c] = aq[c] = 0.f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float kr = kk[warp + 8 * i], qr = qq[warp + 8 * i];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        ak[c] = fmaf(s[i][c], kr, ak[c]);
        aq[c] = fmaf(s[i][c], qr, aq[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      pk[warp][NC * lane + c] = ak[c];
      pq[warp][NC * lane + c] = aq[c];
    }
    __syncthreads();
    if (tid < W) {
      float sk = 0.f, sq = 0.f, qk = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        sk += pk[w][tid];
        sq += pq[w][tid];
        qk += dots[w];
      }
      const float u = be * fmaf(-a, sk, vj);
      uu[tid] = u;
      st_val(o + row + c0 + tid, fmaf(qk, u, a * sq));
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float u = uu[NC * lane + c];
#pragma unroll
      for (int i = 0; i < NR; ++i) s[i][c] = fmaf(kk[warp + 8 * i], u, a * s[i][c]);
    }
    __syncthreads();  // kk, qq and the partial sums are rewritten by the next token
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
    __stcs(reinterpret_cast<float2 *>(base + (warp + 8 * i) * D), make_float2(s[i][0], s[i][1]));
}

template <int D, typename T>
cudaError_t decode_launch(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v, void *o,
                          float *state, cudaStream_t s) {
  TimedLaunch t(K_DELTA_DECODE, s);
  constexpr int CS = D == 128 ? 2 : 1;
  delta_decode_kernel<D, CS, T><<<dim3(p.B * p.H, CS), kDecThreads, 0, s>>>(p, g, (const T *)q, (const T *)k,
                                                                            (const T *)v, (T *)o, state);
  return cudaGetLastError();
}

template <int D, int MODE>
cudaError_t walk(const Problem &p, const DeltaGates &g, const WalkArgs &w, cudaStream_t s) {
  TimedLaunch t(K_DELTA_WALK, s);
  const int64_t walks = (int64_t)p.B * p.H * (MODE == W_WRITES || MODE == W_READS ? (p.T + 63) / 64 : 1);
  delta_walk<D, MODE><<<(unsigned)(walks * (D / kVecs)), kWalkThreads, 0, s>>>(p, g, w);
  return cudaGetLastError();
}

template <int D>
cudaError_t walk_fwd(const Problem &p, const DeltaGates &g, const float *q, const float *k, const float *v, float *o,
                     const float *init, float *fin, void *ckpt, cudaStream_t s) {
  WalkArgs w{};
  w.q = q;
  w.k = k;
  w.v = v;
  w.o = o;
  w.in = init;
  w.out = fin;
  w.y = static_cast<float *>(ckpt);
  w.states = ckpt ? w.y + (int64_t)p.B * p.H * p.T * D : nullptr;
  return walk<D, W_OUTPUTS>(p, g, w, s);
}

template <int D>
cudaError_t walk_bwd(const Problem &p, const DeltaGates &g, const float *q, const float *k, const float *dO,
                     const float *d_final, const void *ckpt, float *dq, float *dk, float *dv, void *dlg, void *dbeta,
                     float *dinit, void *ws, cudaStream_t s) {
  const int64_t tokens = (int64_t)p.B * p.H * p.T, chunks = (int64_t)p.B * p.H * ((p.T + 63) / 64), n = tokens * D;
  WalkArgs w{};
  w.q = q;
  w.k = k;
  w.dO = dO;
  w.dq = dq;
  w.dk = dk;
  w.dv = dv;
  w.y = static_cast<float *>(const_cast<void *>(ckpt));
  w.states = w.y + n;
  w.grads = static_cast<float *>(ws);
  w.dy = w.grads + chunks * D * D;
  w.dkw = w.dy + n;
  float *x0 = w.dkw + n, *x1 = x0 + n / 4;
  w.dbpart = x1 + n / 4;
  w.apart = w.dbpart + n / 4;
  float *gx = w.apart + chunks * (D / 4), *anchor = gx + tokens;
  w.in = d_final;
  w.out = dinit;
  cudaError_t e = walk<D, W_REVERSE>(p, g, w, s);
  w.xpart = x0;
  if (e == cudaSuccess) e = walk<D, W_WRITES>(p, g, w, s);
  w.xpart = x1;
  if (e == cudaSuccess) e = walk<D, W_READS>(p, g, w, s);
  if (e != cudaSuccess) return e;
  {
    TimedLaunch t(K_DELTA_WALK, s);
    delta_walk_sums<<<(unsigned)((tokens + chunks + 255) / 256), 256, 0, s>>>(
        tokens, chunks, D / 4, x0, x1, w.dbpart, w.apart, gx, dbeta, g.f32, anchor);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return dlg ? delta_gate_sums(p, gx, anchor, dlg, g.f32, s) : cudaSuccess;
}

}  // namespace

cudaError_t delta_gate_sums(const Problem &p, const float *gx, const float *anchor, void *dlg, int f32,
                            cudaStream_t s) {
  TimedLaunch t(K_DELTA_GATE, s);
  const int64_t BH = (int64_t)p.B * p.H;
  const int N = (p.T + 63) / 64;
  delta_gate_grad<<<(unsigned)((BH * N + 7) / 8), 256, 0, s>>>(BH, p.T, N, gx, anchor, dlg, f32);
  return cudaGetLastError();
}

size_t delta_walk_ckpt_bytes(const Problem &p) {
  const size_t BH = (size_t)p.B * p.H, N = (p.T + 63) / 64;
  return p.T == 0 ? 0 : align256(4 * (BH * p.T * p.d + BH * (N + 1) * p.d * p.d));
}
size_t delta_walk_bwd_ws_bytes(const Problem &p) {
  const size_t BH = (size_t)p.B * p.H, N = (p.T + 63) / 64;
  return p.T == 0 ? 0 : align256(4 * (BH * p.T * (2 * p.d + 3 * p.d / 4 + 1) + BH * N * (p.d * p.d + p.d / 4 + 1)));
}

cudaError_t delta_walk_fwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v,
                           void *o, const float *init, float *fin, void *ckpt, cudaStream_t s) {
  auto run = p.d == 64 ? walk_fwd<64> : walk_fwd<128>;
  return run(p, g, static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v),
             static_cast<float *>(o), init, fin, ckpt, s);
}
cudaError_t delta_walk_bwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *dO,
                           const float *d_final, const void *ckpt, void *dq, void *dk, void *dv, void *dlg,
                           void *dbeta, float *dinit, void *ws, cudaStream_t s) {
  auto run = p.d == 64 ? walk_bwd<64> : walk_bwd<128>;
  return run(p, g, static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(dO),
             d_final, ckpt, static_cast<float *>(dq), static_cast<float *>(dk), static_cast<float *>(dv), dlg, dbeta,
             dinit, ws, s);
}
cudaError_t delta_decode(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v, void *o,
                         float *state, cudaStream_t s) {
  if (p.d == 64)
    return p.dtype == 1 ? decode_launch<64, float>(p, g, q, k, v, o, state, s)
                        : decode_launch<64, __nv_bfloat16>(p, g, q, k, v, o, state, s);
  return p.dtype == 1 ? decode_launch<128, float>(p, g, q, k, v, o, state, s)
                      : decode_launch<128, __nv_bfloat16>(p, g, q, k, v, o, state, s);
}

}  // namespace linattn
