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
// One CTA of 512 threads walks one (batch, head); the whole d x d matrix stays in registers
// (warp w rows w D/16 .., lane l columns l D/32 ..), so a token costs three block barriers and no
// memory traffic besides its own rows.  Forward, then for the backward one reverse walk of R and
// one forward walk of S: bound by the latency of those barriers, about 1 us a token, and by
// having only B * H CTAs -- the path for fp32 checks, as the library's other fp32 walks are.
#include <cuda_bf16.h>

#include "internal.h"

namespace linattn {
namespace {

constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;

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

// A thread's part of the matrix: D/16 rows of its warp, D/32 columns of its lane.
template <int D>
struct Tile {
  static constexpr int NR = D / kWalkWarps, NC = D / 32;
  float s[NR][NC];
  __device__ void load(const float *m, int warp, int lane) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) s[i][c] = m ? m[(warp * NR + i) * D + lane * NC + c] : 0.f;
  }
  __device__ void store(float *m, int warp, int lane) const {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) m[(warp * NR + i) * D + lane * NC + c] = s[i][c];
  }
  // part[warp][j] = sum over the warp's rows of s[.][j] x[row]
  __device__ void col_sums(const float *x, float (*part)[D], int warp, int lane) const {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < NR; ++i) a = fmaf(s[i][c], x[warp * NR + i], a);
      part[warp][lane * NC + c] = a;
    }
  }
  // out[row] = sum over all columns of s[row][.] x[.]: the warp's NR rows are halved over the
  // lanes, then the remaining lane bits are summed
  __device__ void row_sums(const float *x, float *out, int warp, int lane) const {
    float a[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      a[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) a[i] = fmaf(s[i][c], x[lane * NC + c], a[i]);
    }
    int row = 0, off = 16;
#pragma unroll
    for (int n = NR / 2; n >= 1; n /= 2, off /= 2) {
      const bool up = lane & off;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? a[i] : a[i + n], keep = up ? a[i + n] : a[i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
      row += up ? n : 0;
    }
    for (; off >= 1; off /= 2) a[0] += __shfl_xor_sync(0xffffffffu, a[0], off);
    if (lane % (32 / NR) == 0) out[warp * NR + row] = a[0];
  }
  // s = f s + x y^T
  __device__ void update(float f, const float *x, const float *y, int warp, int lane) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) s[i][c] = fmaf(x[warp * NR + i], y[lane * NC + c], f * s[i][c]);
  }
};

template <int D>
__device__ __forceinline__ float sum_parts(const float (*part)[D], int j) {
  float a = 0.f;
#pragma unroll
  for (int w = 0; w < kWalkWarps; ++w) a += part[w][j];
  return a;
}

// Block-wide sum of one value per thread of the first D threads; valid in thread 0.
template <int D>
__device__ __forceinline__ float sum_rows(float x, float *buf, int tid) {
#pragma unroll
  for (int o = 16; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (tid < D && tid % 32 == 0) buf[tid / 32] = x;
  __syncthreads();
  float r = 0.f;
  if (tid == 0)
    for (int i = 0; i < D / 32; ++i) r += buf[i];
  return r;
}

// y [BH][T][D] fp32 and states [BH][N + 1][D][D] (the state entering every chunk of 64 tokens,
// then the final one) are kept for the backward when not null.
template <int D, typename T>
__global__ void __launch_bounds__(kWalkThreads) delta_fwd_walk(Problem p, DeltaGates g, const T *q, const T *k,
                                                               const T *v, T *o, const float *init, float *fin,
                                                               float *ykeep, float *states) {
  __shared__ float kk[D], qq[D], uu[D], part[kWalkWarps][D];
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t base = (int64_t)b * p.sb + (int64_t)h * p.sh, gb = (int64_t)bh * p.T;
  const int N = (p.T + 63) / 64;
  Tile<D> S;
  S.load(init ? init + (int64_t)bh * D * D : nullptr, warp, lane);
  for (int t = 0; t < p.T; ++t) {
    if (states && t % 64 == 0) S.store(states + ((int64_t)bh * (N + 1) + t / 64) * D * D, warp, lane);
    const int64_t row = base + (int64_t)t * p.st;
    const float a = g.lg ? expf(ld_gate(g.lg, gb + t, g.f32)) : 1.f, be = ld_gate(g.beta, gb + t, g.f32);
    float vj = 0.f;
    if (tid < D) {
      kk[tid] = ld_val(k + row + tid);
      qq[tid] = ld_val(q + row + tid);
      vj = ld_val(v + row + tid);
    }
    __syncthreads();
    S.col_sums(kk, part, warp, lane);
    __syncthreads();
    if (tid < D) {
      const float y = fmaf(-a, sum_parts<D>(part, tid), vj);
      uu[tid] = be * y;
      if (ykeep) ykeep[(gb + t) * D + tid] = y;
    }
    __syncthreads();
    S.update(a, kk, uu, warp, lane);
    S.col_sums(qq, part, warp, lane);
    __syncthreads();
    if (tid < D) st_val(o + row + tid, sum_parts<D>(part, tid));
    // the next token rewrites kk, qq (read before the barrier above) and, after two more
    // barriers, part and uu
  }
  if (fin) S.store(fin + (int64_t)bh * D * D, warp, lane);
  if (states) S.store(states + ((int64_t)bh * (N + 1) + N) * D * D, warp, lane);
}

// The reverse walk of R: dv, db, the write part of dk (fp32, dkw), dy (fp32) and the anchors
// <R, S> at the chunks' ends.
template <int D, typename T>
__global__ void __launch_bounds__(kWalkThreads)
    delta_rev_walk(Problem p, DeltaGates g, const T *q, const T *k, const T *dO, const float *ykeep,
                   const float *states, const float *d_final, T *dv, void *dbeta, float *dkw, float *dyk,
                   float *anchor, float *dinit) {
  __shared__ float kk[D], qq[D], oo[D], uu[D], part[kWalkWarps][D], rowv[D], buf[kWalkWarps];
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t base = (int64_t)b * p.sb + (int64_t)h * p.sh, gb = (int64_t)bh * p.T;
  const int N = (p.T + 63) / 64;
  Tile<D> R;
  R.load(d_final ? d_final + (int64_t)bh * D * D : nullptr, warp, lane);
  for (int t = p.T - 1; t >= 0; --t) {
    if (t == p.T - 1 || t % 64 == 63) {
      const float *S = states + ((int64_t)bh * (N + 1) + t / 64 + 1) * D * D;
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < Tile<D>::NR; ++i)
#pragma unroll
        for (int c = 0; c < Tile<D>::NC; ++c)
          x = fmaf(R.s[i][c], S[(warp * Tile<D>::NR + i) * D + lane * Tile<D>::NC + c], x);
#pragma unroll
      for (int o = 16; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) buf[warp] = x;
      __syncthreads();
      if (tid == 0) {
        float r = 0.f;
        for (int i = 0; i < kWalkWarps; ++i) r += buf[i];
        anchor[(int64_t)bh * N + t / 64] = r;
      }
      __syncthreads();
    }
    const int64_t row = base + (int64_t)t * p.st;
    const float a = g.lg ? expf(ld_gate(g.lg, gb + t, g.f32)) : 1.f, be = ld_gate(g.beta, gb + t, g.f32);
    float y = 0.f;
    if (tid < D) {
      kk[tid] = ld_val(k + row + tid);
      qq[tid] = ld_val(q + row + tid);
      oo[tid] = ld_val(dO + row + tid);
      y = ykeep[(gb + t) * D + tid];
      uu[tid] = be * y;
    }
    __syncthreads();
    R.update(1.f, qq, oo, warp, lane);
    R.col_sums(kk, part, warp, lane);
    R.row_sums(uu, rowv, warp, lane);
    __syncthreads();
    float db = 0.f;
    if (tid < D) {
      const float du = sum_parts<D>(part, tid), dy = be * du;
      db = du * y;
      oo[tid] = -dy;
      st_val(dv + row + tid, dy);
      dyk[(gb + t) * D + tid] = dy;
      dkw[(gb + t) * D + tid] = rowv[tid];
    }
    db = sum_rows<D>(db, buf, tid);  // (a barrier inside: oo is complete after it)
    if (tid == 0) st_gate(dbeta, gb + t, g.f32, db);
    R.update(1.f, kk, oo, warp, lane);
#pragma unroll
    for (int i = 0; i < Tile<D>::NR; ++i)
#pragma unroll
      for (int c = 0; c < Tile<D>::NC; ++c) R.s[i][c] *= a;
    __syncthreads();
  }
  if (dinit) R.store(dinit + (int64_t)bh * D * D, warp, lane);
}

// The forward walk of S in the backward: dq, dk and G of every token (gx [BH][T] fp32).
template <int D, typename T>
__global__ void __launch_bounds__(kWalkThreads)
    delta_grad_walk(Problem p, DeltaGates g, const T *q, const T *k, const T *dO, const float *ykeep,
                    const float *dyk, const float *dkw, const float *init, T *dq, T *dk, float *gx) {
  __shared__ float kk[D], oo[D], uu[D], yy[D], r1[D], r2[D], buf[kWalkWarps];
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t base = (int64_t)b * p.sb + (int64_t)h * p.sh, gb = (int64_t)bh * p.T;
  Tile<D> S;
  S.load(init ? init + (int64_t)bh * D * D : nullptr, warp, lane);
  for (int t = 0; t < p.T; ++t) {
    const int64_t row = base + (int64_t)t * p.st;
    const float a = g.lg ? expf(ld_gate(g.lg, gb + t, g.f32)) : 1.f, be = ld_gate(g.beta, gb + t, g.f32);
    float qv = 0.f, kv = 0.f, w = 0.f;
    if (tid < D) {
      kk[tid] = kv = ld_val(k + row + tid);
      qv = ld_val(q + row + tid);
      oo[tid] = ld_val(dO + row + tid);
      uu[tid] = be * ykeep[(gb + t) * D + tid];
      yy[tid] = dyk[(gb + t) * D + tid];
      w = dkw[(gb + t) * D + tid];
    }
    __syncthreads();
    S.row_sums(yy, r1, warp, lane);
    S.update(a, kk, uu, warp, lane);
    S.row_sums(oo, r2, warp, lane);
    __syncthreads();
    float x = 0.f;
    if (tid < D) {
      const float read = -a * r1[tid];
      st_val(dq + row + tid, r2[tid]);
      st_val(dk + row + tid, read + w);
      x = fmaf(qv, r2[tid], kv * (read - w));
    }
    x = sum_rows<D>(x, buf, tid);
    if (tid == 0) gx[gb + t] = x;
    __syncthreads();
  }
}

// d_log_gate: the sums of G from every token to its chunk's end, plus the chunk's anchor.
// One warp per chunk of 64 tokens.
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
// so a token takes one reduction across the warps.  Bound by the state's read and write
// (2 x 64 KiB per head at d = 128).
constexpr int kDecThreads = 256;

template <int D, int CS, typename T>
__global__ void __launch_bounds__(kDecThreads) delta_decode_kernel(Problem p, DeltaGates g, const T *q, const T *k,
                                                                   const T *v, T *o, float *state) {
  constexpr int W = D / CS, NC = W / 32, NR = D / 8;
  __shared__ float kk[D], qq[D], pk[8][W], pq[8][W], uu[W], dots[8];
  const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * W;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t off = (int64_t)b * p.sb + (int64_t)h * p.sh, gb = (int64_t)bh * p.T;
  float *base = state + (int64_t)bh * D * D + c0 + NC * lane;
  float s[NR][NC];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) s[i][c] = base[(warp + 8 * i) * D + c];
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
#pragma unroll
    for (int c = 0; c < NC; ++c) base[(warp + 8 * i) * D + c] = s[i][c];
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

template <int D, typename T>
cudaError_t fwd_launch(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v, void *o,
                       const float *init, float *fin, void *ckpt, cudaStream_t s) {
  TimedLaunch t(K_DELTA_WALK, s);
  float *y = static_cast<float *>(ckpt);
  float *states = ckpt ? y + (int64_t)p.B * p.H * p.T * D : nullptr;
  delta_fwd_walk<D, T><<<p.B * p.H, kWalkThreads, 0, s>>>(p, g, (const T *)q, (const T *)k, (const T *)v, (T *)o,
                                                          init, fin, y, states);
  return cudaGetLastError();
}

template <int D, typename T>
cudaError_t bwd_launch(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *dO,
                       const float *init, const float *d_final, const void *ckpt, void *dq, void *dk, void *dv,
                       void *dlg, void *dbeta, float *dinit, void *ws, cudaStream_t s) {
  const int64_t BH = (int64_t)p.B * p.H, n = BH * p.T * D;
  const int N = (p.T + 63) / 64;
  const float *y = static_cast<const float *>(ckpt), *states = y + n;
  float *dyk = static_cast<float *>(ws), *dkw = dyk + n, *gx = dkw + n, *anchor = gx + BH * p.T;
  {
    TimedLaunch t(K_DELTA_WALK, s);
    delta_rev_walk<D, T><<<(int)BH, kWalkThreads, 0, s>>>(p, g, (const T *)q, (const T *)k, (const T *)dO, y, states,
                                                          d_final, (T *)dv, dbeta, dkw, dyk, anchor, dinit);
  }
  {
    TimedLaunch t(K_DELTA_WALK, s);
    delta_grad_walk<D, T><<<(int)BH, kWalkThreads, 0, s>>>(p, g, (const T *)q, (const T *)k, (const T *)dO, y, dyk,
                                                           dkw, init, (T *)dq, (T *)dk, gx);
  }
  if (dlg) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return delta_gate_sums(p, gx, anchor, dlg, g.f32, s);
  }
  return cudaGetLastError();
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
  return p.T == 0 ? 0 : align256(4 * (BH * p.T * (2 * p.d + 1) + BH * N));
}

cudaError_t delta_walk_fwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *v,
                           void *o, const float *init, float *fin, void *ckpt, cudaStream_t s) {
  return p.d == 64 ? fwd_launch<64, float>(p, g, q, k, v, o, init, fin, ckpt, s)
                   : fwd_launch<128, float>(p, g, q, k, v, o, init, fin, ckpt, s);
}
cudaError_t delta_walk_bwd(const Problem &p, const DeltaGates &g, const void *q, const void *k, const void *dO,
                           const float *init, const float *d_final, const void *ckpt, void *dq, void *dk, void *dv,
                           void *dlg, void *dbeta, float *dinit, void *ws, cudaStream_t s) {
  return p.d == 64
             ? bwd_launch<64, float>(p, g, q, k, dO, init, d_final, ckpt, dq, dk, dv, dlg, dbeta, dinit, ws, s)
             : bwd_launch<128, float>(p, g, q, k, dO, init, d_final, ckpt, dq, dk, dv, dlg, dbeta, dinit, ws, s);
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
