// Gated linear recurrence (ssm_glr_* of ssm_hybrid.h) for gfx950.
//
//   r = sigmoid(gr), i = sigmoid(gi), la = A r, a = e^la, s = sqrt(max(0, 1 - e^(2 la)))
//   h_t = a_t h_{t-1} + s_t i_t x_t,   y_t = h_t
//
// A thread owns VEC neighbouring channels of one chunk of steps. A chunk's
// effect on the state is the affine map h -> P h + H; a first kernel forms
// (P, H) of every chunk, a second folds them along the sequence into the
// state entering each chunk, the third runs every chunk from that state.
// The backward does the same with the adjoint, in reverse time.
#include "hybrid_common.h"

namespace {

constexpr int kCk = SSM_GLR_CKPT_STEPS;

// ---------------------------------------------------------------------------
// VEC-wide element access
// ---------------------------------------------------------------------------
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 f = Vec4<T>::load(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
    v[0] = to_f32(p[0]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    Vec4<T>::store(p, make_float4(v[0], v[1], v[2], v[3]));
  } else {
    p[0] = from_f32<T>(v[0]);
  }
}

// ---------------------------------------------------------------------------
// the gates of one element
// ---------------------------------------------------------------------------
// 1 / (1 + e^-v) from the hardware exponential and reciprocal. The rounding
// of the exponent's argument is |v| 2^-24 relative; e^-v = inf gives 0.
__device__ __forceinline__ float sigmoid_fast(float v) {
  return rcp_fast(1.f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

struct Gates {
  float r, i, a, s;
};

// A2 = A log2(e). 1 - e^z, z = 2 la: the series in z for z > -1/4 (relative
// error below z^6 / 5040 = 5e-8; the difference from 1 would lose the leading
// digits there), else 1 - a^2 (relative error at most 2^-24 (1 / 0.22)).
__device__ __forceinline__ Gates gates(float gr, float gi, float A2) {
  Gates g;
  g.r = sigmoid_fast(gr);
  g.i = sigmoid_fast(gi);
  const float la2 = A2 * g.r;
  g.a = __builtin_amdgcn_exp2f(la2);
  const float z = la2 * (2.f / kLog2e);
  float q = __builtin_fmaf(z, 1.f / 720.f, 1.f / 120.f);
  q = __builtin_fmaf(z, q, 1.f / 24.f);
  q = __builtin_fmaf(z, q, 1.f / 6.f);
  q = __builtin_fmaf(z, q, 0.5f);
  q = __builtin_fmaf(z, q, 1.f);
  const float near = -z * q, far = __builtin_fmaf(-g.a, g.a, 1.f);
  const float v = z > -0.25f ? near : far;
  // (a NaN stays one: the comparison is false for it)
  g.s = v <= 0.f ? 0.f : __builtin_amdgcn_sqrtf(v);
  return g;
}

template <typename T>
struct GlrArgs {
  const T* x;
  const T* gr;
  const T* gi;
  const float* A;
  const float* h0;
  T* y;
  float* h_last;
  float* ckpt;
  const T* dy;
  const float* dh_last;
  T* dx;
  T* dgr;
  T* dgi;
  float* dh0;
  float2* agg;     // (Bs, nchunks, ED): (P, H) of each chunk
  float* enter;    // (Bs, nchunks, ED): the state (backward: the adjoint) entering each chunk
  float* dA_part;  // (Bs, nchunks, ED)
  int64_t Bs, L, ED, ncg, nchunks, steps, ckrows;
};

// The chunk and channels of this thread; false past the end.
template <typename T, int VEC>
__device__ __forceinline__ bool place(const GlrArgs<T>& p, int64_t* b, int64_t* k, int64_t* e) {
  const int64_t item = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (item >= p.Bs * p.nchunks * p.ncg) return false;
  *e = (item % p.ncg) * VEC;
  *k = (item / p.ncg) % p.nchunks;
  *b = item / p.ncg / p.nchunks;
  return true;
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_agg_kernel(const GlrArgs<T> p) {
  int64_t b, k, e;
  if (!place<T, VEC>(p, &b, &k, &e)) return;
  const int64_t t0 = k * p.steps, n = p.L - t0 < p.steps ? p.L - t0 : p.steps;
  int64_t at = (b * p.L + t0) * p.ED + e;
  float A2[VEC], P[VEC], H[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) A2[c] = p.A[e + c] * kLog2e, P[c] = 1.f, H[c] = 0.f;
#pragma unroll 4
  for (int64_t t = 0; t < n; ++t, at += p.ED) {
    float x[VEC], gr[VEC], gi[VEC];
    load_vec<T, VEC>(p.x + at, x);
    load_vec<T, VEC>(p.gr + at, gr);
    load_vec<T, VEC>(p.gi + at, gi);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const Gates g = gates(gr[c], gi[c], A2[c]);
      P[c] *= g.a;
      H[c] = __builtin_fmaf(g.a, H[c], g.s * g.i * x[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) p.agg[(b * p.nchunks + k) * p.ED + e + c] = make_float2(P[c], H[c]);
}

// enter[k] = fold of the chunks before k (rev: after k) from `init`.
__global__ __launch_bounds__(64) void glr_join_kernel(const float2* agg, const float* init, float* enter, int64_t n,
                                                      int64_t nchunks, int64_t ED, int rev) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  const int64_t b = i / ED, e = i % ED;
  float h = init ? init[i] : 0.f;
#pragma unroll 8
  for (int64_t j = 0; j < nchunks; ++j) {
    const int64_t k = rev ? nchunks - 1 - j : j;
    const int64_t o = (b * nchunks + k) * ED + e;
    const float2 m = agg[o];
    enter[o] = h;
    h = __builtin_fmaf(m.x, h, m.y);
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_apply_kernel(const GlrArgs<T> p) {
  int64_t b, k, e;
  if (!place<T, VEC>(p, &b, &k, &e)) return;
  const int64_t t0 = k * p.steps, n = p.L - t0 < p.steps ? p.L - t0 : p.steps;
  int64_t at = (b * p.L + t0) * p.ED + e;
  float A2[VEC], h[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    A2[c] = p.A[e + c] * kLog2e;
    h[c] = p.enter ? p.enter[(b * p.nchunks + k) * p.ED + e + c] : p.h0 ? p.h0[b * p.ED + e + c] : 0.f;
  }
#pragma unroll 4
  for (int64_t t = 0; t < n; ++t, at += p.ED) {
    if (p.ckpt && (t0 + t) % kCk == 0) store_vec<float, VEC>(p.ckpt + (b * p.ckrows + (t0 + t) / kCk) * p.ED + e, h);
    float x[VEC], gr[VEC], gi[VEC];
    load_vec<T, VEC>(p.x + at, x);
    load_vec<T, VEC>(p.gr + at, gr);
    load_vec<T, VEC>(p.gi + at, gi);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const Gates g = gates(gr[c], gi[c], A2[c]);
      h[c] = __builtin_fmaf(g.a, h[c], g.s * g.i * x[c]);
    }
    store_vec<T, VEC>(p.y + at, h);
  }
  if (p.h_last && k == p.nchunks - 1) store_vec<float, VEC>(p.h_last + b * p.ED + e, h);
}

// The adjoint's aggregate of a chunk: G -> P G + H with G entering after the
// chunk's last step and leaving before its first (a_t applied).
template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_bwd_agg_kernel(const GlrArgs<T> p) {
  int64_t b, k, e;
  if (!place<T, VEC>(p, &b, &k, &e)) return;
  const int64_t t0 = k * p.steps, n = p.L - t0 < p.steps ? p.L - t0 : p.steps;
  int64_t at = (b * p.L + t0 + n - 1) * p.ED + e;
  float A2[VEC], P[VEC], H[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) A2[c] = p.A[e + c] * kLog2e, P[c] = 1.f, H[c] = 0.f;
#pragma unroll 4
  for (int64_t t = 0; t < n; ++t, at -= p.ED) {
    float gr[VEC], dy[VEC];
    load_vec<T, VEC>(p.gr + at, gr);
    load_vec<T, VEC>(p.dy + at, dy);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const float a = __builtin_amdgcn_exp2f(A2[c] * sigmoid_fast(gr[c]));
      P[c] *= a;
      H[c] = a * (H[c] + dy[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) p.agg[(b * p.nchunks + k) * p.ED + e + c] = make_float2(P[c], H[c]);
}

// Blocks of kCk steps in reverse order: the states of the block again from
// its checkpoint, then its adjoint steps backwards.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_bwd_apply_kernel(const GlrArgs<T> p) {
  int64_t b, k, e;
  if (!place<T, VEC>(p, &b, &k, &e)) return;
  const int64_t t0 = k * p.steps, n = p.L - t0 < p.steps ? p.L - t0 : p.steps;
  float A[VEC], A2[VEC], G[VEC], dA[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    A[c] = p.A[e + c];
    A2[c] = A[c] * kLog2e;
    dA[c] = 0.f;
    G[c] = p.enter[(b * p.nchunks + k) * p.ED + e + c];
  }
  for (int64_t blk = (n + kCk - 1) / kCk - 1; blk >= 0; --blk) {
    const int64_t tb = t0 + blk * kCk;
    const int m = static_cast<int>(t0 + n - tb < kCk ? t0 + n - tb : kCk);
    const int64_t at = (b * p.L + tb) * p.ED + e;
    float hp[kCk][VEC], h[VEC];  // h_{t-1} of the block's steps
    load_vec<float, VEC>(p.ckpt + (b * p.ckrows + tb / kCk) * p.ED + e, h);
#pragma unroll
    for (int t = 0; t < kCk; ++t) {
      if (t < m) {
        float x[VEC], gr[VEC], gi[VEC];
        load_vec<T, VEC>(p.x + at + t * p.ED, x);
        load_vec<T, VEC>(p.gr + at + t * p.ED, gr);
        load_vec<T, VEC>(p.gi + at + t * p.ED, gi);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const Gates g = gates(gr[c], gi[c], A2[c]);
          hp[t][c] = h[c];
          h[c] = __builtin_fmaf(g.a, h[c], g.s * g.i * x[c]);
        }
      }
    }
#pragma unroll
    for (int t = kCk - 1; t >= 0; --t) {
      if (t < m) {
        const int64_t o = at + t * p.ED;
        float x[VEC], gr[VEC], gi[VEC], dy[VEC], dx[VEC], dgr[VEC], dgi[VEC];
        load_vec<T, VEC>(p.x + o, x);
        load_vec<T, VEC>(p.gr + o, gr);
        load_vec<T, VEC>(p.gi + o, gi);
        load_vec<T, VEC>(p.dy + o, dy);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const Gates q = gates(gr[c], gi[c], A2[c]);
          const float g = G[c] + dy[c];
          const float ix = q.i * x[c], gs = g * q.s;
          const float root = q.s > 0.f ? q.a * q.a * rcp_fast(q.s) * ix : 0.f;
          const float dlr = g * (q.a * hp[t][c] - root) * q.r;  // dla r
          dx[c] = gs * q.i;
          dgi[c] = gs * ix * (1.f - q.i);
          dgr[c] = dlr * A[c] * (1.f - q.r);
          dA[c] += dlr;
          G[c] = q.a * g;
        }
        store_vec<T, VEC>(p.dx + o, dx);
        store_vec<T, VEC>(p.dgr + o, dgr);
        store_vec<T, VEC>(p.dgi + o, dgi);
      }
    }
  }
  if (p.dh0 && k == 0) store_vec<float, VEC>(p.dh0 + b * p.ED + e, G);
#pragma unroll
  for (int c = 0; c < VEC; ++c) p.dA_part[(b * p.nchunks + k) * p.ED + e + c] = dA[c];
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_step_kernel(const T* x, const T* gr, const T* gi, const float* A,
                                                       const float* h, T* y, float* h_out, int64_t Bs, int64_t ED) {
  const int64_t item = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  const int64_t ncg = ED / VEC;
  if (item >= Bs * ncg) return;
  const int64_t e = (item % ncg) * VEC, at = item * VEC;
  float xv[VEC], rv[VEC], iv[VEC], hv[VEC];
  load_vec<T, VEC>(x + at, xv);
  load_vec<T, VEC>(gr + at, rv);
  load_vec<T, VEC>(gi + at, iv);
  load_vec<float, VEC>(h + at, hv);
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const Gates g = gates(rv[c], iv[c], A[e + c] * kLog2e);
    hv[c] = __builtin_fmaf(g.a, hv[c], g.s * g.i * xv[c]);
  }
  store_vec<float, VEC>(h_out + at, hv);
  store_vec<T, VEC>(y + at, hv);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct GlrPlan {
  int64_t nchunks, steps, ckrows;
};

// Chunks are whole blocks of kCk steps, as long as there are at least about
// four waves of threads per CU (256 CUs), at most 128 steps.
GlrPlan glr_plan(int64_t Bs, int64_t L, int64_t ED) {
  const int64_t lanes = Bs * (ED % 4 == 0 ? ED / 4 : ED);
  int64_t steps = 128;
  while (steps > kCk && lanes * ((L + steps - 1) / steps) < 4 * 64 * 256) steps /= 2;
  return GlrPlan{(L + steps - 1) / steps, steps, (L + kCk - 1) / kCk};
}

int glr_sizes(int64_t Bs, int64_t L, int64_t ED, int dtype, int64_t* n, int64_t* nck) {
  int64_t c, rows = L >= 0 ? (L + kCk - 1) / kCk : -1, bytes;
  if (!mul_nn(Bs, ED, &c) || !mul_nn(c, L, n) || !mul_nn(*n, 4, &bytes)) return SSM_ERR_DIM;
  if (!mul_nn(c, rows, nck) || !mul_nn(*nck, 16, &bytes)) return SSM_ERR_DIM;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t glr_agg_bytes(const GlrPlan& pl, int64_t c) { return static_cast<size_t>(pl.nchunks * c) * 8; }
size_t glr_enter_bytes(const GlrPlan& pl, int64_t c) { return (static_cast<size_t>(pl.nchunks * c) * 4 + 15) & ~size_t(15); }

template <typename T, int VEC>
int launch_fwd(GlrArgs<T> a, hipStream_t st) {
  const int64_t blocks = (a.Bs * a.nchunks * a.ncg + 255) / 256;
  if (blocks > kMaxGrid) return SSM_ERR_DIM;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.nchunks > 1) {
    hipLaunchKernelGGL((glr_agg_kernel<T, VEC>), grid, dim3(256), 0, st, a);
    const int64_t n = a.Bs * a.ED;
    hipLaunchKernelGGL(glr_join_kernel, dim3(static_cast<unsigned>((n + 63) / 64)), dim3(64), 0, st, a.agg, a.h0,
                       a.enter, n, a.nchunks, a.ED, 0);
  }
  hipLaunchKernelGGL((glr_apply_kernel<T, VEC>), grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

template <typename T, int VEC>
int launch_bwd(GlrArgs<T> a, float* dA, hipStream_t st) {
  const int64_t blocks = (a.Bs * a.nchunks * a.ncg + 255) / 256;
  if (blocks > kMaxGrid) return SSM_ERR_DIM;
  const dim3 grid(static_cast<unsigned>(blocks));
  const int64_t n = a.Bs * a.ED;
  hipLaunchKernelGGL((glr_bwd_agg_kernel<T, VEC>), grid, dim3(256), 0, st, a);
  hipLaunchKernelGGL(glr_join_kernel, dim3(static_cast<unsigned>((n + 63) / 64)), dim3(64), 0, st, a.agg, a.dh_last,
                     a.enter, n, a.nchunks, a.ED, 1);
  hipLaunchKernelGGL((glr_bwd_apply_kernel<T, VEC>), grid, dim3(256), 0, st, a);
  hipLaunchKernelGGL(sum_rows_kernel, dim3(static_cast<unsigned>((a.ED + 15) / 16)), dim3(256), 0, st, a.dA_part, dA,
                     a.Bs * a.nchunks, a.ED);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

template <typename T>
int run_fwd(const void* x, const void* gr, const void* gi, const float* A, const float* h0, void* y, float* h_last,
            float* ckpt, int64_t Bs, int64_t L, int64_t ED, void* ws, hipStream_t st) {
  const GlrPlan pl = glr_plan(Bs, L, ED);
  GlrArgs<T> a{};
  a.x = static_cast<const T*>(x), a.gr = static_cast<const T*>(gr), a.gi = static_cast<const T*>(gi);
  a.A = A, a.h0 = h0, a.y = static_cast<T*>(y), a.h_last = h_last, a.ckpt = ckpt;
  a.Bs = Bs, a.L = L, a.ED = ED, a.nchunks = pl.nchunks, a.steps = pl.steps, a.ckrows = pl.ckrows;
  if (pl.nchunks > 1) {
    a.agg = static_cast<float2*>(ws);
    a.enter = reinterpret_cast<float*>(static_cast<char*>(ws) + glr_agg_bytes(pl, Bs * ED));
  }
  if (ED % 4 == 0) {
    a.ncg = ED / 4;
    return launch_fwd<T, 4>(a, st);
  }
  a.ncg = ED;
  return launch_fwd<T, 1>(a, st);
}

template <typename T>
int run_bwd(const void* x, const void* gr, const void* gi, const float* A, const float* ckpt, const void* dy,
            const float* dh_last, void* dx, void* dgr, void* dgi, float* dA, float* dh0, int64_t Bs, int64_t L,
            int64_t ED, void* ws, hipStream_t st) {
  const GlrPlan pl = glr_plan(Bs, L, ED);
  GlrArgs<T> a{};
  a.x = static_cast<const T*>(x), a.gr = static_cast<const T*>(gr), a.gi = static_cast<const T*>(gi);
  a.A = A, a.ckpt = const_cast<float*>(ckpt), a.dy = static_cast<const T*>(dy), a.dh_last = dh_last;
  a.dx = static_cast<T*>(dx), a.dgr = static_cast<T*>(dgr), a.dgi = static_cast<T*>(dgi), a.dh0 = dh0;
  a.Bs = Bs, a.L = L, a.ED = ED, a.nchunks = pl.nchunks, a.steps = pl.steps, a.ckrows = pl.ckrows;
  char* w = static_cast<char*>(ws);
  a.agg = reinterpret_cast<float2*>(w);
  a.enter = reinterpret_cast<float*>(w + glr_agg_bytes(pl, Bs * ED));
  a.dA_part = reinterpret_cast<float*>(w + glr_agg_bytes(pl, Bs * ED) + glr_enter_bytes(pl, Bs * ED));
  if (ED % 4 == 0) {
    a.ncg = ED / 4;
    return launch_bwd<T, 4>(a, dA, st);
  }
  a.ncg = ED;
  return launch_bwd<T, 1>(a, dA, st);
}

}  // namespace

extern "C" size_t ssm_glr_ckpt_bytes(int64_t Bs, int64_t L, int64_t ED) {
  int64_t n, nck;
  if (glr_sizes(Bs, L, ED, SSM_F32, &n, &nck) != SSM_OK) return 0;
  return static_cast<size_t>(nck) * 4;
}

extern "C" size_t ssm_glr_workspace_bytes(int64_t Bs, int64_t L, int64_t ED, int dtype) {
  int64_t n, nck;
  if (glr_sizes(Bs, L, ED, dtype, &n, &nck) != SSM_OK || n == 0) return 0;
  const GlrPlan pl = glr_plan(Bs, L, ED);
  return pl.nchunks > 1 ? glr_agg_bytes(pl, Bs * ED) + glr_enter_bytes(pl, Bs * ED) : 0;
}

extern "C" size_t ssm_glr_bwd_workspace_bytes(int64_t Bs, int64_t L, int64_t ED, int dtype) {
  int64_t n, nck;
  if (glr_sizes(Bs, L, ED, dtype, &n, &nck) != SSM_OK || n == 0) return 0;
  const GlrPlan pl = glr_plan(Bs, L, ED);
  return glr_agg_bytes(pl, Bs * ED) + 2 * glr_enter_bytes(pl, Bs * ED);
}

extern "C" int ssm_glr_fwd(const void* x, const void* gr, const void* gi, const float* A, const float* h0, void* y,
                           float* h_last, float* ckpt, int64_t Bs, int64_t L, int64_t ED, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int64_t n, nck;
  int rc = glr_sizes(Bs, L, ED, dtype, &n, &nck);
  if (rc != SSM_OK) return rc;
  const int64_t nb = n * (dtype == SSM_F32 ? 4 : 2), cb = Bs * ED * 4;
  const size_t need = ssm_glr_workspace_bytes(Bs, L, ED, dtype);
  const Buf bufs[] = {{x, nb, true, false},      {gr, nb, true, false},      {gi, nb, true, false},
                      {A, ED * 4, true, false},  {h0, cb, false, false},     {y, nb, true, true},
                      {h_last, cb, false, true}, {ckpt, nck * 4, false, true}, {workspace, static_cast<int64_t>(need), false, true}};
  rc = check_bufs(bufs, 9);
  if (rc != SSM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n == 0) return fill_async(h_last, h0, cb, st) ? SSM_OK : SSM_ERR_LAUNCH;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  return dtype == SSM_F32 ? run_fwd<float>(x, gr, gi, A, h0, y, h_last, ckpt, Bs, L, ED, workspace, st)
                          : run_fwd<uint16_t>(x, gr, gi, A, h0, y, h_last, ckpt, Bs, L, ED, workspace, st);
}

extern "C" int ssm_glr_bwd(const void* x, const void* gr, const void* gi, const float* A, const float* ckpt,
                           const void* dy, const float* dh_last, void* dx, void* dgr, void* dgi, float* dA,
                           float* dh0, int64_t Bs, int64_t L, int64_t ED, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int64_t n, nck;
  int rc = glr_sizes(Bs, L, ED, dtype, &n, &nck);
  if (rc != SSM_OK) return rc;
  const int64_t nb = n * (dtype == SSM_F32 ? 4 : 2), cb = Bs * ED * 4;
  const size_t need = ssm_glr_bwd_workspace_bytes(Bs, L, ED, dtype);
  const Buf bufs[] = {{x, nb, true, false},         {gr, nb, true, false},       {gi, nb, true, false},
                      {A, ED * 4, true, false},     {ckpt, nck * 4, true, false}, {dy, nb, true, false},
                      {dh_last, cb, false, false},  {dx, nb, true, true},        {dgr, nb, true, true},
                      {dgi, nb, true, true},        {dA, ED * 4, true, true},    {dh0, cb, false, true},
                      {workspace, static_cast<int64_t>(need), false, true}};
  rc = check_bufs(bufs, 13);
  if (rc != SSM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n == 0)
    return fill_async(dA, nullptr, ED * 4, st) && fill_async(dh0, dh_last, cb, st) ? SSM_OK : SSM_ERR_LAUNCH;
  if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
  return dtype == SSM_F32
             ? run_bwd<float>(x, gr, gi, A, ckpt, dy, dh_last, dx, dgr, dgi, dA, dh0, Bs, L, ED, workspace, st)
             : run_bwd<uint16_t>(x, gr, gi, A, ckpt, dy, dh_last, dx, dgr, dgi, dA, dh0, Bs, L, ED, workspace, st);
}

extern "C" int ssm_glr_step(const void* x, const void* gr, const void* gi, const float* A, const float* h, void* y,
                            float* h_out, int64_t Bs, int64_t ED, int dtype, void* stream) {
  int64_t n, nck;
  int rc = glr_sizes(Bs, 1, ED, dtype, &n, &nck);
  if (rc != SSM_OK) return rc;
  const int64_t nb = n * (dtype == SSM_F32 ? 4 : 2), cb = n * 4;
  // (h_out may be h itself: h is then left out of the overlap check)
  const Buf bufs[] = {{x, nb, true, false},     {gr, nb, true, false}, {gi, nb, true, false}, {A, ED * 4, true, false},
                      {h == h_out ? nullptr : h, cb, h != h_out, false}, {y, nb, true, true},  {h_out, cb, true, true}};
  rc = check_bufs(bufs, 7);
  if (rc != SSM_OK) return rc;
  if (n == 0) return SSM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t items = ED % 4 == 0 ? n / 4 : n, blocks = (items + 255) / 256;
  if (blocks > kMaxGrid) return SSM_ERR_DIM;
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
  const bool f32 = dtype == SSM_F32;
#define SSM_GLR_STEP(T, V)                                                                                         \
  hipLaunchKernelGGL((glr_step_kernel<T, V>), grid, block, 0, st, static_cast<const T*>(x), static_cast<const T*>(gr), \
                     static_cast<const T*>(gi), A, h, static_cast<T*>(y), h_out, Bs, ED)
  if (ED % 4 == 0) {
    if (f32) SSM_GLR_STEP(float, 4); else SSM_GLR_STEP(uint16_t, 4);
  } else {
    if (f32) SSM_GLR_STEP(float, 1); else SSM_GLR_STEP(uint16_t, 1);
  }
#undef SSM_GLR_STEP
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}
