// Norm and rotation of queries and keys (ssm_qk_rope_* of ssm_hybrid.h) for
// gfx950.
//
//   n = x w / sqrt(mean(x^2) + eps);  (n_j, n_{j+R/2}) turned by pos * freq_j
//
// A head is held by D entries / 16 bytes lanes, 16 bytes each, so that every
// access is a full 16-byte vector; the mean is a butterfly over those lanes
// and the partner of a pair comes from another lane of the same head. A
// workgroup takes a few tokens: it forms their angles once (64-bit reduction
// to a fraction of a turn, then float32) in LDS, for all heads of q and k.
#include "hybrid_common.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a workgroup
constexpr int kMaxBlocks = 1024;  // workgroups of the backward (rows of partial weight gradients)

template <typename T>
struct RopeArgs {
  const T* q;
  const T* k;
  const T* v;
  ssm_strides qs, ks, vs;
  const float* wq;
  const float* wk;
  const double* freq;
  const int32_t* pos;
  float eps;
  T* q_out;
  T* k_out;  // append: the key cache
  T* v_out;  // append: the value cache
  const T* dq_out;
  const T* dk_out;
  float* part;
  int64_t Bs, L;
  int Hq, Hk, half, tokens;  // half: R / 2; tokens: of a workgroup
  int window, sinks;
};

// cos and sin of pos * freq[j], j < half, for the workgroup's tokens. The
// angle in turns is a float64 product: its fraction is good to 2^-52 of the
// number of turns.
template <typename T, bool APPEND>
__device__ __forceinline__ void angles(const RopeArgs<T>& p, int64_t first, int n, float2* cs) {
  for (int i = threadIdx.x; i < n * p.half; i += kThreads) {
    const int t = i / p.half, j = i % p.half;
    const int64_t tok = first + t;
    double at;
    if (APPEND) {
      at = static_cast<double>(p.pos[tok / p.L]) + static_cast<double>(tok % p.L);
    } else {
      at = p.pos ? static_cast<double>(p.pos[tok]) : static_cast<double>(tok % p.L);
    }
    const double turns = at * (p.freq[j] * 0.15915494309189533577);
    const float f = static_cast<float>(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.f * f, &s, &c);
    cs[i] = make_float2(c, s);
  }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = 1; m < LPH; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <typename T, int D, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs<T> p) {
  constexpr int E = Vec16<T>::kN, LPH = D / E;
  extern __shared__ float2 cs[];
  const int64_t first = blockIdx.x * static_cast<int64_t>(p.tokens), all = p.Bs * p.L;
  const int n = static_cast<int>(all - first < p.tokens ? all - first : p.tokens);
  angles<T, APPEND>(p, first, n, cs);
  __syncthreads();
  const int li = threadIdx.x % LPH;
  const int H = p.Hq + p.Hk + (APPEND ? p.Hk : 0);
  const int lane = threadIdx.x & 63;
  float wq[E], wk[E];
#pragma unroll
  for (int c = 0; c < E; ++c) {
    wq[c] = p.wq ? p.wq[li * E + c] : 1.f;
    wk[c] = p.wk ? p.wk[li * E + c] : 1.f;
  }
  // where this lane's entries sit in the rotation
  const int j0 = li * E;
  const bool turned = j0 < 2 * p.half, upper = j0 >= p.half;
  const int partner = !turned ? lane : upper ? lane - p.half / E : lane + p.half / E;
  const int jc = upper ? j0 - p.half : j0;
  for (int item = threadIdx.x / LPH; item < n * H; item += kThreads / LPH) {
    const int t = item / H, h = item % H;
    const int64_t tok = first + t, b = tok / p.L, l = tok % p.L;
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hk;
    const int hh = is_q ? h : is_v ? h - p.Hq - p.Hk : h - p.Hq;
    const T* src = is_q ? p.q + b * p.qs.batch + l * p.qs.token + hh * p.qs.head
                 : is_v ? p.v + b * p.vs.batch + l * p.vs.token + hh * p.vs.head
                        : p.k + b * p.ks.batch + l * p.ks.token + hh * p.ks.head;
    const uint4 raw = *reinterpret_cast<const uint4*>(src + j0);
    float x[E], o[E];
    Vec16<T>::widen(raw, x);
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < E; ++c) ss = __builtin_fmaf(x[c], x[c], ss);
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<LPH>(ss), 1.f / D, p.eps));
#pragma unroll
    for (int c = 0; c < E; ++c) x[c] = x[c] * inv * (is_q ? wq[c] : wk[c]);
#pragma unroll
    for (int c = 0; c < E; ++c) {
      const float other = __shfl(x[c], partner);
      if (turned) {
        const float2 a = cs[t * p.half + jc + c];
        o[c] = upper ? __builtin_fmaf(x[c], a.x, other * a.y) : __builtin_fmaf(x[c], a.x, -other * a.y);
      } else {
        o[c] = x[c];
      }
    }
    uint4 res = is_v ? raw : Vec16<T>::narrow(o);
    if constexpr (APPEND) {
      const int64_t p0 = p.pos[b], at = p0 + l;
      if (p0 < 0) {
        if (!is_q) continue;
        res = make_uint4(0u, 0u, 0u, 0u);
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + (tok * p.Hq + hh) * D + j0) = res;
      } else {
        const int64_t slot = at < p.sinks ? at : p.sinks + (at - p.sinks) % p.window;
        const bool stays = at < p.sinks || p.L - 1 - l < p.window;  // no later token of this call takes the slot
        T* cache = is_v ? p.v_out : p.k_out;
        if (stays)
          *reinterpret_cast<uint4*>(cache + ((b * p.Hk + hh) * (static_cast<int64_t>(p.sinks) + p.window) + slot) * D +
                                    j0) = res;
      }
    } else {
      T* dst = is_q ? p.q_out + (tok * p.Hq + hh) * D : p.k_out + (tok * p.Hk + hh) * D;
      *reinterpret_cast<uint4*>(dst + j0) = res;
    }
  }
}

// With dn the gradient turned back, u = x inv: dw += dn u,
// dx = inv (dn w - u mean(dn w u)). A workgroup takes every gridDim.x-th group
// of tokens; each of its threads keeps the weight gradients of its entries.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void rope_bwd_kernel(const RopeArgs<T> p) {
  constexpr int E = Vec16<T>::kN, LPH = D / E, G = kThreads / LPH;
  extern __shared__ float2 cs[];
  __shared__ float red[G][D];
  const int64_t all = p.Bs * p.L;
  const int li = threadIdx.x % LPH, H = p.Hq + p.Hk, lane = threadIdx.x & 63;
  float wq[E], wk[E], dwq[E], dwk[E];
#pragma unroll
  for (int c = 0; c < E; ++c) {
    wq[c] = p.wq ? p.wq[li * E + c] : 1.f;
    wk[c] = p.wk ? p.wk[li * E + c] : 1.f;
    dwq[c] = dwk[c] = 0.f;
  }
  const int j0 = li * E;
  const bool turned = j0 < 2 * p.half, upper = j0 >= p.half;
  const int partner = !turned ? lane : upper ? lane - p.half / E : lane + p.half / E;
  const int jc = upper ? j0 - p.half : j0;
  for (int64_t first = blockIdx.x * static_cast<int64_t>(p.tokens); first < all;
       first += gridDim.x * static_cast<int64_t>(p.tokens)) {
    const int n = static_cast<int>(all - first < p.tokens ? all - first : p.tokens);
    __syncthreads();  // the last group's angles are no longer read
    angles<T, false>(p, first, n, cs);
    __syncthreads();
    for (int item = threadIdx.x / LPH; item < n * H; item += G) {
      const int t = item / H, h = item % H;
      const int64_t tok = first + t, b = tok / p.L, l = tok % p.L;
      const bool is_q = h < p.Hq;
      const int hh = is_q ? h : h - p.Hq;
      const T* src = is_q ? p.q + b * p.qs.batch + l * p.qs.token + hh * p.qs.head
                          : p.k + b * p.ks.batch + l * p.ks.token + hh * p.ks.head;
      const int64_t o = (is_q ? (tok * p.Hq + hh) : (tok * p.Hk + hh)) * D + j0;
      float x[E], d[E];
      Vec16<T>::widen(*reinterpret_cast<const uint4*>(src + j0), x);
      Vec16<T>::widen(*reinterpret_cast<const uint4*>((is_q ? p.dq_out : p.dk_out) + o), d);
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) ss = __builtin_fmaf(x[c], x[c], ss);
      const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<LPH>(ss), 1.f / D, p.eps));
      float m = 0.f;
#pragma unroll
      for (int c = 0; c < E; ++c) {
        const float other = __shfl(d[c], partner);
        if (turned) {
          const float2 a = cs[t * p.half + jc + c];
          d[c] = upper ? __builtin_fmaf(d[c], a.x, -other * a.y) : __builtin_fmaf(d[c], a.x, other * a.y);
        }
        x[c] *= inv;
        const float g = d[c] * x[c];
        if (is_q) dwq[c] += g; else dwk[c] += g;
        d[c] *= is_q ? wq[c] : wk[c];
        m = __builtin_fmaf(d[c], x[c], m);
      }
      m = head_sum<LPH>(m) * (1.f / D);
#pragma unroll
      for (int c = 0; c < E; ++c) d[c] = inv * __builtin_fmaf(-x[c], m, d[c]);
      *reinterpret_cast<uint4*>((is_q ? p.q_out : p.k_out) + o) = Vec16<T>::narrow(d);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < E; ++c) red[threadIdx.x / LPH][j0 + c] = w ? dwk[c] : dwq[c];
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kThreads) {
      float v = 0.f;
      for (int g = 0; g < G; ++g) v += red[g][j];
      p.part[(blockIdx.x * 2ll + w) * D + j] = v;
    }
  }
}

// dwq, dwk (D) = sums over rows of part (rows, 2, D), in a fixed order: 64
// threads of a column each sum every 64th row, their sums are added in thread
// order.
__global__ __launch_bounds__(1024) void rope_dw_kernel(const float* part, float* dwq, float* dwk, int rows, int D) {
  __shared__ float sum[64][17];
  const int ce = threadIdx.x & 15, cr = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + ce;  // of 2 D
  float v = 0.f;
#pragma unroll 8
  for (int r = cr; r < rows; r += 64) v += part[static_cast<int64_t>(r) * 2 * D + e];
  sum[cr][ce] = v;
  __syncthreads();
  if (cr != 0) return;
#pragma unroll
  for (int j = 1; j < 64; ++j) v += sum[j][ce];
  if (e < D) {
    if (dwq) dwq[e] = v;
  } else if (dwk) {
    dwk[e - D] = v;
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int rope_sizes(int64_t Bs, int64_t L, int64_t Hq, int64_t Hk, int64_t D, int64_t R, double eps, int dtype,
               int64_t* nq, int64_t* nk) {
  int64_t t, bytes;
  if (!mul_nn(Bs, L, &t) || !mul_nn(Hq, D, nq) || !mul_nn(Hk, D, nk) || !mul_nn(t, *nq, nq) || !mul_nn(t, *nk, nk) ||
      !mul_nn(*nq, 8, &bytes) || !mul_nn(*nk, 8, &bytes) || R < 0)
    return SSM_ERR_DIM;
  if (Hq + Hk > (1 << 20)) return SSM_ERR_DIM;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if ((D != 64 && D != 128) || R > D || R % 16) return SSM_ERR_UNSUPPORTED;
  if (!(eps >= 0) || eps > 1e30) return SSM_ERR_ARG;
  return SSM_OK;
}

// Tokens of a workgroup: about eight heads' vectors a thread, at most
// kMaxTokens (their angles fit LDS), fewer when there are few tokens.
int rope_tokens(int64_t all, int64_t H, int64_t D, int E) {
  int64_t t = 8 * kThreads / std::max<int64_t>(1, H * D / E);
  t = std::min<int64_t>(std::max<int64_t>(t, 1), kMaxTokens);
  while (t > 1 && all / t < 1024) t /= 2;
  return static_cast<int>(t);
}

int rope_bwd_blocks(int64_t all, int tokens) {
  return static_cast<int>(std::min<int64_t>((all + tokens - 1) / tokens, kMaxBlocks));
}

template <typename T>
RopeArgs<T> rope_args(const void* q, ssm_strides qs, const void* k, ssm_strides ks, const float* wq, const float* wk,
                      const double* freq, const int32_t* pos, double eps, int64_t Bs, int64_t L, int64_t Hq,
                      int64_t Hk, int64_t D, int64_t R, int64_t heads) {
  RopeArgs<T> a{};
  a.q = static_cast<const T*>(q), a.k = static_cast<const T*>(k), a.qs = qs, a.ks = ks;
  a.wq = wq, a.wk = wk, a.freq = freq, a.pos = pos, a.eps = static_cast<float>(eps);
  a.Bs = Bs, a.L = L, a.Hq = static_cast<int>(Hq), a.Hk = static_cast<int>(Hk), a.half = static_cast<int>(R / 2);
  a.tokens = rope_tokens(Bs * L, heads, D, Vec16<T>::kN);
  return a;
}

template <typename T, bool APPEND>
int launch_rope(const RopeArgs<T>& a, int64_t D, hipStream_t st) {
  const int64_t blocks = (a.Bs * a.L + a.tokens - 1) / a.tokens;
  if (blocks > kMaxGrid) return SSM_ERR_DIM;
  const dim3 grid(static_cast<unsigned>(blocks));
  const size_t lds = static_cast<size_t>(a.tokens) * a.half * sizeof(float2);
  if (D == 64)
    hipLaunchKernelGGL((rope_kernel<T, 64, APPEND>), grid, dim3(kThreads), lds, st, a);
  else
    hipLaunchKernelGGL((rope_kernel<T, 128, APPEND>), grid, dim3(kThreads), lds, st, a);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

template <typename T>
int launch_rope_bwd(RopeArgs<T> a, float* dwq, float* dwk, int64_t D, hipStream_t st) {
  const int blocks = rope_bwd_blocks(a.Bs * a.L, a.tokens);
  const size_t lds = static_cast<size_t>(a.tokens) * a.half * sizeof(float2);
  if (D == 64)
    hipLaunchKernelGGL((rope_bwd_kernel<T, 64>), dim3(blocks), dim3(kThreads), lds, st, a);
  else
    hipLaunchKernelGGL((rope_bwd_kernel<T, 128>), dim3(blocks), dim3(kThreads), lds, st, a);
  if (a.part)
    hipLaunchKernelGGL(rope_dw_kernel, dim3(static_cast<unsigned>(2 * D / 16)), dim3(1024), 0, st, a.part, dwq, dwk,
                       blocks, static_cast<int>(D));
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

}  // namespace

extern "C" int ssm_qk_rope_fwd(const void* q, const ssm_strides* qs, const void* k, const ssm_strides* ks,
                               const float* wq, const float* wk, const double* freq, const int32_t* pos, double eps,
                               void* q_out, void* k_out, int64_t Bs, int64_t L, int64_t Hq, int64_t Hk, int64_t D,
                               int64_t R, int dtype, void* stream) {
  int64_t nq, nk, bq, bk;
  int rc = rope_sizes(Bs, L, Hq, Hk, D, R, eps, dtype, &nq, &nk);
  if (rc != SSM_OK) return rc;
  const int es = dtype == SSM_F32 ? 4 : 2;
  ssm_strides sq, sk;
  if ((rc = strided(qs, Bs, L, Hq, D, es, &sq, &bq)) != SSM_OK) return rc;
  if ((rc = strided(ks, Bs, L, Hk, D, es, &sk, &bk)) != SSM_OK) return rc;
  const int64_t any = nq + nk > 0;
  const Buf bufs[] = {{q, bq, true, false},       {k, bk, true, false},          {wq, D * 4, false, false},
                      {wk, D * 4, false, false},  {freq, any * R * 4, true, false}, {pos, any * Bs * L * 4, false, false, 4},
                      {q_out, nq * es, true, true}, {k_out, nk * es, true, true}};
  if ((rc = check_bufs(bufs, 8)) != SSM_OK) return rc;
  if (!any) return SSM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    RopeArgs<T> a = rope_args<T>(q, sq, k, sk, wq, wk, freq, pos, eps, Bs, L, Hq, Hk, D, R, Hq + Hk);
    a.q_out = static_cast<T*>(q_out), a.k_out = static_cast<T*>(k_out);
    return launch_rope<T, false>(a, D, st);
  };
  return dtype == SSM_F32 ? go(float{}) : go(uint16_t{});
}

extern "C" size_t ssm_qk_rope_bwd_workspace_bytes(int64_t Bs, int64_t L, int64_t Hq, int64_t Hk, int64_t D,
                                                  int dtype) {
  int64_t nq, nk;
  if (rope_sizes(Bs, L, Hq, Hk, D, 0, 0.0, dtype, &nq, &nk) != SSM_OK || nq + nk == 0) return 0;
  const int tokens = rope_tokens(Bs * L, Hq + Hk, D, dtype == SSM_F32 ? 4 : 8);
  return static_cast<size_t>(rope_bwd_blocks(Bs * L, tokens)) * 2 * D * 4;
}

extern "C" int ssm_qk_rope_bwd(const void* q, const ssm_strides* qs, const void* k, const ssm_strides* ks,
                               const float* wq, const float* wk, const double* freq, const int32_t* pos, double eps,
                               const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                               int64_t Bs, int64_t L, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int dtype,
                               void* workspace, size_t workspace_bytes, void* stream) {
  int64_t nq, nk, bq, bk;
  int rc = rope_sizes(Bs, L, Hq, Hk, D, R, eps, dtype, &nq, &nk);
  if (rc != SSM_OK) return rc;
  const int es = dtype == SSM_F32 ? 4 : 2;
  ssm_strides sq, sk;
  if ((rc = strided(qs, Bs, L, Hq, D, es, &sq, &bq)) != SSM_OK) return rc;
  if ((rc = strided(ks, Bs, L, Hk, D, es, &sk, &bk)) != SSM_OK) return rc;
  const int64_t any = nq + nk > 0;
  const bool weights = dwq || dwk;
  const size_t need = weights ? ssm_qk_rope_bwd_workspace_bytes(Bs, L, Hq, Hk, D, dtype) : 0;
  const Buf bufs[] = {{q, bq, true, false},        {k, bk, true, false},           {wq, D * 4, false, false},
                      {wk, D * 4, false, false},   {freq, any * R * 4, true, false}, {pos, any * Bs * L * 4, false, false, 4},
                      {dq_out, nq * es, true, false}, {dk_out, nk * es, true, false}, {dq, nq * es, true, true},
                      {dk, nk * es, true, true},   {dwq, D * 4, false, true},      {dwk, D * 4, false, true},
                      {workspace, static_cast<int64_t>(need), false, true}};
  if ((rc = check_bufs(bufs, 13)) != SSM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (!any) return fill_async(dwq, nullptr, D * 4, st) && fill_async(dwk, nullptr, D * 4, st) ? SSM_OK : SSM_ERR_LAUNCH;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  auto go = [&](auto tag) {
    using T = decltype(tag);
    RopeArgs<T> a = rope_args<T>(q, sq, k, sk, wq, wk, freq, pos, eps, Bs, L, Hq, Hk, D, R, Hq + Hk);
    a.dq_out = static_cast<const T*>(dq_out), a.dk_out = static_cast<const T*>(dk_out);
    a.q_out = static_cast<T*>(dq), a.k_out = static_cast<T*>(dk);
    a.part = weights ? static_cast<float*>(workspace) : nullptr;
    return launch_rope_bwd<T>(a, dwq, dwk, D, st);
  };
  return dtype == SSM_F32 ? go(float{}) : go(uint16_t{});
}

extern "C" int ssm_qk_rope_append(const void* q, const ssm_strides* qs, const void* k, const ssm_strides* ks,
                                  const void* v, const ssm_strides* vs, const float* wq, const float* wk,
                                  const double* freq, const int32_t* pos, double eps, void* q_out, void* k_cache,
                                  void* v_cache, int64_t Bs, int64_t L, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                                  int64_t window, int64_t sinks, int dtype, void* stream) {
  int64_t nq, nk, bq, bk, bv, rows, slots, bc;
  int rc = rope_sizes(Bs, L, Hq, Hk, D, R, eps, dtype, &nq, &nk);
  if (rc != SSM_OK) return rc;
  if (window < 1 || sinks < 0 || window > INT32_MAX || sinks > INT32_MAX || window + sinks > INT32_MAX)
    return SSM_ERR_DIM;
  const int es = dtype == SSM_F32 ? 4 : 2;
  if (!mul_nn(Bs, Hk, &rows) || !mul_nn(rows, window + sinks, &slots) || !mul_nn(slots, D * es, &bc)) return SSM_ERR_DIM;
  ssm_strides sq, sk, sv;
  if ((rc = strided(qs, Bs, L, Hq, D, es, &sq, &bq)) != SSM_OK) return rc;
  if ((rc = strided(ks, Bs, L, Hk, D, es, &sk, &bk)) != SSM_OK) return rc;
  if ((rc = strided(vs, Bs, L, Hk, D, es, &sv, &bv)) != SSM_OK) return rc;
  const int64_t any = nq + nk > 0;
  const Buf bufs[] = {{q, bq, true, false},      {k, bk, true, false},           {v, bv, true, false},
                      {wq, D * 4, false, false}, {wk, D * 4, false, false},      {freq, any * R * 4, true, false},
                      {pos, any * Bs * 4, true, false, 4}, {q_out, nq * es, true, true}, {k_cache, any * bc, true, true},
                      {v_cache, any * bc, true, true}};
  if ((rc = check_bufs(bufs, 10)) != SSM_OK) return rc;
  if (!any) return SSM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    RopeArgs<T> a = rope_args<T>(q, sq, k, sk, wq, wk, freq, pos, eps, Bs, L, Hq, Hk, D, R, Hq + 2 * Hk);
    a.v = static_cast<const T*>(v), a.vs = sv;
    a.q_out = static_cast<T*>(q_out), a.k_out = static_cast<T*>(k_cache), a.v_out = static_cast<T*>(v_cache);
    a.window = static_cast<int>(window), a.sinks = static_cast<int>(sinks);
    return launch_rope<T, true>(a, D, st);
  };
  return dtype == SSM_F32 ? go(float{}) : go(uint16_t{});
}
