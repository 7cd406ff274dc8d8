// Attention with a sliding window and sinks (ssm_swa_fwd, ssm_swa_bwd of
// ssm_hybrid.h) for gfx950.
//
//   s_ij = scale q_i . k_j over the keys j that query i sees
//   o_i = sum_j e^(s_ij - lse_i) v_j,   lse_i = log sum_j e^(s_ij)
//   with p = e^(s - lse), delta_i = do_i . o_i, ds = p (do_i . v_j - delta_i):
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// Forward and dq: a wave owns 32 queries (a lane's column) and goes over tiles
// of keys in LDS; dk and dv: a wave owns 32 keys and goes over tiles of
// queries, of all the heads that share them. The pairs with the sinks are kept
// out of the latter and taken by workgroups that share them by ranges of
// queries, since every query sees the sinks. All sums run in a fixed order.
//
// A matrix product takes every pair of a tile, seen or not, the unseen ones
// with weight 0: 0 times a value that is not finite would spoil the sum. Rows
// past the valid ones are never read; if a result is not finite all the same,
// the wave computes its rows again from the pairs that are seen alone.
#include "swa_common.h"

namespace {

constexpr int kWaves = 4, kNT = 64 * kWaves;
constexpr int kOwn = 32 * kWaves;  // queries (or keys) of a workgroup

// rows of an LDS tile: 16 KiB of them, at most 64
template <typename T, int D>
constexpr int kRows = 16384 / (D * static_cast<int>(sizeof(T))) < 64 ? 32 : 64;

template <typename T>
struct Place {
  int b, hk, h, blk;
};
// Work order: batch row, key head, block of queries, head of the group.
template <typename T>
__device__ __forceinline__ Place<T> place_q(const SwaArgs<T>& p) {
  int w = xcd_order(blockIdx.x, p.nwork);
  Place<T> r;
  const int g = w % p.G;
  w /= p.G;
  r.blk = w % p.nblk;
  w /= p.nblk;
  r.hk = w % p.Hk;
  r.b = w / p.Hk;
  r.h = r.hk * p.G + g;
  return r;
}

// ---------------------------------------------------------------------------
// pair by pair: what a wave falls back to. A lane holds D / 64 entries.
// ---------------------------------------------------------------------------
template <typename T, int D>
struct Lane {
  float v[D / 64];
  __device__ __forceinline__ Lane() {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) v[c] = 0.f;
  }
  __device__ __forceinline__ explicit Lane(const T* p, int lane) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) v[c] = to_f32(p[64 * c + lane]);
  }
  __device__ __forceinline__ float dot(const Lane& o) const {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) s = __builtin_fmaf(v[c], o.v[c], s);
    return wave_sum(s);
  }
  __device__ __forceinline__ void add(float w, const Lane& o) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) v[c] = __builtin_fmaf(w, o.v[c], v[c]);
  }
};

template <typename T>
__device__ __forceinline__ const T* row_of(const T* x, const ssm_strides& s, int b, int t, int h) {
  return x + b * s.batch + t * s.token + h * s.head;
}
template <typename T>
__device__ __forceinline__ int64_t dense_row(const SwaArgs<T>& p, int b, int i, int h) {
  return (static_cast<int64_t>(b) * p.Lq + i) * p.Hq + h;
}

// f(j) for the keys that position pos sees, in order.
template <typename F>
__device__ __forceinline__ void seen_keys(const Mask& m, int pos, F f) {
  const int top = pos < m.nk - 1 ? pos : m.nk - 1, lo = pos - m.W + 1 > 0 ? pos - m.W + 1 : 0;
  for (int j = 0; j < m.S && j < lo && j <= top; ++j) f(j);
  for (int j = lo; j <= top; ++j) f(j);
}

template <typename T, int D>
__device__ __forceinline__ void fwd_by_pairs(const SwaArgs<T>& p, const Mask& m, int b, int hk, int h, int i0,
                                                       int lane) {
  const float sc = p.scale * kLog2e;
  for (int i = i0; i < i0 + 32 && i < p.Lq; ++i) {
    const Lane<T, D> q(row_of(p.q, p.qs, b, i, h), lane);
    Lane<T, D> o;
    float top = -INFINITY, l = 0.f;
    seen_keys(m, i + p.Lk - p.Lq, [&](int j) {
      const float s = q.dot(Lane<T, D>(row_of(p.k, p.ks, b, j, hk), lane)) * sc;
      const float t = s > top || s != s ? s : top;
      const float keep = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - t);
      const float w = t == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s - t);
      top = t;
      l = __builtin_fmaf(l, keep, w);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) o.v[c] *= keep;
      o.add(w, Lane<T, D>(row_of(p.v, p.vs, b, j, hk), lane));
    });
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) p.out[dense_row(p, b, i, h) * D + 64 * c + lane] = from_f32<T>(o.v[c] * inv);
    if (p.lse && lane == 0)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i] = l == 0.f ? -INFINITY : top / kLog2e + logf(l);
  }
}

template <typename T, int D>
__device__ __forceinline__ void dq_by_pairs(const SwaArgs<T>& p, const Mask& m, int b, int hk, int h, int i0,
                                                      int lane) {
  const float sc = p.scale * kLog2e;
  for (int i = i0; i < i0 + 32 && i < p.Lq; ++i) {
    const Lane<T, D> q(row_of(p.q, p.qs, b, i, h), lane), go(p.dout + dense_row(p, b, i, h) * D, lane);
    const int64_t st = (static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i;
    const float lse = p.lse[st] * kLog2e, delta = p.delta[st];
    Lane<T, D> dq;
    seen_keys(m, i + p.Lk - p.Lq, [&](int j) {
      const Lane<T, D> k(row_of(p.k, p.ks, b, j, hk), lane);
      const float w = __builtin_amdgcn_exp2f(q.dot(k) * sc - lse);
      dq.add(w * (go.dot(Lane<T, D>(row_of(p.v, p.vs, b, j, hk), lane)) - delta), k);
    });
#pragma unroll
    for (int c = 0; c < D / 64; ++c) p.dq[dense_row(p, b, i, h) * D + 64 * c + lane] = from_f32<T>(dq.v[c] * p.scale);
  }
}

// dk and dv of key j from the queries i0 .. i1 - 1 of head h (scale left out).
template <typename T, int D>
__device__ __forceinline__ void dkdv_pairs(const SwaArgs<T>& p, const Mask& m, int b, int hk, int h, int j, int i0, int i1,
                                           int lane, Lane<T, D>& dk, Lane<T, D>& dv) {
  const float sc = p.scale * kLog2e;
  const Lane<T, D> k(row_of(p.k, p.ks, b, j, hk), lane), v(row_of(p.v, p.vs, b, j, hk), lane);
  for (int i = i0; i < i1; ++i) {
    if (!m.sees(i + p.Lk - p.Lq, j)) continue;
    const Lane<T, D> q(row_of(p.q, p.qs, b, i, h), lane), go(p.dout + dense_row(p, b, i, h) * D, lane);
    const int64_t st = (static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i;
    const float w = __builtin_amdgcn_exp2f(q.dot(k) * sc - p.lse[st] * kLog2e);
    dv.add(w, go);
    dk.add(w * (go.dot(v) - p.delta[st]), q);
  }
}

template <typename T, int D>
__device__ __forceinline__ void dkdv_by_pairs(const SwaArgs<T>& p, const Mask& m, int b, int hk, int j0,
                                                        int lane) {
  for (int j = j0 > p.S ? j0 : p.S; j < j0 + 32 && j < p.Lk; ++j) {
    Lane<T, D> dk, dv;
    const int64_t first = static_cast<int64_t>(j) - p.Lk + p.Lq, end = first + p.W;
    for (int g = 0; g < p.G && j < m.nk; ++g)
      dkdv_pairs<T, D>(p, m, b, hk, hk * p.G + g, j, first < 0 ? 0 : static_cast<int>(first),
                       end > p.Lq ? p.Lq : static_cast<int>(end), lane, dk, dv);
    const int64_t o = ((static_cast<int64_t>(b) * p.Lk + j) * p.Hk + hk) * D;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      p.dk[o + 64 * c + lane] = from_f32<T>(dk.v[c] * p.scale);
      p.dv[o + 64 * c + lane] = from_f32<T>(dv.v[c]);
    }
  }
}

// Column n of a result tile set X (D / 32 tiles: rows d) as row `row` of a
// (.., D) tensor: a lane holds 4 neighbouring d at a time.
template <typename T, int D>
__device__ __forceinline__ void store_col(T* row, const v16f (&x)[D / 32], float mul, int hi) {
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      Vec4<T>::store(row + 32 * db + 8 * r + 4 * hi, make_float4(x[db][4 * r] * mul, x[db][4 * r + 1] * mul,
                                                                 x[db][4 * r + 2] * mul, x[db][4 * r + 3] * mul));
}
template <int D>
__device__ __forceinline__ bool all_finite(const v16f (&x)[D / 32], float mul) {
  float s = 0.f;  // 0 times a value that is not finite is NaN
#pragma unroll
  for (int db = 0; db < D / 32; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) s = __builtin_fmaf(0.f, x[db][r] * mul, s);
  return s == 0.f;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ __launch_bounds__(kNT, 2) void swa_fwd_kernel(const SwaArgs<T> p) {
  constexpr int KB = kRows<T, D>, NB = KB / 32, KK = D / 16, DB = D / 32;
  using KT = Tile<T, D, KB>;
  __shared__ __attribute__((aligned(16))) char sm[2][2][KT::kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, hi = lane >> 5;
  const Place<T> w = place_q(p);
  const Mask m = mask_of(p, w.b);
  const int off = p.Lk - p.Lq, i0 = w.blk * kOwn + 32 * wave, i = i0 + n;
  const int pos = i + off, pw0 = i0 + off, pw1 = pw0 + 31;
  const int last_i = w.blk * kOwn + kOwn - 1 < p.Lq - 1 ? w.blk * kOwn + kOwn - 1 : p.Lq - 1;
  const KeyTiles tiles(m, w.blk * kOwn + off, last_i + off, KB);
  const T* kbase = p.k + w.b * p.ks.batch + w.hk * p.ks.head;
  const T* vbase = p.v + w.b * p.vs.batch + w.hk * p.vs.head;

  Frag<T> q[KK];
  {
    const T* qr = row_of(p.q, p.qs, w.b, i < p.Lq ? i : p.Lq - 1, w.h);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) q[kk] = load_frag(qr + 16 * kk + 8 * hi);
  }
  const float sc = p.scale * kLog2e;
  float top = -INFINITY, l = 0.f;  // the running maximum (of s log2 e) and this lane's part of the sum
  v16f o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = v16f{};

  if (tiles.n > 0) {
    const int k0 = tiles.key0(0, KB);
    KT::template load<kNT>(kbase, p.ks.token, k0, m.nk - 1, sm[0][0], wave, lane);
    KT::template load<kNT>(vbase, p.vs.token, k0, m.nk - 1, sm[0][1], wave, lane);
  }
  for (int t = 0; t < tiles.n; ++t) {
    wait_loads();
    __syncthreads();  // tile t is in LDS; nobody reads the other buffer any more
    if (t + 1 < tiles.n) {
      const int k1 = tiles.key0(t + 1, KB);
      KT::template load<kNT>(kbase, p.ks.token, k1, m.nk - 1, sm[(t + 1) & 1][0], wave, lane);
      KT::template load<kNT>(vbase, p.vs.token, k1, m.nk - 1, sm[(t + 1) & 1][1], wave, lane);
    }
    const int k0 = tiles.key0(t, KB);
    if (m.none(pw0, pw1, k0, k0 + KB - 1)) continue;
    const char *ks = sm[t & 1][0], *vs = sm[t & 1][1];
    v16f s[NB];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      s[kb] = v16f{};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) s[kb] = mma(KT::row(ks, 32 * kb + n, kk, hi), q[kk], s[kb]);
    }
    if (!m.all(pw0, pw1, k0, k0 + KB - 1)) {
#pragma unroll
      for (int kb = 0; kb < NB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!m.sees(pos, k0 + 32 * kb + 8 * (r >> 2) + 4 * hi + (r & 3))) s[kb][r] = -INFINITY;
    }
    float mx = s[0][0];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[kb][r]);
    const float now = fmaxf(top, pair_max(mx) * sc);
    const float keep = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - now);
    const float ref = now == -INFINITY ? 0.f : now;  // (a row that has seen nothing: every weight is 0)
    top = now;
    l *= keep;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[kb][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][r], sc, -ref));
        l += s[kb][r];
      }
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] *= keep;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> w8 = as_operand<T>(s[kb], h);
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = mma(KT::col(vs, 32 * kb + 16 * h, d, lane), w8, o[d]);
      }
  }
  l = pair_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (__ballot(!all_finite<D>(o, inv) || l != l)) {
    fwd_by_pairs<T, D>(p, m, w.b, w.hk, w.h, i0, lane);
    return;
  }
  if (i >= p.Lq) return;
  store_col<T, D>(p.out + dense_row(p, w.b, i, w.h) * D, o, inv, hi);
  if (p.lse && hi == 0)
    p.lse[(static_cast<int64_t>(w.b) * p.Hq + w.h) * p.Lq + i] = l == 0.f ? -INFINITY : top / kLog2e + logf(l);
}

// ---------------------------------------------------------------------------
// dq (and delta)
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ __launch_bounds__(kNT, 2) void swa_dq_kernel(const SwaArgs<T> p) {
  constexpr int KB = kRows<T, D>, NB = KB / 32, KK = D / 16, DB = D / 32;
  using KT = Tile<T, D, KB>;
  __shared__ __attribute__((aligned(16))) char sm[2][2][KT::kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, hi = lane >> 5;
  const Place<T> w = place_q(p);
  const Mask m = mask_of(p, w.b);
  const int off = p.Lk - p.Lq, i0 = w.blk * kOwn + 32 * wave, i = i0 + n;
  const int pos = i + off, pw0 = i0 + off, pw1 = pw0 + 31;
  const int last_i = w.blk * kOwn + kOwn - 1 < p.Lq - 1 ? w.blk * kOwn + kOwn - 1 : p.Lq - 1;
  const KeyTiles tiles(m, w.blk * kOwn + off, last_i + off, KB);
  const T* kbase = p.k + w.b * p.ks.batch + w.hk * p.ks.head;
  const T* vbase = p.v + w.b * p.vs.batch + w.hk * p.vs.head;
  const int ic = i < p.Lq ? i : p.Lq - 1;
  const int64_t st = (static_cast<int64_t>(w.b) * p.Hq + w.h) * p.Lq + ic;

  Frag<T> q[KK], go[KK];
  float delta = 0.f;
  {
    const T* qr = row_of(p.q, p.qs, w.b, ic, w.h);
    const T* gr = p.dout + dense_row(p, w.b, ic, w.h) * D;
    const T* orow = p.o + dense_row(p, w.b, ic, w.h) * D;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      q[kk] = load_frag(qr + 16 * kk + 8 * hi);
      go[kk] = load_frag(gr + 16 * kk + 8 * hi);
      delta += frag_dot(go[kk], load_frag(orow + 16 * kk + 8 * hi));
    }
  }
  delta = pair_sum(delta);
  if (hi == 0 && i < p.Lq) p.delta[st] = delta;
  float lse = p.lse[st] * kLog2e;
  if (lse == -INFINITY) lse = 0.f;  // nothing seen: every weight is masked
  const float sc = p.scale * kLog2e;
  v16f dq[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dq[d] = v16f{};

  if (tiles.n > 0) {
    const int k0 = tiles.key0(0, KB);
    KT::template load<kNT>(kbase, p.ks.token, k0, m.nk - 1, sm[0][0], wave, lane);
    KT::template load<kNT>(vbase, p.vs.token, k0, m.nk - 1, sm[0][1], wave, lane);
  }
  for (int t = 0; t < tiles.n; ++t) {
    wait_loads();
    __syncthreads();
    if (t + 1 < tiles.n) {
      const int k1 = tiles.key0(t + 1, KB);
      KT::template load<kNT>(kbase, p.ks.token, k1, m.nk - 1, sm[(t + 1) & 1][0], wave, lane);
      KT::template load<kNT>(vbase, p.vs.token, k1, m.nk - 1, sm[(t + 1) & 1][1], wave, lane);
    }
    const int k0 = tiles.key0(t, KB);
    if (m.none(pw0, pw1, k0, k0 + KB - 1)) continue;
    const bool full = m.all(pw0, pw1, k0, k0 + KB - 1);
    const char *ks = sm[t & 1][0], *vs = sm[t & 1][1];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      v16f s = v16f{}, dp = v16f{};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        s = mma(KT::row(ks, 32 * kb + n, kk, hi), q[kk], s);
        dp = mma(KT::row(vs, 32 * kb + n, kk, hi), go[kk], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float wt = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], sc, -lse));
        s[r] = wt * (dp[r] - delta);
      }
      if (!full) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!m.sees(pos, k0 + 32 * kb + 8 * (r >> 2) + 4 * hi + (r & 3))) s[r] = 0.f;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> ds = as_operand<T>(s, h);
#pragma unroll
        for (int d = 0; d < DB; ++d) dq[d] = mma(KT::col(ks, 32 * kb + 16 * h, d, lane), ds, dq[d]);
      }
    }
  }
  if (__ballot(!all_finite<D>(dq, p.scale))) {
    __threadfence_block();  // delta, written by this wave, is read back
    dq_by_pairs<T, D>(p, m, w.b, w.hk, w.h, i0, lane);
    return;
  }
  if (i < p.Lq) store_col<T, D>(p.dq + dense_row(p, w.b, i, w.h) * D, dq, p.scale, hi);
}

// ---------------------------------------------------------------------------
// dk and dv. SINK: the keys below S, 32 to a workgroup, whose waves take the
// rows of the query tiles in turn and add their sums at the end; the
// workgroups of a block of keys share the query tiles by ranges and leave
// float32 partial sums.
// ---------------------------------------------------------------------------
template <typename T, int D, bool SINK>
__global__ __launch_bounds__(kNT, 1) void swa_dkdv_kernel(const SwaArgs<T> p) {
  constexpr int QB = kRows<T, D>, NB = QB / 32, KK = D / 16, DB = D / 32;
  using QT = Tile<T, D, QB>;
  __shared__ __attribute__((aligned(16))) char sm[2][2][QT::kBytes];
  __shared__ __attribute__((aligned(16))) float stat[2][2][64];  // lse, delta of a tile's rows
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, hi = lane >> 5;
  int w = SINK ? blockIdx.x : xcd_order(blockIdx.x, p.nwork);
  int chunk = 0;
  if (SINK) {
    chunk = w % p.nchunk;
    w /= p.nchunk;
  }
  const int blk = w % p.nblk;
  w /= p.nblk;
  const int hk = w % p.Hk, b = w / p.Hk;
  const Mask m = mask_of(p, b);
  const int off = p.Lk - p.Lq, j0 = SINK ? 32 * blk : blk * kOwn + 32 * wave, j = j0 + n;
  // the queries that may see the workgroup's keys, by tiles
  const int jb = SINK ? j0 : blk * kOwn, jend = SINK ? j0 + 31 : jb + kOwn - 1;
  const int ilo = jb - off > 0 ? jb - off : 0;
  const int64_t far = SINK ? p.Lq - 1 : static_cast<int64_t>(jend) + p.W - 1 - off;
  const int ihi = far < p.Lq - 1 ? static_cast<int>(far) : p.Lq - 1;
  const int t0 = ilo / QB, nt = m.nk > jb && ihi >= ilo && (SINK || jend >= p.S) ? ihi / QB - t0 + 1 : 0;
  int first = 0, end = nt * p.G;  // (head of the group, tile), flattened
  if (SINK) {
    const int all = end;
    first = static_cast<int>(static_cast<int64_t>(all) * chunk / p.nchunk);
    end = static_cast<int>(static_cast<int64_t>(all) * (chunk + 1) / p.nchunk);
  }

  Frag<T> k[KK], v[KK];
  if (end > first) {
    const int jc = j < m.nk ? j : m.nk - 1;
    const T* kr = row_of(p.k, p.ks, b, jc, hk);
    const T* vr = row_of(p.v, p.vs, b, jc, hk);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      k[kk] = load_frag(kr + 16 * kk + 8 * hi);
      v[kk] = load_frag(vr + 16 * kk + 8 * hi);
    }
  }
  const float sc = p.scale * kLog2e;
  v16f dk[DB], dv[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dk[d] = v16f{}, dv[d] = v16f{};

  auto load = [&](int f, int buf) {
    const int h = hk * p.G + f / nt, i0 = (t0 + f % nt) * QB;
    QT::template load<kNT>(p.q + b * p.qs.batch + h * p.qs.head, p.qs.token, i0, p.Lq - 1, sm[buf][0], wave, lane);
    QT::template load<kNT>(p.dout + (static_cast<int64_t>(b) * p.Lq * p.Hq + h) * D, static_cast<int64_t>(p.Hq) * D, i0,
                           p.Lq - 1, sm[buf][1], wave, lane);
    if (wave < 2) {
      const int i = i0 + lane < p.Lq - 1 ? i0 + lane : p.Lq - 1;
      const float* src = (wave ? p.delta : p.lse) + (static_cast<int64_t>(b) * p.Hq + h) * p.Lq + i;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                       (__attribute__((address_space(3))) void*)stat[buf][wave], 4, 0, 0);
    }
  };
  if (first < end) load(first, 0);
  for (int f = first; f < end; ++f) {
    const int cur = (f - first) & 1;
    wait_loads();
    __syncthreads();
    if (f + 1 < end) load(f + 1, cur ^ 1);
    const int i0 = (t0 + f % nt) * QB;
    const char *qs = sm[cur][0], *gs = sm[cur][1];
#pragma unroll
    for (int rb = 0; rb < NB; ++rb) {
      const int ib = i0 + 32 * rb;
      if (SINK && ((f - first) * NB + rb) % kWaves != wave) continue;
      const int pb0 = ib + off, pb1 = pb0 + 31;
      if (ib >= p.Lq || m.none(pb0, pb1, j0, j0 + 31)) continue;
      v16f s = v16f{}, dp = v16f{};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        s = mma(QT::row(qs, 32 * rb + n, kk, hi), k[kk], s);
        dp = mma(QT::row(gs, 32 * rb + n, kk, hi), v[kk], dp);
      }
      const bool full = m.all(pb0, pb1, j0, j0 + 31) && ib + 31 < p.Lq && (SINK ? j0 + 31 < p.S : j0 >= p.S);
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const float4 ls = *reinterpret_cast<const float4*>(&stat[cur][0][32 * rb + 8 * r4 + 4 * hi]);
        const float4 de = *reinterpret_cast<const float4*>(&stat[cur][1][32 * rb + 8 * r4 + 4 * hi]);
        const float lv[4] = {ls.x, ls.y, ls.z, ls.w}, dl[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = 4 * r4 + c;
          float wt = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], sc, -lv[c] * kLog2e));
          float ds = wt * (dp[r] - dl[c]);
          if (!full) {
            const int i = ib + 8 * r4 + 4 * hi + c;
            const bool seen = i < p.Lq && m.sees(i + off, j) && (SINK ? j < p.S : j >= p.S);
            wt = seen ? wt : 0.f;
            ds = seen ? ds : 0.f;
          }
          s[r] = wt;
          dp[r] = ds;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> wt = as_operand<T>(s, h), ds = as_operand<T>(dp, h);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          dv[d] = mma(QT::col(gs, 32 * rb + 16 * h, d, lane), wt, dv[d]);
          dk[d] = mma(QT::col(qs, 32 * rb + 16 * h, d, lane), ds, dk[d]);
        }
      }
    }
  }
  if constexpr (!SINK) {
    if (__ballot(!all_finite<D>(dk, p.scale) || !all_finite<D>(dv, 1.f))) {
      dkdv_by_pairs<T, D>(p, m, b, hk, j0, lane);
      return;
    }
    if (j >= p.S && j < p.Lk) {
      const int64_t o = ((static_cast<int64_t>(b) * p.Lk + j) * p.Hk + hk) * D;
      store_col<T, D>(p.dk + o, dk, p.scale, hi);
      store_col<T, D>(p.dv + o, dv, 1.f, hi);
    }
  } else {
    // the four waves' sums, in wave order, through LDS (32 x D float32, dk then dv)
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 64 * D;
    float* acc = reinterpret_cast<float*>(&sm[0][0][0]);  // [2][32][D]: at most 32 KiB of the tiles' 64
    for (int x = 0; x < kWaves; ++x) {
      __syncthreads();
      if (wave == x)
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int e = 32 * d + 8 * (r >> 2) + 4 * hi + (r & 3);
            float* a = acc + n * D + e;
            a[0] = x ? a[0] + dk[d][r] : dk[d][r];
            a[32 * D] = x ? a[32 * D] + dv[d][r] : dv[d][r];
          }
    }
    __syncthreads();
    bool bad = false;
    for (int e = threadIdx.x; e < 64 * D; e += kNT) {
      bad = bad || !finite(acc[e]);
      part[e] = acc[e];
    }
    if (__syncthreads_or(bad)) {
      for (int c = wave; c < 32 && j0 + c < p.S && j0 + c < p.Lk; c += kWaves) {
        Lane<T, D> sk, sv;
        if (j0 + c < m.nk)
          for (int f = first; f < end; ++f) {
            const int i = (t0 + f % nt) * QB;
            dkdv_pairs<T, D>(p, m, b, hk, hk * p.G + f / nt, j0 + c, i, i + QB < p.Lq ? i + QB : p.Lq, lane, sk, sv);
          }
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          part[c * D + 64 * e + lane] = sk.v[e];
          part[(32 + c) * D + 64 * e + lane] = sv.v[e];
        }
      }
    }
  }
}

// dk and dv of the sinks: the sum of the partial sums, in order.
template <typename T>
__global__ __launch_bounds__(256) void swa_sink_join_kernel(const SwaArgs<T> p, int Bs, int D) {
  const int keys = p.S < p.Lk ? p.S : p.Lk;
  const int64_t item = blockIdx.x * 256ll + threadIdx.x, all = static_cast<int64_t>(Bs) * keys * p.Hk * 2 * D;
  if (item >= all) return;
  const int d = static_cast<int>(item % D), which = static_cast<int>(item / D % 2);
  const int64_t row = item / D / 2;
  const int hk = static_cast<int>(row % p.Hk), j = static_cast<int>(row / p.Hk % keys), b = static_cast<int>(row / p.Hk / keys);
  const float* part = p.part + ((static_cast<int64_t>(b) * p.Hk + hk) * p.nblk + j / 32) * p.nchunk * 64 * D +
                      (which * 32 + j % 32) * D + d;
  float v = 0.f;
  for (int c = 0; c < p.nchunk; ++c) v += part[static_cast<int64_t>(c) * 64 * D];
  T* dst = (which ? p.dv : p.dk) + ((static_cast<int64_t>(b) * p.Lk + j) * p.Hk + hk) * D + d;
  *dst = from_f32<T>(which ? v : v * p.scale);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int64_t kMostL = 1 << 30;

struct SwaSizes {
  int64_t nq, nk;  // elements of q and of k
  int es;
};

int swa_sizes(int64_t Bs, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks,
              double scale, int dtype, SwaSizes* z) {
  int64_t t, bytes;
  if (Lq < 0 || Lk < 0 || Lq > kMostL || Lk > kMostL || Hk < 1 || Hq < 1 || Hq % Hk || window < 1 || sinks < 0)
    return SSM_ERR_DIM;
  if (!mul_nn(Bs, Lq, &t) || !mul_nn(t, Hq, &t) || !mul_nn(t, D, &z->nq) || !mul_nn(z->nq, 8, &bytes)) return SSM_ERR_DIM;
  if (!mul_nn(Bs, Lk, &t) || !mul_nn(t, Hk, &t) || !mul_nn(t, D, &z->nk) || !mul_nn(z->nk, 8, &bytes)) return SSM_ERR_DIM;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return SSM_ERR_UNSUPPORTED;
  if (!(scale > 0) || scale > 1e30) return SSM_ERR_ARG;
  z->es = dtype == SSM_F32 ? 4 : 2;
  // workgroups of the largest launch
  int64_t w;
  if (!mul_nn(Bs * Hq, (std::max(Lq, Lk) + 31) / 32, &w) || w > kMaxGrid) return SSM_ERR_DIM;
  return SSM_OK;
}

// A tile's rows lie within 32-bit offsets of its first.
bool token_ok(const ssm_strides& s, int es) { return s.token * es <= (1 << 25); }

template <typename T>
SwaArgs<T> swa_args(const void* q, ssm_strides qs, const void* k, ssm_strides ks, const void* v, ssm_strides vs,
                    const int32_t* lens, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hk, int64_t window, int64_t sinks,
                    double scale) {
  SwaArgs<T> a{};
  a.q = static_cast<const T*>(q), a.k = static_cast<const T*>(k), a.v = static_cast<const T*>(v);
  a.qs = qs, a.ks = ks, a.vs = vs, a.lens = lens;
  a.Lq = static_cast<int>(Lq), a.Lk = static_cast<int>(Lk), a.Hq = static_cast<int>(Hq), a.Hk = static_cast<int>(Hk);
  a.G = static_cast<int>(Hq / Hk);
  a.W = static_cast<int>(std::min(window, kMostL)), a.S = static_cast<int>(std::min(sinks, kMostL));
  a.scale = static_cast<float>(scale);
  return a;
}

// Workgroups that share a block of 32 sinks: about two for each compute unit
// over all blocks, at least eight query tiles each.
int sink_chunks(int64_t Bs, int64_t Lq, int64_t Hq, int64_t Hk, int64_t blocks) {
  const int64_t tiles = (Lq + 63) / 64 * (Hq / Hk);
  const int64_t want = 512 / std::max<int64_t>(1, Bs * Hk * blocks);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, tiles / 8)));
}

int64_t sink_blocks(int64_t sinks, int64_t Lk) { return (std::min(sinks, Lk) + 31) / 32; }

int64_t stat_bytes(int64_t Bs, int64_t Lq, int64_t Hq) { return (Bs * Lq * Hq * 4 + 15) & ~int64_t(15); }

}  // namespace

extern "C" int ssm_swa_fwd(const void* q, const ssm_strides* qs, const void* k, const ssm_strides* ks, const void* v,
                           const ssm_strides* vs, const int32_t* lens, double scale, void* o, float* lse, int64_t Bs,
                           int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks,
                           int dtype, void* stream) {
  SwaSizes z;
  int rc = swa_sizes(Bs, Lq, Lk, Hq, Hk, D, window, sinks, scale, dtype, &z);
  if (rc != SSM_OK) return rc;
  ssm_strides sq, sk, sv;
  int64_t bq, bk, bv;
  if ((rc = strided(qs, Bs, Lq, Hq, D, z.es, &sq, &bq)) != SSM_OK) return rc;
  if ((rc = strided(ks, Bs, Lk, Hk, D, z.es, &sk, &bk)) != SSM_OK) return rc;
  if ((rc = strided(vs, Bs, Lk, Hk, D, z.es, &sv, &bv)) != SSM_OK) return rc;
  if (!token_ok(sq, z.es) || !token_ok(sk, z.es) || !token_ok(sv, z.es)) return SSM_ERR_UNSUPPORTED;
  const Buf bufs[] = {{q, bq, true, false}, {k, bk, true, false}, {v, bv, true, false}, {lens, Bs * 4, false, false, 4},
                      {o, z.nq * z.es, true, true}, {lse, Bs * Hq * Lq * 4, false, true}};
  if ((rc = check_bufs(bufs, 6)) != SSM_OK) return rc;
  if (z.nq == 0) return SSM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    SwaArgs<T> a = swa_args<T>(q, sq, k, sk, v, sv, lens, Lq, Lk, Hq, Hk, window, sinks, scale);
    a.out = static_cast<T*>(o), a.lse = lse;
    a.nblk = static_cast<int>((Lq + kOwn - 1) / kOwn), a.nwork = static_cast<int>(Bs * Hq * a.nblk);
    if (D == 64)
      hipLaunchKernelGGL((swa_fwd_kernel<T, 64>), dim3(a.nwork), dim3(kNT), 0, st, a);
    else
      hipLaunchKernelGGL((swa_fwd_kernel<T, 128>), dim3(a.nwork), dim3(kNT), 0, st, a);
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
  };
  return dtype == SSM_F32 ? go(float{}) : go(uint16_t{});
}

extern "C" size_t ssm_swa_bwd_workspace_bytes(int64_t Bs, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hk, int64_t D,
                                              int64_t sinks, int dtype) {
  SwaSizes z;
  if (swa_sizes(Bs, Lq, Lk, Hq, Hk, D, 1, sinks, 1.0, dtype, &z) != SSM_OK || z.nq == 0 || z.nk == 0) return 0;
  const int64_t nb = sink_blocks(sinks, Lk);
  const int64_t part = nb ? Bs * Hk * nb * sink_chunks(Bs, Lq, Hq, Hk, nb) * 64 * D * 4 : 0;
  return static_cast<size_t>(stat_bytes(Bs, Lq, Hq) + part);
}

extern "C" int ssm_swa_bwd(const void* q, const ssm_strides* qs, const void* k, const ssm_strides* ks, const void* v,
                           const ssm_strides* vs, const int32_t* lens, double scale, const void* o, const float* lse,
                           const void* dout, void* dq, void* dk, void* dv, int64_t Bs, int64_t Lq, int64_t Lk,
                           int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  SwaSizes z;
  int rc = swa_sizes(Bs, Lq, Lk, Hq, Hk, D, window, sinks, scale, dtype, &z);
  if (rc != SSM_OK) return rc;
  ssm_strides sq, sk, sv;
  int64_t bq, bk, bv;
  if ((rc = strided(qs, Bs, Lq, Hq, D, z.es, &sq, &bq)) != SSM_OK) return rc;
  if ((rc = strided(ks, Bs, Lk, Hk, D, z.es, &sk, &bk)) != SSM_OK) return rc;
  if ((rc = strided(vs, Bs, Lk, Hk, D, z.es, &sv, &bv)) != SSM_OK) return rc;
  if (!token_ok(sq, z.es) || !token_ok(sk, z.es) || !token_ok(sv, z.es) || Hq * D * z.es > (1 << 25))
    return SSM_ERR_UNSUPPORTED;
  const size_t need = ssm_swa_bwd_workspace_bytes(Bs, Lq, Lk, Hq, Hk, D, sinks, dtype);
  const int64_t oq = z.nq * z.es, ok = z.nk * z.es;
  const Buf bufs[] = {{q, bq, true, false}, {k, bk, true, false}, {v, bv, true, false}, {lens, Bs * 4, false, false, 4},
                      {o, oq, true, false}, {lse, Bs * Hq * Lq * 4, true, false}, {dout, oq, true, false},
                      {dq, oq, true, true}, {dk, ok, true, true}, {dv, ok, true, true},
                      {workspace, static_cast<int64_t>(need), false, true}};
  if ((rc = check_bufs(bufs, 11)) != SSM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (z.nq == 0 || z.nk == 0)  // no pairs (an odd count of bfloat16 pairs cannot occur: D is even)
    return fill_async(dq, nullptr, oq, st) && fill_async(dk, nullptr, ok, st) && fill_async(dv, nullptr, ok, st)
               ? SSM_OK
               : SSM_ERR_LAUNCH;
  if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
  auto go = [&](auto tag, auto dim) {
    using T = decltype(tag);
    constexpr int DD = decltype(dim)::value;
    SwaArgs<T> a = swa_args<T>(q, sq, k, sk, v, sv, lens, Lq, Lk, Hq, Hk, window, sinks, scale);
    a.o = static_cast<const T*>(o), a.dout = static_cast<const T*>(dout), a.lse = const_cast<float*>(lse);
    a.dq = static_cast<T*>(dq), a.dk = static_cast<T*>(dk), a.dv = static_cast<T*>(dv);
    a.delta = static_cast<float*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + stat_bytes(Bs, Lq, Hq));
    a.nblk = static_cast<int>((Lq + kOwn - 1) / kOwn), a.nwork = static_cast<int>(Bs * Hq * a.nblk);
    hipLaunchKernelGGL((swa_dq_kernel<T, DD>), dim3(a.nwork), dim3(kNT), 0, st, a);
    if (sinks < Lk) {
      a.nblk = static_cast<int>((Lk + kOwn - 1) / kOwn), a.nwork = static_cast<int>(Bs * Hk * a.nblk);
      hipLaunchKernelGGL((swa_dkdv_kernel<T, DD, false>), dim3(a.nwork), dim3(kNT), 0, st, a);
    }
    if (sinks > 0) {
      const int64_t nb = sink_blocks(sinks, Lk);
      a.nblk = static_cast<int>(nb), a.nchunk = sink_chunks(Bs, Lq, Hq, Hk, nb);
      a.nwork = static_cast<int>(Bs * Hk * nb * a.nchunk);
      hipLaunchKernelGGL((swa_dkdv_kernel<T, DD, true>), dim3(a.nwork), dim3(kNT), 0, st, a);
      const int64_t items = Bs * std::min(sinks, Lk) * Hk * 2 * D;
      hipLaunchKernelGGL((swa_sink_join_kernel<T>), dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, st,
                         a, static_cast<int>(Bs), static_cast<int>(D));
    }
    return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (dtype == SSM_F32) return D == 64 ? go(float{}, D64{}) : go(float{}, D128{});
  return D == 64 ? go(uint16_t{}, D64{}) : go(uint16_t{}, D128{});
}
