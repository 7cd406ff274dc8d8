// Gated linear recurrence (ssm_glr_* of ssm_hybrid.h) for gfx950.
//
//   r = sigmoid(gr), i = sigmoid(gi), la = A r, a = e^la, s = sqrt(max(0, 1 - e^(2 la)))
//   h_t = a_t h_{t-1} + s_t i_t x_t,   y_t = h_t
//
// A run of steps takes the state through an affine map h -> P h + H. Forward,
// one pass over the data: a wave forms the map of 16 steps and keeps every
// step's part of it in registers, its workgroup joins eight of them to a chunk
// of 128 steps, and chunks pass maps and states on through the workspace (see
// Handoff); then every step's state follows from the one entering the wave.
// Backward: the maps of the adjoint, chunk by chunk, their fold along the
// sequence, then every chunk again from its entering adjoint, in blocks of 16
// steps whose states start from the forward's checkpoints.
#include <type_traits>

#include "hybrid_common.h"

namespace {

constexpr int kCk = SSM_GLR_CKPT_STEPS;

// ---------------------------------------------------------------------------
// VEC-wide element access
// ---------------------------------------------------------------------------
// A row's address kept in scalar registers: with a lane's 32-bit offset added
// last, an access takes one vector register for its address and not two for
// every row. (Device memory: the cast keeps the accesses global.)
#define SSM_GLOBAL __attribute__((address_space(1)))
template <typename P>
__device__ __forceinline__ SSM_GLOBAL P* scalar(P* p) {
  SSM_GLOBAL P* g = (SSM_GLOBAL P*)p;
  asm("" : "+s"(g));
  return g;
}

// the loaded bits, widened when they are used (a wave can then have many loads
// in flight). The sequences' elements are touched once in a launch, so their
// accesses are nontemporal: 4x8192x5120 bf16 forward and backward 949 -> 887 us.
template <typename T, int VEC>
struct RawOf {
  using type = T;
};
template <>
struct RawOf<uint16_t, 2> {
  using type = uint32_t;
};
template <typename T, int VEC>
__device__ __forceinline__ typename RawOf<T, VEC>::type load_raw(const SSM_GLOBAL T* p) {
  return __builtin_nontemporal_load((const SSM_GLOBAL typename RawOf<T, VEC>::type*)p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_raw(SSM_GLOBAL T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 2 && sizeof(T) == 2) {
    __builtin_nontemporal_store(pack_bf16(v[0], v[1]), (SSM_GLOBAL uint32_t*)p);
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c) __builtin_nontemporal_store(from_f32<T>(v[c]), p + c);
  }
}
__device__ __forceinline__ void widen_pair(uint32_t r, float (&v)[2]) {
  v[0] = __uint_as_float(r << 16), v[1] = __uint_as_float(r & 0xffff0000u);
}
template <typename T, int VEC>
__device__ __forceinline__ void widen(typename RawOf<T, VEC>::type r, float (&v)[VEC]) {
  if constexpr (VEC == 2) {
    widen_pair(r, v);
  } else {
    v[0] = to_f32(r);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 f = Vec4<T>::load(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c) v[c] = to_f32(p[c]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    Vec4<T>::store(p, make_float4(v[0], v[1], v[2], v[3]));
  } else if constexpr (VEC == 2 && sizeof(T) == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c) p[c] = from_f32<T>(v[c]);
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
  int64_t Bs, L, ED, ckrows;
  // forward: the hand-off
  unsigned* hdr;        // tickets, 64 bytes apart
  unsigned* flag;       // [chunk][group]: the chunk's map is there
  uint64_t* state;      // [span][group][channel]: the state entering the span, and 1 once it is there
  uint64_t* map;        // [chunk][group][channel]: (P, H)
  int64_t nchunks, ngroups, ncg;  // ncg: groups of 64 VEC channels of a row; ngroups = Bs ncg
  unsigned spin_limit;
  // backward
  float2* agg;     // (Bs, nchunks, ED): (P, H) of each chunk
  float* enter;    // (Bs, nchunks, ED): the adjoint entering each chunk
  float* dA_part;  // (Bs, nchunks, ED)
  int64_t steps;
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Handoff between the chunks of a channel group. Chunks are dealt out by
// tickets, from eight queues that hold an eighth of the groups each, chunk k of
// all of them before any chunk k + 1; a workgroup takes from the queue of its
// XCD first. So whatever a chunk waits for has been taken by a workgroup that
// runs. (With one queue the workgroups of a full device queue up for its word:
// 8x1024x1536 float32 50 us instead of 46.) kSpan chunks make a
// span. A chunk publishes its map at once (waiting for nothing), then needs
// the maps of the chunks before it in its span and the state entering the
// span, which the last chunk of the span before publishes. A chain of states
// through all chunks would cost a trip between compute units each (about 2
// us, 2 ms over 1024 chunks); here the chain has a step a span, and the maps
// read in between are kSpan / 2 of 8 bytes a channel on average beside the
// chunk's 128 steps. The order of every sum is fixed by the chunk's place.
//   Maps, states and flags are written and read by agent-scope atomics, which
// go past the caches that are not shared. A map's publisher waits for its
// stores (vmcnt(0)) before it raises the flag; a state, on the chain, carries
// its flag in its own 8 bytes, which spares it that wait and a second trip.
// Waits are bounded: if one ever gives up, the chunk takes NaN as its entering
// state.
constexpr int kSpan = 16;
constexpr int kFwdWaves = 8, kChunk = kFwdWaves * kCk;

__device__ __forceinline__ void publish_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void put_flag(unsigned* f) {
  __hip_atomic_store(f, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits until there(), asked by every lane, holds for all of them.
template <typename F>
__device__ __forceinline__ bool wait_for(F there, unsigned limit) {
  bool done = false;
  for (unsigned it = 0;; ++it) {
    if (!done) done = there();
    if (__all(done)) break;
    if (it >= limit) return false;
    __builtin_amdgcn_s_sleep(1);
  }
  asm volatile("" ::: "memory");
  return true;
}

// body(true) for a whole block of kCk steps, body(false) for the sequence's last.
template <typename F>
__device__ __forceinline__ void run_steps(int m, F body) {
  if (m == kCk)
    body(std::integral_constant<bool, true>{});
  else
    body(std::integral_constant<bool, false>{});
}

// Chunk, group, batch row and channel group of a work item. (A division runs on
// the vector unit; the results go back to scalars so that addresses do too.)
template <typename T>
__device__ __forceinline__ void locate(const GlrArgs<T>& p, unsigned item, int64_t* k, int64_t* group, int64_t* b,
                                       int64_t* cg) {
  const unsigned ng = static_cast<unsigned>(p.ngroups), nc = static_cast<unsigned>(p.ncg);
  const unsigned kk = __builtin_amdgcn_readfirstlane(item / ng), g = item - kk * ng;
  const unsigned bb = __builtin_amdgcn_readfirstlane(g / nc);
  *k = kk, *group = g, *b = bb, *cg = g - bb * nc;
}

constexpr int kQueues = 8, kTicketWords = 16;
// Chunk and group of the next ticket; (-1, -1) if every queue is empty.
template <typename T>
__device__ __forceinline__ void take_chunk(const GlrArgs<T>& p, int (&out)[2]) {
  // XCC_ID hardware register (bits 3:0): the XCD this wave runs on
  const unsigned xcc = static_cast<unsigned>(__builtin_amdgcn_s_getreg((3 << 11) | (0 << 6) | 20));
  const unsigned ng = static_cast<unsigned>(p.ngroups);
  out[0] = out[1] = -1;
  for (unsigned d = 0; d < kQueues; ++d) {
    const unsigned q = (xcc + d) % kQueues;
    const unsigned g0 = static_cast<unsigned>(static_cast<uint64_t>(q) * ng / kQueues);
    const unsigned n = static_cast<unsigned>(static_cast<uint64_t>(q + 1) * ng / kQueues) - g0;
    if (n == 0) continue;
    const unsigned j = __hip_atomic_fetch_add(p.hdr + q * kTicketWords, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (j < n * static_cast<unsigned>(p.nchunks)) {
      out[0] = static_cast<int>(j / n), out[1] = static_cast<int>(g0 + j % n);
      return;
    }
  }
}

// What the loads cannot do without: 3 inputs and 1 output of an element;
// the gates cost about 25 vector and 6 transcendental instructions each.
template <typename T, int VEC>
__global__ __launch_bounds__(64 * kFwdWaves, 4) void glr_fwd_kernel(const GlrArgs<T> p) {
  __shared__ float2 maps[kFwdWaves][64][VEC];
  __shared__ float entering[64][VEC];
  __shared__ int s_taken[2];
  using Raw = typename RawOf<T, VEC>::type;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t k = 0, group = blockIdx.x;
  if (p.nchunks > 1) {
    if (threadIdx.x == 0) take_chunk(p, s_taken);
    __syncthreads();
    k = __builtin_amdgcn_readfirstlane(s_taken[0]);
    group = __builtin_amdgcn_readfirstlane(s_taken[1]);
    if (k < 0) return;  // (cannot happen: as many workgroups as chunks)
  }
  const int64_t b = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(group) / static_cast<unsigned>(p.ncg));
  const int64_t cg = group - b * p.ncg;
  const int64_t e = cg * 64 * VEC + lane * VEC;
  const bool ok = e < p.ED;  // (ED is a multiple of VEC)
  const unsigned lo = ok ? lane * VEC : 0;  // the lane's channel after the group's first
  const int64_t t0 = k * kChunk + wave * kCk, left = p.L - t0;
  const int m = left < 0 ? 0 : left < kCk ? static_cast<int>(left) : kCk;  // steps of this wave
  const int64_t at = (b * p.L + t0) * p.ED + cg * 64 * VEC;

  float P[VEC], H[VEC], Pt[kCk][VEC], Ht[kCk][VEC];
  run_steps(m, [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    Raw xr[kCk], rr[kCk], ir[kCk];
#pragma unroll
    for (int t = 0; t < kCk; ++t)
      if (FULL || t < m) {
        xr[t] = load_raw<T, VEC>(scalar(p.x + at + t * p.ED) + lo);
        rr[t] = load_raw<T, VEC>(scalar(p.gr + at + t * p.ED) + lo);
        ir[t] = load_raw<T, VEC>(scalar(p.gi + at + t * p.ED) + lo);
      }
    float A2[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) A2[c] = p.A[cg * 64 * VEC + lo + c] * kLog2e, P[c] = 1.f, H[c] = 0.f;
#pragma unroll
    for (int t = 0; t < kCk; ++t)
      if (FULL || t < m) {
        float x[VEC], gr[VEC], gi[VEC];
        widen<T, VEC>(xr[t], x);
        widen<T, VEC>(rr[t], gr);
        widen<T, VEC>(ir[t], gi);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const Gates g = gates(gr[c], gi[c], A2[c]);
          P[c] *= g.a;
          H[c] = __builtin_fmaf(g.a, H[c], g.s * g.i * x[c]);
          Pt[t][c] = P[c];
          Ht[t][c] = H[c];
        }
      }
  });
#pragma unroll
  for (int c = 0; c < VEC; ++c) maps[wave][lane][c] = make_float2(P[c], H[c]);
  __syncthreads();
  if (wave == 0) {
    float h[VEC];
    float cp[VEC], ch[VEC];  // the chunk's map
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      cp[c] = 1.f, ch[c] = 0.f;
#pragma unroll
      for (int w = 0; w < kFwdWaves; ++w) {
        const float2 v = maps[w][lane][c];
        cp[c] *= v.x;
        ch[c] = __builtin_fmaf(v.x, ch[c], v.y);
      }
      h[c] = p.h0 && ok ? p.h0[b * p.ED + e + c] : 0.f;
    }
    if (p.nchunks > 1) {
      const int64_t span = k / kSpan, cw = 64 * VEC, mine = lane * VEC;
      const int place = static_cast<int>(k % kSpan);
      const bool more = k + 1 < p.nchunks;
      if (more && place < kSpan - 1) {
        uint64_t* to = p.map + (k * p.ngroups + group) * cw + mine;
#pragma unroll
        for (int c = 0; c < VEC; ++c)
          __hip_atomic_store(to + c, __builtin_bit_cast(uint64_t, make_float2(cp[c], ch[c])), __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
        publish_fence();
        if (lane == 0) put_flag(p.flag + k * p.ngroups + group);
      }
      // the maps before this chunk in its span, joined
      unsigned* flag = p.flag + (span * kSpan + lane) * p.ngroups + group;
      bool good = wait_for(
          [&] { return lane >= place || __hip_atomic_load(flag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0; },
          p.spin_limit);
      float bp[VEC], bh[VEC];
#pragma unroll
      for (int c = 0; c < VEC; ++c) bp[c] = 1.f, bh[c] = 0.f;
#pragma unroll 5
      for (int j = 0; j < place; ++j) {
        uint64_t* from = p.map + ((span * kSpan + j) * p.ngroups + group) * cw + mine;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float2 v = __builtin_bit_cast(float2, __hip_atomic_load(from + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
          bp[c] *= v.x;
          bh[c] = __builtin_fmaf(v.x, bh[c], v.y);
        }
      }
      if (span > 0) {
        uint64_t* from = p.state + (span * p.ngroups + group) * cw + mine;
        good = wait_for(
                   [&] {
                     bool all = true;
#pragma unroll
                     for (int c = 0; c < VEC; ++c) {
                       const uint64_t v = __hip_atomic_load(from + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                       h[c] = __uint_as_float(static_cast<unsigned>(v));
                       all = all && (v >> 32) != 0;
                     }
                     return all;
                   },
                   p.spin_limit) &&
               good;
      }
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = good ? __builtin_fmaf(bp[c], h[c], bh[c]) : __builtin_nanf("");
      if (more && place == kSpan - 1) {
        uint64_t* to = p.state + ((span + 1) * p.ngroups + group) * cw + mine;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const uint64_t v = __float_as_uint(__builtin_fmaf(cp[c], h[c], ch[c]));
          __hip_atomic_store(to + c, v | (uint64_t(1) << 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      entering[lane][c] = h[c];
      if (p.h_last && ok && k + 1 == p.nchunks) p.h_last[b * p.ED + e + c] = __builtin_fmaf(cp[c], h[c], ch[c]);
    }
  }
  __syncthreads();
  if (m == 0 || !ok) return;
  float h[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    h[c] = entering[lane][c];
#pragma unroll
    for (int w = 0; w < kFwdWaves - 1; ++w)
      if (w < wave) {
        const float2 v = maps[w][lane][c];
        h[c] = __builtin_fmaf(v.x, h[c], v.y);
      }
  }
  if (p.ckpt) store_vec<float, VEC>(p.ckpt + (b * p.ckrows + t0 / kCk) * p.ED + e, h);
  run_steps(m, [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
#pragma unroll
    for (int t = 0; t < kCk; ++t)
      if (FULL || t < m) {
        float y[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) y[c] = __builtin_fmaf(Pt[t][c], h[c], Ht[t][c]);
        store_raw<T, VEC>(scalar(p.y + at + t * p.ED) + lo, y);
      }
  });
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// enter[k] = the adjoint entering chunk k from the chunks after it and `init`.
// 16 channels a workgroup; a channel's chunks are shared by 16 threads, which
// join the maps of a run each, then walk their run from its entering adjoint.
__global__ __launch_bounds__(256) void glr_join_kernel(const float2* agg, const float* init, float* enter,
                                                       int64_t nchunks, int64_t ED, int64_t ncol) {
  __shared__ float2 runs[16][16];
  const int ce = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int64_t b = blockIdx.x / ncol, e = (blockIdx.x % ncol) * 16 + ce;
  const bool ok = e < ED;
  // run `seg` of the reversed order: chunks hi - 1 down to lo
  const int64_t hi = nchunks - nchunks * seg / 16, lo = nchunks - nchunks * (seg + 1) / 16;
  const int64_t at = b * nchunks * ED + e;
  float P = 1.f, H = 0.f;
  if (ok)
#pragma unroll 8
    for (int64_t k = hi - 1; k >= lo; --k) {
      const float2 m = agg[at + k * ED];
      P *= m.x;
      H = __builtin_fmaf(m.x, H, m.y);
    }
  runs[seg][ce] = make_float2(P, H);
  __syncthreads();
  if (!ok) return;
  float g = init ? init[b * ED + e] : 0.f;
  for (int s = 0; s < seg; ++s) g = __builtin_fmaf(runs[s][ce].x, g, runs[s][ce].y);
#pragma unroll 8
  for (int64_t k = hi - 1; k >= lo; --k) {
    const float2 m = agg[at + k * ED];
    enter[at + k * ED] = g;
    g = __builtin_fmaf(m.x, g, m.y);
  }
}

// A wave's chunk and its group of 64 VEC channels; false past the end.
template <typename T, int VEC>
struct BwdPlace {
  int64_t b, k, e0, t0, n;  // first channel, first step, steps
  unsigned lo;              // the lane's channel after e0
  bool ok;
  __device__ __forceinline__ bool find(const GlrArgs<T>& p) {
    const int lane = threadIdx.x & 63;
    const unsigned item = blockIdx.x * 4u + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (item >= p.ngroups * p.nchunks) return false;
    int64_t group, cg;
    locate(p, item, &k, &group, &b, &cg);
    e0 = cg * 64 * VEC;
    ok = e0 + lane * VEC < p.ED;
    lo = ok ? lane * VEC : 0;
    t0 = k * p.steps;
    n = p.L - t0 < p.steps ? p.L - t0 : p.steps;
    return true;
  }
  // of an array (Bs, nchunks, ED)
  __device__ __forceinline__ int64_t slot(const GlrArgs<T>& p) const { return (b * p.nchunks + k) * p.ED + e0 + lo; }
};

// The adjoint's aggregate of a chunk: G -> P G + H with G entering after the
// chunk's last step and leaving before its first (a_t applied).
template <typename T, int VEC>
__global__ __launch_bounds__(256) void glr_bwd_agg_kernel(const GlrArgs<T> p) {
  using Raw = typename RawOf<T, VEC>::type;
  BwdPlace<T, VEC> w;
  if (!w.find(p)) return;
  float A2[VEC], P[VEC], H[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) A2[c] = p.A[w.e0 + w.lo + c] * kLog2e, P[c] = 1.f, H[c] = 0.f;
  for (int64_t blk = (w.n + kCk - 1) / kCk - 1; blk >= 0; --blk) {
    const int m = static_cast<int>(w.n - blk * kCk < kCk ? w.n - blk * kCk : kCk);
    const int64_t at = (w.b * p.L + w.t0 + blk * kCk) * p.ED + w.e0;
    run_steps(m, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      Raw rr[kCk], dr[kCk];
#pragma unroll
      for (int t = kCk - 1; t >= 0; --t)
        if (FULL || t < m) {
          rr[t] = load_raw<T, VEC>(scalar(p.gr + at + t * p.ED) + w.lo);
          dr[t] = load_raw<T, VEC>(scalar(p.dy + at + t * p.ED) + w.lo);
        }
#pragma unroll
      for (int t = kCk - 1; t >= 0; --t)
        if (FULL || t < m) {
          float gr[VEC], dy[VEC];
          widen<T, VEC>(rr[t], gr);
          widen<T, VEC>(dr[t], dy);
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            const float a = __builtin_amdgcn_exp2f(A2[c] * sigmoid_fast(gr[c]));
            P[c] *= a;
            H[c] = a * (H[c] + dy[c]);
          }
        }
    });
  }
  if (w.ok)
#pragma unroll
    for (int c = 0; c < VEC; ++c) p.agg[w.slot(p) + c] = make_float2(P[c], H[c]);
}

// Blocks of kCk steps in reverse order. A block's gates are formed once, going
// forwards from its checkpoint; what the way back needs of a step stays in
// registers: a and the factors of g in dx, dgi, dla r and dgr.
template <typename T, int VEC>
__global__ __launch_bounds__(256, 2) void glr_bwd_apply_kernel(const GlrArgs<T> p) {
  using Raw = typename RawOf<T, VEC>::type;
  BwdPlace<T, VEC> w;
  if (!w.find(p)) return;
  float A[VEC], G[VEC], dA[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    A[c] = p.A[w.e0 + w.lo + c];
    dA[c] = 0.f;
    G[c] = p.enter[w.slot(p) + c];
  }
  for (int64_t blk = (w.n + kCk - 1) / kCk - 1; blk >= 0; --blk) {
    const int64_t tb = w.t0 + blk * kCk;
    const int m = static_cast<int>(w.n - blk * kCk < kCk ? w.n - blk * kCk : kCk);
    const int64_t at = (w.b * p.L + tb) * p.ED + w.e0;
    run_steps(m, [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      Raw xr[kCk], rr[kCk], ir[kCk], dr[kCk];
      float h[VEC];
      load_vec<float, VEC>(p.ckpt + (w.b * p.ckrows + tb / kCk) * p.ED + w.e0 + w.lo, h);
#pragma unroll
      for (int t = 0; t < kCk; ++t)
        if (FULL || t < m) {
          xr[t] = load_raw<T, VEC>(scalar(p.x + at + t * p.ED) + w.lo);
          rr[t] = load_raw<T, VEC>(scalar(p.gr + at + t * p.ED) + w.lo);
          ir[t] = load_raw<T, VEC>(scalar(p.gi + at + t * p.ED) + w.lo);
        }
#pragma unroll
      for (int t = kCk - 1; t >= 0; --t)
        if (FULL || t < m) dr[t] = load_raw<T, VEC>(scalar(p.dy + at + t * p.ED) + w.lo);
      float fa[kCk][VEC], fx[kCk][VEC], fi[kCk][VEC], fl[kCk][VEC], fr[kCk][VEC];
#pragma unroll
      for (int t = 0; t < kCk; ++t)
        if (FULL || t < m) {
          float x[VEC], gr[VEC], gi[VEC];
          widen<T, VEC>(xr[t], x);
          widen<T, VEC>(rr[t], gr);
          widen<T, VEC>(ir[t], gi);
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            const Gates q = gates(gr[c], gi[c], A[c] * kLog2e);
            const float ix = q.i * x[c], ah = q.a * h[c];
            const float root = q.s > 0.f ? q.a * q.a * rcp_fast(q.s) * ix : 0.f;
            fa[t][c] = q.a;
            fx[t][c] = q.s * q.i;
            fi[t][c] = q.s * ix * (1.f - q.i);
            fl[t][c] = (ah - root) * q.r;
            fr[t][c] = A[c] * (1.f - q.r);
            h[c] = __builtin_fmaf(q.s, ix, ah);
          }
        }
#pragma unroll
      for (int t = kCk - 1; t >= 0; --t)
        if (FULL || t < m) {
          const int64_t o = at + t * p.ED;
          float dy[VEC], dx[VEC], dgr[VEC], dgi[VEC];
          widen<T, VEC>(dr[t], dy);
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            const float g = G[c] + dy[c];
            const float dlr = g * fl[t][c];
            dx[c] = g * fx[t][c];
            dgi[c] = g * fi[t][c];
            dgr[c] = dlr * fr[t][c];
            dA[c] += dlr;
            G[c] = fa[t][c] * g;
          }
          if (w.ok) {
            store_raw<T, VEC>(scalar(p.dx + o) + w.lo, dx);
            store_raw<T, VEC>(scalar(p.dgr + o) + w.lo, dgr);
            store_raw<T, VEC>(scalar(p.dgi + o) + w.lo, dgi);
          }
        }
    });
  }
  if (!w.ok) return;
  if (p.dh0 && w.k == 0) store_vec<float, VEC>(p.dh0 + w.b * p.ED + w.e0 + w.lo, G);
#pragma unroll
  for (int c = 0; c < VEC; ++c) p.dA_part[w.slot(p) + c] = dA[c];
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
// VEC: 4 bytes a lane (256 a wave and row), or single channels where a pair
// would straddle the row's end.
int fwd_vec(int64_t ED, int dtype) { return dtype == SSM_BF16 && ED % 2 == 0 ? 2 : 1; }

struct FwdPlan {
  int64_t nchunks, nspans, ncg, ngroups, cw;
  int64_t flag, state, map, bytes;  // workspace offsets; what lies before `map` starts as zero
};

FwdPlan fwd_plan(int64_t Bs, int64_t L, int64_t ED, int dtype) {
  FwdPlan f{};
  f.cw = 64 * fwd_vec(ED, dtype);
  f.nchunks = (L + kChunk - 1) / kChunk;
  f.nspans = (f.nchunks + kSpan - 1) / kSpan;
  f.ncg = (ED + f.cw - 1) / f.cw;
  f.ngroups = Bs * f.ncg;
  if (f.nchunks <= 1) return f;
  const auto up = [](int64_t v) { return (v + 255) & ~int64_t(255); };
  f.flag = kQueues * kTicketWords * 4;
  f.state = f.flag + up(f.nchunks * f.ngroups * 4);
  f.map = f.state + f.nspans * f.ngroups * f.cw * 8;
  f.bytes = f.map + f.nchunks * f.ngroups * f.cw * 8;
  return f;
}

struct BwdPlan {
  int64_t nchunks, steps, ckrows;
};

// Chunks are whole blocks of kCk steps, as long as there are at least about
// eight waves of threads per CU (256 CUs), at most 128 steps.
BwdPlan bwd_plan(int64_t Bs, int64_t L, int64_t ED, int dtype) {
  const int64_t cw = 64 * fwd_vec(ED, dtype), waves = Bs * ((ED + cw - 1) / cw);
  int64_t steps = 128;
  while (steps > kCk && waves * ((L + steps - 1) / steps) < 8 * 256) steps /= 2;
  return BwdPlan{(L + steps - 1) / steps, steps, (L + kCk - 1) / kCk};
}

int glr_sizes(int64_t Bs, int64_t L, int64_t ED, int dtype, int64_t* n, int64_t* nck) {
  int64_t c, rows = L >= 0 ? (L + kCk - 1) / kCk : -1, bytes;
  if (!mul_nn(Bs, ED, &c) || !mul_nn(c, L, n) || !mul_nn(*n, 8, &bytes)) return SSM_ERR_DIM;
  // (the backward's workspace holds 16 bytes a chunk and channel)
  if (!mul_nn(c + 64 * Bs, rows, nck) || !mul_nn(*nck, 32, &bytes) || !mul_nn(c, rows, nck)) return SSM_ERR_DIM;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t glr_agg_bytes(const BwdPlan& pl, int64_t c) { return (static_cast<size_t>(pl.nchunks * c) * 8 + 15) & ~size_t(15); }
size_t glr_enter_bytes(const BwdPlan& pl, int64_t c) { return (static_cast<size_t>(pl.nchunks * c) * 4 + 15) & ~size_t(15); }

template <typename T, int VEC>
int launch_fwd(const GlrArgs<T>& a, const FwdPlan& f, void* ws, hipStream_t st) {
  if (f.nchunks * f.ngroups > kMaxGrid) return SSM_ERR_DIM;
  if (f.nchunks > 1)
    hipLaunchKernelGGL(zero_words_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((f.map / 4 + 255) / 256, 1024))),
                       dim3(256), 0, st, static_cast<unsigned*>(ws), f.map / 4);
  hipLaunchKernelGGL((glr_fwd_kernel<T, VEC>), dim3(static_cast<unsigned>(f.nchunks * f.ngroups)), dim3(64 * kFwdWaves),
                     0, st, a);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

template <typename T, int VEC>
int launch_bwd(GlrArgs<T> a, float* dA, hipStream_t st) {
  a.ncg = (a.ED + 64 * VEC - 1) / (64 * VEC), a.ngroups = a.Bs * a.ncg;
  const int64_t blocks = (a.ngroups * a.nchunks + 3) / 4, ncol = (a.ED + 15) / 16;
  if (a.ngroups * a.nchunks > kMaxGrid || a.Bs * ncol > kMaxGrid) return SSM_ERR_DIM;
  const dim3 grid(static_cast<unsigned>(blocks));
  hipLaunchKernelGGL((glr_bwd_agg_kernel<T, VEC>), grid, dim3(256), 0, st, a);
  hipLaunchKernelGGL(glr_join_kernel, dim3(static_cast<unsigned>(a.Bs * ncol)), dim3(256), 0, st, a.agg, a.dh_last,
                     a.enter, a.nchunks, a.ED, ncol);
  hipLaunchKernelGGL((glr_bwd_apply_kernel<T, VEC>), grid, dim3(256), 0, st, a);
  hipLaunchKernelGGL(sum_rows_kernel, dim3(static_cast<unsigned>(ncol)), dim3(1024), 0, st, a.dA_part, dA,
                     a.Bs * a.nchunks, a.ED);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH;
}

template <typename T>
int run_fwd(const void* x, const void* gr, const void* gi, const float* A, const float* h0, void* y, float* h_last,
            float* ckpt, int64_t Bs, int64_t L, int64_t ED, int dtype, void* ws, hipStream_t st) {
  const FwdPlan f = fwd_plan(Bs, L, ED, dtype);
  GlrArgs<T> a{};
  a.x = static_cast<const T*>(x), a.gr = static_cast<const T*>(gr), a.gi = static_cast<const T*>(gi);
  a.A = A, a.h0 = h0, a.y = static_cast<T*>(y), a.h_last = h_last, a.ckpt = ckpt;
  a.Bs = Bs, a.L = L, a.ED = ED, a.ckrows = (L + kCk - 1) / kCk;
  a.nchunks = f.nchunks, a.ngroups = f.ngroups, a.ncg = f.ncg;
  if (f.nchunks > 1) {
    char* w = static_cast<char*>(ws);
    a.hdr = reinterpret_cast<unsigned*>(w), a.flag = reinterpret_cast<unsigned*>(w + f.flag);
    a.state = reinterpret_cast<uint64_t*>(w + f.state), a.map = reinterpret_cast<uint64_t*>(w + f.map);
    a.spin_limit = split_spin_limit();
  }
  if constexpr (sizeof(T) == 2)
    if (fwd_vec(ED, dtype) == 2) return launch_fwd<T, 2>(a, f, ws, st);
  return launch_fwd<T, 1>(a, f, ws, st);
}

template <typename T>
int run_bwd(const void* x, const void* gr, const void* gi, const float* A, const float* ckpt, const void* dy,
            const float* dh_last, void* dx, void* dgr, void* dgi, float* dA, float* dh0, int64_t Bs, int64_t L,
            int64_t ED, int dtype, void* ws, hipStream_t st) {
  const BwdPlan pl = bwd_plan(Bs, L, ED, dtype);
  GlrArgs<T> a{};
  a.x = static_cast<const T*>(x), a.gr = static_cast<const T*>(gr), a.gi = static_cast<const T*>(gi);
  a.A = A, a.ckpt = const_cast<float*>(ckpt), a.dy = static_cast<const T*>(dy), a.dh_last = dh_last;
  a.dx = static_cast<T*>(dx), a.dgr = static_cast<T*>(dgr), a.dgi = static_cast<T*>(dgi), a.dh0 = dh0;
  a.Bs = Bs, a.L = L, a.ED = ED, a.nchunks = pl.nchunks, a.steps = pl.steps, a.ckrows = pl.ckrows;
  char* w = static_cast<char*>(ws);
  a.agg = reinterpret_cast<float2*>(w);
  a.enter = reinterpret_cast<float*>(w + glr_agg_bytes(pl, Bs * ED));
  a.dA_part = reinterpret_cast<float*>(w + glr_agg_bytes(pl, Bs * ED) + glr_enter_bytes(pl, Bs * ED));
  if constexpr (sizeof(T) == 2)
    if (fwd_vec(ED, dtype) == 2) return launch_bwd<T, 2>(a, dA, st);
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
  return static_cast<size_t>(fwd_plan(Bs, L, ED, dtype).bytes);
}

extern "C" size_t ssm_glr_bwd_workspace_bytes(int64_t Bs, int64_t L, int64_t ED, int dtype) {
  int64_t n, nck;
  if (glr_sizes(Bs, L, ED, dtype, &n, &nck) != SSM_OK || n == 0) return 0;
  const BwdPlan pl = bwd_plan(Bs, L, ED, dtype);
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
  return dtype == SSM_F32 ? run_fwd<float>(x, gr, gi, A, h0, y, h_last, ckpt, Bs, L, ED, dtype, workspace, st)
                          : run_fwd<uint16_t>(x, gr, gi, A, h0, y, h_last, ckpt, Bs, L, ED, dtype, workspace, st);
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
             ? run_bwd<float>(x, gr, gi, A, ckpt, dy, dh_last, dx, dgr, dgi, dA, dh0, Bs, L, ED, dtype, workspace, st)
             : run_bwd<uint16_t>(x, gr, gi, A, ckpt, dy, dh_last, dx, dgr, dgi, dA, dh0, Bs, L, ED, dtype, workspace, st);
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
