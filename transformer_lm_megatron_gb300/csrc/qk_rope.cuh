// Norms of queries and keys for each head with the position rotation in the same
// pass, forward and backward (HBM-bound).
//
// For one head vector x of d elements, weights w and the angles t_i of its token:
//   n = x r w,  r = (mean(x^2) + eps)^(-1/2)             (or n = x without weights)
//   y: the pairs of the first `rot` elements of n turned, (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// and backward, with g = the gradient of y turned by -t:
//   dw = sum g x r,   dx = r (w g - x r^2 mean(w g x))   (or dx = g)
// Pair i is (i, i + rot/2), or (2i, 2i + 1) when interleaved; t_i = position[axis(i)] * inv_freq[i].
//
// Angles.  A position times a frequency loses all its digits in fp32 once it is
// some 10^6 radians, so the frequency is taken once per thread in turns as a 64-bit
// fixed-point fraction; the product with the integer position, modulo 2^64, is then
// the angle modulo one turn, off by 2^-64 of a turn times the position.  Its top 32
// bits go through sincospi as an fp32, whose rounding of up to 2^-26 of a turn is the
// largest part of the angle's error.
//
// Work.  A head is 2 * VEC elements per lane, two vectors of VEC that hold VEC whole
// pairs, so a lane needs no other lane's elements to turn its own, and a warp holds
// several heads at once (d = 128: 4 heads of 8 lanes): a step.  The steps of all tokens in
// a row are shared out over the warps evenly (whole tokens to a warp left a third of the
// SMs idle at 2048 tokens); a warp forms the sines and cosines of a token's pairs once,
// its lanes a share each, for each token that it comes to.  The heads
// come through a ring in shared memory, several steps ahead and across tokens; a lane
// reads back only what it copied itself, so the ring needs no barrier.  Arithmetic is
// fp32, two values an instruction; outputs are rounded once.
// dw: every lane sums its elements over one token's heads in registers and over its
// tokens in shared memory; the warps of a CTA add theirs in a fixed order into one row
// of the workspace, and a second launch adds the rows in a fixed order: the result does
// not depend on timing.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace gbmlp {

constexpr int kQkWarps = 8;
constexpr int kQkThreads = 32 * kQkWarps;
constexpr int kQkMaxHead = 256;     // largest d: 32 lanes of 2 * 4 elements
constexpr int kQkWsRows = 1024;     // most CTAs of a backward: rows of 2 d floats in its workspace
constexpr int kQkMaxPerSm = 6;      // most CTAs on an SM: 6 * 152 rows stay within the workspace

struct QkRopeParams {
  int64_t tokens;
  int nq, nk, d, rot;
  int axis1, axis2;           // pairs [0, axis1) turn with axis 0, [axis1, axis2) with axis 1, the rest with axis 2
  int steps_q, steps_k;       // a warp's steps over one token's queries and keys
  float eps;
  const uint16_t* wq;         // [d], null without the norm
  const uint16_t* wk;
  const int32_t* pos;         // [axes, tokens]
  const float* inv_freq;      // [rot / 2]
  const uint16_t* q;          // raw queries and keys (forward input; backward with the norm)
  const uint16_t* k;
  int64_t ldq, ldk;
  const uint16_t* gq;         // backward: gradient of the forward's outputs
  const uint16_t* gk;
  int64_t ldgq, ldgk;
  uint16_t* oq;               // forward outputs, or dq and dk
  uint16_t* ok;
  int64_t ldoq, ldok;
  float* ws;                  // backward with the norm: [gridDim.x, 2 d]
};

// ---- two fp32 values in one register pair: half the instructions of scalar arithmetic
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float f2_sum(uint64_t v) { return f2_lo(v) + f2_hi(v); }
__device__ __forceinline__ uint64_t f2_swap(uint64_t v) { return f2(f2_hi(v), f2_lo(v)); }

template <int VEC>
struct QkVec {
  uint32_t w[VEC / 2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (VEC == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) w[j] = 0;
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    if constexpr (VEC == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ float at(int j) const { return (j & 1) ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]); }
  __device__ __forceinline__ uint64_t pair(int j) const { return f2(bf16lo(w[j]), bf16hi(w[j])); }
};

// The place of a lane: which of the warp's heads, and which elements of it.
template <int VEC, bool INTER>
struct QkLane {
  int lph, hpw;      // lanes per head, heads per warp
  int grp, li;       // this lane's head of the warp and its place in it
  int e0, e1;        // its two vectors
  bool active, turns;
  static constexpr int kTop = VEC == 8 ? 8 : 16;  // lph is at most 16 or 32
  __device__ __forceinline__ QkLane(int d, int rot, int lane) {
    lph = d / (2 * VEC);
    hpw = 32 / lph;
    grp = lane / lph;
    li = lane - grp * lph;
    active = grp < hpw;
    const int turning = rot / (2 * VEC);
    turns = li < turning;
    if (INTER || !turns) {
      e0 = 2 * VEC * li;  // elements behind `rot` follow the turning ones in order
      e1 = e0 + VEC;
    } else {
      e0 = VEC * li;
      e1 = e0 + rot / 2;
    }
  }
  // The sum over a head's lanes, in every lane of it, in a fixed order.
  __device__ __forceinline__ float sum(float v) const {
    if ((lph & (lph - 1)) == 0) {
#pragma unroll
      for (int o = kTop; o > 0; o >>= 1)
        if (o < lph) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    }
#pragma unroll
    for (int o = kTop; o > 0; o >>= 1) {
      const float t = __shfl_down_sync(0xffffffffu, v, o);
      if (li < min(o, lph - o)) v += t;
    }
    return __shfl_sync(0xffffffffu, v, (grp * lph) & 31);
  }
};

// A lane's way through its warp's work: `left` steps of hpw heads from some step of some
// token on, each token's queries before its keys.  A run is what is left of one tensor at
// one token; `room` counts the heads from the lane's own to the last of the run (the lane
// has none where it is 0 or less).
struct QkWalk {
  int left, token, is_k, run, room;
  // The first of `n` steps: the `step`th of the token.
  __device__ __forceinline__ void start(const QkRopeParams& p, int n, int first_token, int step, int hpw, int grp) {
    left = n;
    token = first_token;
    enter(p, step >= p.steps_q ? 1 : 0, step >= p.steps_q ? step - p.steps_q : step, hpw, grp);
  }
  __device__ __forceinline__ void enter(const QkRopeParams& p, int tensor, int step, int hpw, int grp) {
    is_k = tensor;
    run = (tensor ? p.steps_k : p.steps_q) - step;
    room = grp < hpw ? (tensor ? p.nk : p.nq) - step * hpw - grp : 0;
  }
  // One step on; true where a new run begins.
  __device__ __forceinline__ bool advance(const QkRopeParams& p, int hpw, int grp) {
    --left;
    room -= hpw;
    if (--run > 0) return false;
    if (is_k) ++token;
    enter(p, is_k ^ 1, 0, hpw, grp);
    return true;
  }
  // The lane's first element in a tensor with these rows.
  template <typename T>
  __device__ __forceinline__ T* place(const QkRopeParams& p, T* q, int64_t ldq, T* k, int64_t ldk, int e0) const {
    const int64_t row = is_k ? token * ldk : token * ldq;
    const int head = room > 0 ? (is_k ? p.nk : p.nq) - room : 0;
    return (is_k ? k : q) + row + (int64_t)head * p.d + (room > 0 ? e0 : 0);
  }
};

// VEC elements from global into shared memory, without waiting; zeros where !ok.
template <int VEC>
__device__ __forceinline__ void qk_copy(uint32_t dst, const uint16_t* src, bool ok) {
  if constexpr (VEC == 8)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}

// A frequency (radians per position) in turns, as a fraction of 2^64: the fp32 value
// m 2^x times 2^66 / (2 pi), rounded to 64 bits, shifted.  Off by one unit at most for
// |inv_freq| <= 1 (a frequency above 2^25 keeps fewer digits).  In integers, since fp64
// is slow on this GPU.
__device__ __forceinline__ uint64_t qk_turns(float inv_freq) {
  const uint32_t bits = __float_as_uint(inv_freq);
  const int e = (bits >> 23) & 0xff;
  const uint32_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  constexpr uint64_t k = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const uint64_t lo = k * m, hi = __umul64hi(k, m);
  const int right = 152 - (e ? e : 1);             // m 2^(e - 150) * k / 4, in units of 2^-64 turns
  uint64_t t;
  if (right <= 0)
    t = right > -64 ? lo << -right : 0;
  else if (right < 64)
    t = (lo >> right) | (hi << (64 - right));
  else
    t = right < 128 ? hi >> (right - 64) : 0;
  return (bits >> 31) ? 0 - t : t;
}

// The positions of one token.
struct QkPos {
  int32_t at[3];
  __device__ __forceinline__ void load(const QkRopeParams& p, int64_t token) {
    const int half = p.rot >> 1;
    at[0] = p.pos[token];
    at[1] = p.axis1 < half ? p.pos[p.tokens + token] : 0;
    at[2] = p.axis2 < half ? p.pos[2 * p.tokens + token] : 0;
  }
};

constexpr int kQkPairs = kQkMaxHead / 2;  // most pairs of a head

// The cosines and sines of a token's pairs, in a warp's shared memory.
struct QkAngles {
  float cs[kQkPairs], sn[kQkPairs];
};

// Fills them for position x: the warp's lanes share out the pairs, whose frequencies are
// `turn`.
__device__ __forceinline__ void qk_angles(const QkRopeParams& p, const QkPos& x, const uint64_t* turn, QkAngles& out) {
  __syncwarp();  // the last token's have been read
  for (int i = threadIdx.x & 31; i < (p.rot >> 1); i += 32) {
    const int32_t at = i < p.axis1 ? x.at[0] : i < p.axis2 ? x.at[1] : x.at[2];
    const uint64_t phase = (uint64_t)(int64_t)at * turn[i];
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &out.sn[i], &out.cs[i]);
  }
  __syncwarp();
}

// The turn of a lane's two vectors x as out[v] = own P[v] + partner Q[v], two elements a
// word: the partner of an element of one vector is the same one of the other vector, or
// (interleaved) its neighbour.  sign 1 turns forwards; w[v]: the elements' weights
// (NORM), multiplied in.
template <int VEC, bool INTER, bool WEIGHTS>
__device__ __forceinline__ void qk_turn_terms(const QkAngles& angles, const QkLane<VEC, INTER>& L, float sign,
                                              const QkVec<VEC> (&w)[2], uint64_t (&P)[2][VEC / 2],
                                              uint64_t (&Q)[2][VEC / 2]) {
  float cs[VEC], sn[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    cs[j] = L.turns ? angles.cs[VEC * L.li + j] : 1.0f;
    sn[j] = L.turns ? angles.sn[VEC * L.li + j] : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const float w0 = WEIGHTS ? w[v].at(2 * j) : 1.0f, w1 = WEIGHTS ? w[v].at(2 * j + 1) : 1.0f;
      if constexpr (INTER) {
        const float c = cs[v * VEC / 2 + j], s = sign * sn[v * VEC / 2 + j];
        P[v][j] = f2(w0 * c, w1 * c);
        Q[v][j] = f2(-w1 * s, w0 * s);
      } else {
        const float c0 = cs[2 * j], c1 = cs[2 * j + 1];
        const float s0 = (v ? sign : -sign) * sn[2 * j], s1 = (v ? sign : -sign) * sn[2 * j + 1];
        const float u0 = WEIGHTS ? w[v ^ 1].at(2 * j) : 1.0f, u1 = WEIGHTS ? w[v ^ 1].at(2 * j + 1) : 1.0f;
        P[v][j] = f2(w0 * c0, w1 * c1);
        Q[v][j] = f2(u0 * s0, u1 * s1);
      }
    }
}

// turns: whether the lane's elements turn at all.  Those behind `rot` take their weights alone,
// since an infinity times the sine 0 of their pair would be NaN (a lane turns whole or not, and
// where rot = d all do).
template <int VEC, bool INTER, bool WEIGHTS>
__device__ __forceinline__ void qk_turn(uint64_t (&x)[2][VEC / 2], const uint64_t (&P)[2][VEC / 2],
                                        const uint64_t (&Q)[2][VEC / 2], bool turns) {
  if (!turns) {
    if constexpr (WEIGHTS) {
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        x[0][j] = f2_mul(x[0][j], P[0][j]);
        x[1][j] = f2_mul(x[1][j], P[1][j]);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    const uint64_t a = x[0][j], b = x[1][j];
    x[0][j] = f2_fma(INTER ? f2_swap(a) : b, Q[0][j], f2_mul(a, P[0][j]));
    if constexpr (INTER || WEIGHTS)
      x[1][j] = f2_fma(INTER ? f2_swap(b) : a, Q[1][j], f2_mul(b, P[1][j]));
    else  // P[1] = P[0] and Q[1] = -Q[0], not held
      x[1][j] = f2_sub(f2_mul(b, P[0][j]), f2_mul(a, Q[0][j]));
  }
}

template <int VEC>
__device__ __forceinline__ void qk_unpack(const uint8_t* slot, uint64_t (&f)[VEC / 2]) {
  QkVec<VEC> v;
  v.load(reinterpret_cast<const uint16_t*>(slot));
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) f[j] = f2(bf16lo(v.w[j]), bf16hi(v.w[j]));
}

template <int VEC>
__device__ __forceinline__ void qk_pack_store(uint16_t* dst, const uint64_t (&f)[VEC / 2]) {
  QkVec<VEC> v;
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) v.w[j] = pack_bf16x2(f2_lo(f[j]), f2_hi(f[j]));
  v.store(dst);
}

// Steps in a warp's ring: the one at work and those on their way.  2048 x 256 heads of 160
// forward (336 MB: 49 us at the copy rate): 123 us with the loads of one step straight into
// registers, 75 us with four steps in registers; with the ring 57 us at 4 steps, 62 at 6.
// 8209 x 40 heads of 128 backward (252 MB: 37 us), dw's second launch with it: 47 us at 3
// or 4 steps, 57 at 2.  What is left is DRAM latency at 16 warps an SM (128 registers; the
// forward at 24 warps is no faster).
constexpr int kQkDepth = 4;

// Dynamic shared memory of a kernel: the frequencies, every warp's cosines and sines, the
// sums of dw (backward with the norm), and the rings: per warp DEPTH steps of VECS vectors
// a lane.
template <int VEC, bool BWD, bool NORM>
struct QkSmem {
  static constexpr int kVecs = BWD && NORM ? 4 : 2;
  static constexpr int kDepth = kQkDepth;
  static constexpr int kVecBytes = 2 * VEC * 32;  // one vector of every lane
  static constexpr int kTurn = 0;
  static constexpr int kAngles = kTurn + kQkPairs * 8;
  static constexpr int kPart = kAngles + kQkWarps * (int)sizeof(QkAngles);
  static constexpr int kRing = kPart + (BWD && NORM ? kQkWarps * 2 * 2 * VEC * 32 * 4 : 0);
  static constexpr int kBytes = kRing + kQkWarps * kDepth * kVecs * kVecBytes;
};

// VEC, INTER and NORM as above; BWD: the backward.
template <int VEC, bool INTER, bool NORM, bool BWD>
__global__ void __launch_bounds__(kQkThreads, 2) k_qk_norm_rope(QkRopeParams p) {
  using Smem = QkSmem<VEC, BWD, NORM>;
  constexpr int D = Smem::kDepth, H = VEC / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  uint64_t* turn = reinterpret_cast<uint64_t*>(smem + Smem::kTurn);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (uniform to the compiler)
  QkAngles& angles = reinterpret_cast<QkAngles*>(smem + Smem::kAngles)[warp];
  // dw of every lane's elements over its warp's tokens: [warp][q | k][element of the lane][lane]
  float* part = reinterpret_cast<float*>(smem + Smem::kPart);
  uint8_t* ring = smem + Smem::kRing + warp * (D * Smem::kVecs * Smem::kVecBytes) + lane * (2 * VEC);
  const QkLane<VEC, INTER> L(p.d, p.rot, lane);
  grid_dependency_wait();
  grid_launch_dependents();

  // this warp's steps of all, even to within one
  const int per_token = p.steps_q + p.steps_k;
  const int64_t all = p.tokens * per_token, warps = (int64_t)gridDim.x * kQkWarps;
  const int64_t me = (int64_t)blockIdx.x * kQkWarps + warp, each = all / warps, extra = all - each * warps;
  const int64_t first = me * each + (me < extra ? me : extra);
  const int my_steps = (int)each + (me < extra ? 1 : 0), first_token = (int)(first / per_token);
  const int step = L.hpw * p.d, de = L.e1 - L.e0;  // elements from one step to the next, and to the second vector
  QkWalk at, ahead;  // the step at work, and the next one to fetch
  at.start(p, my_steps, first_token, (int)(first - (int64_t)first_token * per_token), L.hpw, L.grp);
  ahead = at;
  const uint16_t *x_src = nullptr, *g_src = nullptr;
  auto sources = [&]() {
    if constexpr (!BWD || NORM) x_src = ahead.place(p, p.q, p.ldq, p.k, p.ldk, L.e0);
    if constexpr (BWD) g_src = ahead.place(p, p.gq, p.ldgq, p.gk, p.ldgk, L.e0);
  };
  if (ahead.left > 0) sources();
  const uint32_t ring_at = smem_u32(ring);
  uint32_t fetched = 0;
  auto fetch = [&]() {
    if (ahead.left > 0) {
      const bool ok = ahead.room > 0;
      const int second = ok ? de : 0;
      uint32_t dst = ring_at + fetched;
      if constexpr (BWD) {
        qk_copy<VEC>(dst, g_src, ok);
        qk_copy<VEC>(dst + Smem::kVecBytes, g_src + second, ok);
        dst += 2 * Smem::kVecBytes;
      }
      if constexpr (!BWD || NORM) {
        qk_copy<VEC>(dst, x_src, ok);
        qk_copy<VEC>(dst + Smem::kVecBytes, x_src + second, ok);
      }
      fetched = fetched == (D - 1) * Smem::kVecs * Smem::kVecBytes ? 0 : fetched + Smem::kVecs * Smem::kVecBytes;
      if (!ahead.advance(p, L.hpw, L.grp)) {
        // (a lane whose heads have ended reads no more of this run)
        const int on = ahead.room > 0 ? step : 0;
        if constexpr (!BWD || NORM) x_src += on;
        if constexpr (BWD) g_src += on;
      } else if (ahead.left > 0) {
        sources();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < D - 1; ++s) fetch();
  QkPos pos;
  if (at.left > 0) pos.load(p, at.token);
  for (int i = threadIdx.x; i < (p.rot >> 1); i += kQkThreads) turn[i] = qk_turns(p.inv_freq[i]);
  float* mine = part + warp * 2 * 2 * VEC * 32 + lane;
  if constexpr (BWD && NORM)
    for (int j = 0; j < 2 * 2 * VEC; ++j) mine[j * 32] = 0.0f;
  __syncthreads();

  const float inv_d = 1.0f / (float)p.d;
  int token = -1;      // whose angles the warp holds
  int tensor = -1;     // whose terms P and Q hold
  uint32_t slot = 0;
  uint16_t* out = nullptr;
  uint64_t P[2][H], Q[2][H];
  uint64_t acc[BWD && NORM ? 2 : 1][H];
  QkVec<VEC> w[2];
  while (at.left > 0) {
    if (at.token != token) {
      token = at.token;
      tensor = -1;
      qk_angles(p, pos, turn, angles);
      if (token + 1 < p.tokens) pos.load(p, token + 1);  // in time for the next token
    }
    if (at.is_k != tensor) {
      tensor = at.is_k;
      out = at.place(p, p.oq, p.ldoq, p.ok, p.ldok, L.e0);
      if constexpr (NORM) {
        w[0].zero();
        w[1].zero();
        if (L.active) {
          const uint16_t* src = tensor ? p.wk : p.wq;
          w[0].load(src + L.e0);
          w[1].load(src + L.e1);
        }
      }
      qk_turn_terms<VEC, INTER, NORM && !BWD>(angles, L, BWD ? -1.0f : 1.0f, w, P, Q);
      if constexpr (BWD && NORM) {
#pragma unroll
        for (int j = 0; j < H; ++j) acc[0][j] = acc[1][j] = 0;
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
    const uint8_t* src = ring + slot;
    slot = slot == (D - 1) * Smem::kVecs * Smem::kVecBytes ? 0 : slot + Smem::kVecs * Smem::kVecBytes;
    uint64_t y[2][H];
    qk_unpack<VEC>(src, y[0]);
    qk_unpack<VEC>(src + Smem::kVecBytes, y[1]);
    if constexpr (!BWD) {
      if constexpr (NORM) {
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int j = 0; j < H; ++j) {
          s0 = f2_fma(y[0][j], y[0][j], s0);
          s1 = f2_fma(y[1][j], y[1][j], s1);
        }
        const float r = rsqrtf(fmaf(L.sum(f2_sum(s0) + f2_sum(s1)), inv_d, p.eps));
        const uint64_t rr = f2(r, r);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          y[0][j] = f2_mul(y[0][j], rr);
          y[1][j] = f2_mul(y[1][j], rr);
        }
      }
      qk_turn<VEC, INTER, NORM>(y, P, Q, L.turns);
    } else {
      qk_turn<VEC, INTER, false>(y, P, Q, L.turns);
      if constexpr (NORM) {
        // x stays packed: unpacked twice it costs fewer registers than it takes
        QkVec<VEC> x[2];
        x[0].load(reinterpret_cast<const uint16_t*>(src + 2 * Smem::kVecBytes));
        x[1].load(reinterpret_cast<const uint16_t*>(src + 3 * Smem::kVecBytes));
        uint64_t ss[2] = {0, 0}, sg[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint64_t xv = x[v].pair(j);
            ss[v] = f2_fma(xv, xv, ss[v]);
            sg[v] = f2_fma(f2_mul(y[v][j], w[v].pair(j)), xv, sg[v]);
          }
        // (a lane without a head has zeros, whose root at eps = 0 would put NaN into dw: it takes eps = 1)
        const float r = rsqrtf(fmaf(L.sum(f2_sum(ss[0]) + f2_sum(ss[1])), inv_d, at.room > 0 ? p.eps : 1.0f));
        const float c = L.sum(f2_sum(sg[0]) + f2_sum(sg[1])) * inv_d * r * r * r;
        const uint64_t rr = f2(r, r), nc = f2(-c, -c);
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            const uint64_t gr = f2_mul(y[v][j], rr), xv = x[v].pair(j);
            acc[v][j] = f2_fma(gr, xv, acc[v][j]);
            y[v][j] = f2_fma(gr, w[v].pair(j), f2_mul(xv, nc));
          }
      }
    }
    if (at.room > 0) {
      qk_pack_store<VEC>(out, y[0]);
      qk_pack_store<VEC>(out + de, y[1]);
      out += step;
    }
    fetch();
    const bool run_ends = at.advance(p, L.hpw, L.grp);
    if constexpr (BWD && NORM) {
      if (at.left == 0 || run_ends) {
        float* m = mine + tensor * 2 * VEC * 32;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            m[(v * VEC + 2 * j) * 32] += f2_lo(acc[v][j]);
            m[(v * VEC + 2 * j + 1) * 32] += f2_hi(acc[v][j]);
          }
      }
    }
  }
  if constexpr (BWD && NORM) {
    __syncthreads();
    // column c of head element e: the lanes of every warp and head group that held it
    for (int c = threadIdx.x; c < 2 * p.d; c += kQkThreads) {
      const int s = c / p.d, e = c - s * p.d;
      int li, j;
      if (INTER || e >= p.rot) {
        li = e / (2 * VEC);
        j = e - li * 2 * VEC;
      } else {
        const int f = e < p.rot / 2 ? e : e - p.rot / 2;
        li = f / VEC;
        j = f - li * VEC + (e < p.rot / 2 ? 0 : VEC);
      }
      float tot = 0.0f;
      for (int v = 0; v < kQkWarps; ++v)
        for (int g = 0; g < L.hpw; ++g) tot += part[((v * 2 + s) * 2 * VEC + j) * 32 + g * L.lph + li];
      p.ws[(int64_t)blockIdx.x * 2 * p.d + c] = tot;
    }
  }
}

// dwq, dwk (+)= the column sums of ws [rows, 2 d].  One CTA per 32 columns; each of its
// 32 rows of threads sums a fixed subset of the rows, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) k_qk_dw(const float* ws, int rows, int d, float* dwq, float* dwk,
                                                int accumulate) {
  __shared__ float part[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float s = 0.0f;
  if (c < 2 * d)
    for (int r = y; r < rows; r += 32) s += ws[(int64_t)r * 2 * d + c];
  part[y][x] = s;
  __syncthreads();
  if (y == 0 && c < 2 * d) {
    float tot = 0.0f;
    for (int k = 0; k < 32; ++k) tot += part[k][x];
    float* out = c < d ? dwq + c : dwk + (c - d);
    *out = accumulate ? *out + tot : tot;
  }
}

}  // namespace gbmlp
