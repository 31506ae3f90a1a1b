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
// the angle modulo one turn without further error, and its top 32 bits go through
// sincospi.  (The fraction is computed in fp64: off by 2^-53 of a turn at most, times
// the position.)
//
// Work.  A head is 2 * VEC elements per lane, two vectors of VEC that hold VEC whole
// pairs, so a lane needs no other lane's elements to turn its own, and a warp holds
// several heads at once (d = 128: 4 heads of 8 lanes).  A warp takes one token, forms
// the sines and cosines of its lanes' pairs once, and walks that token's heads; when
// there are few tokens the heads of one are shared out over several warps.  Statistics,
// products and sums are fp32; outputs are rounded once.
// dw: every lane sums its elements over all heads and tokens of its warp in registers,
// the warps of a CTA add theirs in a fixed order into one row of the workspace, and a
// second launch adds the rows in a fixed order: the result does not depend on timing.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace gbmlp {

constexpr int kQkWarps = 8;
constexpr int kQkThreads = 32 * kQkWarps;
constexpr int kQkMaxHead = 256;     // largest d: 32 lanes of 2 * 4 elements
constexpr int kQkWsRows = 1024;     // most CTAs of a backward: rows of 2 d floats in its workspace

struct QkRopeParams {
  int64_t tokens;
  int nq, nk, d, rot;
  int axis1, axis2;           // pairs [0, axis1) turn with axis 0, [axis1, axis2) with axis 1, the rest with axis 2
  int heads_per_unit, units;  // a warp's share of one token's nq + nk heads, and shares per token
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
};

// The place of a lane: which of the warp's heads, and which elements of it.
template <int VEC, bool INTER>
struct QkLane {
  int lph, hpw;      // lanes per head, heads per warp
  int grp, li;       // this lane's head of the warp and its place in it
  int e0, e1;        // its two vectors
  bool active, turns;
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
      for (int o = lph >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const float t = __shfl_down_sync(0xffffffffu, v, o);
      if (li < o && li + o < lph) v += t;
    }
    return __shfl_sync(0xffffffffu, v, (grp * lph) & 31);
  }
};

// A frequency (radians per position) in turns, as a fraction of 2^64.
__device__ __forceinline__ uint64_t qk_turns(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;
  t -= floor(t);
  return (uint64_t)__double2ull_rz(t * 18446744073709551616.0);
}

// Sines and cosines of a lane's VEC pairs at one token.
template <int VEC>
__device__ __forceinline__ void qk_angles(const QkRopeParams& p, int64_t token, const uint64_t (&turn)[VEC],
                                          uint32_t axes, bool turns, float (&cs)[VEC], float (&sn)[VEC]) {
  int32_t at[3];
  const int half = p.rot >> 1;
  at[0] = p.pos[token];
  at[1] = p.axis1 < half ? p.pos[p.tokens + token] : 0;
  at[2] = p.axis2 < half ? p.pos[2 * p.tokens + token] : 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const uint32_t a = (axes >> (2 * j)) & 3u;
    const int32_t x = a == 0 ? at[0] : a == 1 ? at[1] : at[2];
    const uint64_t phase = (uint64_t)(int64_t)x * turn[j];
    const float half_turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
    sincospif(half_turns, &sn[j], &cs[j]);
    if (!turns) {
      cs[j] = 1.0f;
      sn[j] = 0.0f;
    }
  }
}

// Turns the lane's pairs in a (first vector) and b (second) by their angles.
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_turn(float (&a)[VEC], float (&b)[VEC], const float (&cs)[VEC], const float (&sn)[VEC],
                                        float sign) {
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1], s = sign * sn[j];
      a[2 * j] = x * cs[j] - y * s;
      a[2 * j + 1] = y * cs[j] + x * s;
      const float u = b[2 * j], v = b[2 * j + 1], t = sign * sn[VEC / 2 + j];
      b[2 * j] = u * cs[VEC / 2 + j] - v * t;
      b[2 * j + 1] = v * cs[VEC / 2 + j] + u * t;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float x = a[j], y = b[j], s = sign * sn[j];
      a[j] = x * cs[j] - y * s;
      b[j] = y * cs[j] + x * s;
    }
  }
}

// What a lane keeps over all its tokens.
template <int VEC, bool INTER>
__device__ __forceinline__ uint32_t qk_lane_setup(const QkRopeParams& p, const QkLane<VEC, INTER>& L,
                                                  uint64_t (&turn)[VEC]) {
  uint32_t axes = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    turn[j] = 0;
    const int i = VEC * L.li + j;
    if (L.active && L.turns) {
      turn[j] = qk_turns(p.inv_freq[i]);
      axes |= (i < p.axis1 ? 0u : i < p.axis2 ? 1u : 2u) << (2 * j);
    }
  }
  return axes;
}

template <int VEC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kQkThreads) k_qk_norm_rope(QkRopeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const QkLane<VEC, INTER> L(p.d, p.rot, lane);
  uint64_t turn[VEC];
  const uint32_t axes = qk_lane_setup<VEC, INTER>(p, L, turn);
  const float inv_d = 1.0f / (float)p.d;
  const int64_t n_units = p.tokens * p.units;
  for (int64_t u = (int64_t)blockIdx.x * kQkWarps + (threadIdx.x >> 5); u < n_units;
       u += (int64_t)gridDim.x * kQkWarps) {
    const int64_t token = u / p.units;
    const int h0 = (int)(u - token * p.units) * p.heads_per_unit;
    const int h1 = min(h0 + p.heads_per_unit, p.nq + p.nk);
    float cs[VEC], sn[VEC];
    qk_angles<VEC>(p, token, turn, axes, L.turns, cs, sn);
    for (int h = h0; h < h1; h += L.hpw) {
      const int head = h + L.grp;
      const bool ok = L.active && head < h1;
      const bool is_k = head >= p.nq;
      QkVec<VEC> v0, v1;
      v0.zero();
      v1.zero();
      if (ok) {
        const uint16_t* x = is_k ? p.k + token * p.ldk + (int64_t)(head - p.nq) * p.d
                                 : p.q + token * p.ldq + (int64_t)head * p.d;
        v0.load(x + L.e0);
        v1.load(x + L.e1);
      }
      float a[VEC], b[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        a[j] = v0.at(j);
        b[j] = v1.at(j);
      }
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
        const float r = rsqrtf(fmaf(L.sum(ss), inv_d, p.eps));
        QkVec<VEC> w0, w1;
        w0.zero();
        w1.zero();
        if (ok) {
          const uint16_t* w = is_k ? p.wk : p.wq;
          w0.load(w + L.e0);
          w1.load(w + L.e1);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          a[j] = a[j] * r * w0.at(j);
          b[j] = b[j] * r * w1.at(j);
        }
      }
      qk_turn<VEC, INTER>(a, b, cs, sn, 1.0f);
      if (ok) {
        uint16_t* o = is_k ? p.ok + token * p.ldok + (int64_t)(head - p.nq) * p.d
                           : p.oq + token * p.ldoq + (int64_t)head * p.d;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          v0.w[j] = pack_bf16x2(a[2 * j], a[2 * j + 1]);
          v1.w[j] = pack_bf16x2(b[2 * j], b[2 * j + 1]);
        }
        v0.store(o + L.e0);
        v1.store(o + L.e1);
      }
    }
  }
}

template <int VEC, bool INTER, bool NORM>
__global__ void __launch_bounds__(kQkThreads) k_qk_norm_rope_bwd(QkRopeParams p) {
  // a warp's sums of dw, one 2 * VEC-element piece per lane: [warp][q | k][lane][2 VEC]
  __shared__ float part[NORM ? kQkWarps * 2 * 32 * 2 * VEC : 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane<VEC, INTER> L(p.d, p.rot, lane);
  uint64_t turn[VEC];
  const uint32_t axes = qk_lane_setup<VEC, INTER>(p, L, turn);
  const float inv_d = 1.0f / (float)p.d;
  const int64_t n_units = p.tokens * p.units;
  float dw[2][2 * VEC];
#pragma unroll
  for (int j = 0; j < 2 * VEC; ++j) dw[0][j] = dw[1][j] = 0.0f;
  for (int64_t u = (int64_t)blockIdx.x * kQkWarps + warp; u < n_units; u += (int64_t)gridDim.x * kQkWarps) {
    const int64_t token = u / p.units;
    const int h0 = (int)(u - token * p.units) * p.heads_per_unit;
    const int h1 = min(h0 + p.heads_per_unit, p.nq + p.nk);
    float cs[VEC], sn[VEC];
    qk_angles<VEC>(p, token, turn, axes, L.turns, cs, sn);
    // heads [begin, end) of the queries (IS_K = 0) or the keys (1)
    auto heads = [&](int begin, int end, const uint16_t* xs, int64_t ldx, const uint16_t* gs, int64_t ldg, uint16_t* os,
                     int64_t ldo, const uint16_t* ws, float (&acc)[2 * VEC]) {
      QkVec<VEC> w0, w1;
      w0.zero();
      w1.zero();
      if (NORM && L.active && begin < end) {
        w0.load(ws + L.e0);
        w1.load(ws + L.e1);
      }
      for (int h = begin; h < end; h += L.hpw) {
        const int head = h + L.grp;
        const bool ok = L.active && head < end;
        QkVec<VEC> g0, g1, x0, x1;
        g0.zero();
        g1.zero();
        x0.zero();
        x1.zero();
        if (ok) {
          const uint16_t* g = gs + token * ldg + (int64_t)head * p.d;
          g0.load(g + L.e0);
          g1.load(g + L.e1);
          if (NORM) {
            const uint16_t* x = xs + token * ldx + (int64_t)head * p.d;
            x0.load(x + L.e0);
            x1.load(x + L.e1);
          }
        }
        float a[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          a[j] = g0.at(j);
          b[j] = g1.at(j);
        }
        qk_turn<VEC, INTER>(a, b, cs, sn, -1.0f);
        if constexpr (NORM) {
          float ss = 0.0f, sg = 0.0f;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            ss = fmaf(x0.at(j), x0.at(j), fmaf(x1.at(j), x1.at(j), ss));
            sg = fmaf(a[j] * w0.at(j), x0.at(j), fmaf(b[j] * w1.at(j), x1.at(j), sg));
          }
          const float r = rsqrtf(fmaf(L.sum(ss), inv_d, p.eps));
          const float c = L.sum(sg) * inv_d * r * r;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            acc[j] = fmaf(a[j] * r, x0.at(j), acc[j]);
            acc[VEC + j] = fmaf(b[j] * r, x1.at(j), acc[VEC + j]);
            a[j] = r * (a[j] * w0.at(j) - x0.at(j) * c);
            b[j] = r * (b[j] * w1.at(j) - x1.at(j) * c);
          }
        }
        if (ok) {
          uint16_t* o = os + token * ldo + (int64_t)head * p.d;
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) {
            g0.w[j] = pack_bf16x2(a[2 * j], a[2 * j + 1]);
            g1.w[j] = pack_bf16x2(b[2 * j], b[2 * j + 1]);
          }
          g0.store(o + L.e0);
          g1.store(o + L.e1);
        }
      }
    };
    heads(min(h0, p.nq), min(h1, p.nq), p.q, p.ldq, p.gq, p.ldgq, p.oq, p.ldoq, p.wq, dw[0]);
    heads(max(h0, p.nq) - p.nq, max(h1, p.nq) - p.nq, p.k, p.ldk, p.gk, p.ldgk, p.ok, p.ldok, p.wk, dw[1]);
  }
  if constexpr (NORM) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2 * VEC; ++j) part[(((warp * 2 + s) * 32) + lane) * 2 * VEC + j] = dw[s][j];
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
      for (int w = 0; w < kQkWarps; ++w)
        for (int g = 0; g < L.hpw; ++g) tot += part[((w * 2 + s) * 32 + g * L.lph + li) * 2 * VEC + j];
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
