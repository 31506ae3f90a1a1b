// Attention of each request's new tokens over its cached keys and values (8-bit codes, a maximum
// for each block and head: kv_cache.cuh), for few new tokens.
//
//   O = softmax(scale Q K^T) V,  K = Kc Kmax / 127,  V = Vc Vmax / 127
//
// HBM bounds it: a code is read once and meets 4 * rows operations, rows = new tokens * query heads
// of a key head.  What counts is that every SM has reads in flight all the time and that a
// code becomes a matrix operand in few instructions:
//   - Work is counted in steps of 16 tokens, over all requests, heads and tiles of 16 rows, and cut
//     into equal shares, one for each CTA that fits on the GPU, wherever that falls: a long request
//     spreads over all SMs, a ragged batch leaves none idle.  A tile that ends up with several
//     CTAs leaves its parts (fp32 sums, maximum and denominator of each row) in the workspace, and
//     k_kv_attn_join adds them up in order, so results do not change from run to run.
//   - Each warp takes every fourth step of a share, alone: its lanes copy to shared memory,
//     asynchronously and some steps ahead, the very bytes that they later feed to the tensor
//     cores, so there is no barrier in the loop and no transposition: reductions may run
//     over d and over tokens in any order, so a lane's 16 bytes of a key are the operands of four
//     successive MMAs, and its 16 bytes of four tokens' values those of 16 column tiles.
//   - Codes become fp16 exactly (1024 + (c + 128) by a byte permutation, minus 1152): 5 instructions
//     for 4 keys, 6 for 4 values.  mma.sync, not tcgen05: operands come from registers, where
//     the codes are converted, and a tile has 16 rows or fewer where tcgen05's has 64 at least.
//   - Queries go to fp16 with a power of two for each row that brings its largest element below
//     2^15: exact but for elements under 2^-29 of it.
//   - A block's value scale goes into the exponent: p' = exp2(s + log2(vscale) - max + 14) is the
//     operand of the second product, at most 2^14, so that fp16 holds what is above 2^-28 of
//     the largest in full precision, whatever the scales; the denominator adds p' / vscale in fp32.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace gbmlp {

constexpr int kKaWarps = 4;
constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaRows = 16;        // query rows of a tile
constexpr int kKaStep = 16;        // tokens of a step
constexpr int kKaWsRows = 19456;   // of the workspace, d + 2 floats each: two parts of 16 rows for 608 CTAs
constexpr int kKaMaxCtas = 600;    // ... of which 8 leave room for the descriptors
constexpr int kKaMinPart = 8;      // steps: no tile is cut nearer than this to either end
constexpr float kKaLift = 14.0f;   // p' is at most 2^14

struct KvAttnParams {
  int n, nq, nk, group, width, log_bs, blocks;
  int64_t rows;                 // of Q and O
  int64_t ldq, ldo;
  float scale_log2;             // scale * log2(e) / 127: scores in powers of two, and the keys' 127
  const uint16_t* q;
  const int8_t* kc;
  const int8_t* vc;
  const float* kmax;
  const float* vmax;
  const int* table;
  const int* lens;
  const int* cu;
  uint16_t* o;
  float* ws;
};

// The workspace: a descriptor of 8 ints for each CTA, then two parts for each (the tile that it begins in
// the middle of, or its first; and the one that it ends in the middle of): maxima, denominators, sums.
struct KaJoin {
  int parts, slot, row0, head, tile, rows, pad[2];  // parts: 0 if no tile begins here and goes on elsewhere
};
__host__ __device__ constexpr int64_t ka_part_floats(int d) { return (int64_t)kKaRows * (d + 2); }
static_assert(kKaMaxCtas * (int64_t)sizeof(KaJoin) + 4 * 2 * kKaMaxCtas * ka_part_floats(32) <= 4 * (int64_t)kKaWsRows * (32 + 2), "the workspace");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B: 16 x 16 by 16 x 8, fp16, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two of four biased codes (c + 128) as fp16: the low pair or the high one.
__device__ __forceinline__ uint32_t code_pair(uint32_t biased, uint32_t select) {
  const uint32_t v = __byte_perm(biased, 0x64646464u, select);
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(v), __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t biased) { return code_pair(biased, 0x4140); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t biased) { return code_pair(biased, 0x4342); }

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 r = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(r);
}

template <int D>
struct KaShape {
  static constexpr int kStages = D <= 128 ? 4 : 3;
  static constexpr int kCtasPerSm = D <= 160 ? 3 : 2;
  static constexpr bool kQRegs = D <= 128;              // query operands in registers, else in shared memory
  static constexpr int kK16 = D / 64, kK8 = D / 32 % 2; // key chunks: 16 bytes a lane over 64 d, 8 over 32
  static constexpr int kV16 = D / 128, kV8 = D / 64 % 2, kV4 = D / 32 % 2;  // value chunks: 16, 8, 4 bytes a lane
  static constexpr int kKBytes = 16 * D, kVBytes = 16 * D;
  static constexpr int kStage = kKBytes + kVBytes;      // of a warp
  static constexpr int kRing = kStages * kStage;
  static constexpr int kQPitch = 2 * D + 16;            // bytes of a query row
  static constexpr int kOPitch = D + 4;                 // floats of a row of a warp's sums, over its ring
  static_assert(kKaRows * kOPitch * 4 <= kRing, "a warp's sums go over its ring");
  static constexpr int kOffQ = kKaWarps * kRing;
  static constexpr int kOffScale = kOffQ + kKaRows * kQPitch;          // float4 for each warp and stage
  static constexpr int kOffRow = kOffScale + kKaWarps * kStages * 16;  // fp32 for each row: query scale
  static constexpr int kOffMax = kOffRow + kKaRows * 4;                // [warps][rows] maxima, denominators
  static constexpr int kBytes = kOffMax + 2 * kKaWarps * kKaRows * 4;
};

// A request as the work is counted: its rows and steps.
struct KaRequest {
  int row0, fresh, len, held, tiles, steps;  // held: the tokens that its table row has room for
};
__device__ __forceinline__ KaRequest ka_request(const KvAttnParams& p, int r) {
  KaRequest q;
  const int a = p.cu[r], b = p.cu[r + 1], len = p.lens[r];
  const int64_t most = (int64_t)p.width << p.log_bs;
  q.row0 = a;
  q.fresh = a >= 0 && b > a && b <= p.rows ? b - a : 0;
  q.len = max(0, len);
  q.held = (int)min((int64_t)q.len, most);
  q.tiles = (int)(((int64_t)q.fresh * p.group + kKaRows - 1) / kKaRows);
  q.steps = max(1, (int)(((int64_t)q.held + kKaStep - 1) / kKaStep));
  return q;
}

// Its steps over all heads and tiles (0 behind the last request).
__device__ __forceinline__ int64_t ka_weight(const KvAttnParams& p, int r) {
  if (r >= p.n) return 0;
  const KaRequest q = ka_request(p, r);
  return (int64_t)q.tiles * q.steps * p.nk;
}

template <int D>
__global__ void __launch_bounds__(kKaThreads, KaShape<D>::kCtasPerSm) k_kv_attn(KvAttnParams p) {
  using S = KaShape<D>;
  extern __shared__ __align__(16) uint8_t ka_smem[];
  __shared__ int64_t s_part[kKaWarps];
  __shared__ int64_t s_cut[2], s_begin;
  __shared__ int s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();

  // ------------------------------------------------------------ the share
  int64_t total = 0;
  for (int r = tid; r < p.n; r += kKaThreads) total += ka_weight(p, r);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(~0u, total, k);
  if (lane == 0) s_part[warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kKaWarps; ++w) total += s_part[w];
  const int64_t share = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kKaMinPart);
  const int64_t raw[2] = {min(total, share * blockIdx.x), min(total, share * (blockIdx.x + 1))};
  if (tid == 0) s_cut[0] = raw[0], s_cut[1] = raw[1], s_first = p.n, s_begin = total;
  int64_t carry = 0;
  for (int r0 = 0; r0 < p.n && carry <= raw[1]; r0 += kKaThreads) {
    const int64_t w = ka_weight(p, r0 + tid);
    int64_t inc = w;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int64_t x = __shfl_up_sync(~0u, inc, k);
      if (lane >= k) inc += x;
    }
    __syncthreads();  // s_part, s_cut
    if (lane == 31) s_part[warp] = inc;
    __syncthreads();
    int64_t all = 0, before = carry;
    for (int k = 0; k < kKaWarps; ++k) {
      if (k < warp) before += s_part[k];
      all += s_part[k];
    }
    const int64_t begin = before + inc - w;
    if (w > 0) {
      const int steps = ka_request(p, r0 + tid).steps;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (raw[k] >= begin && raw[k] < begin + w) {
          const int64_t in = (raw[k] - begin) % steps;  // a cut near an end of a tile goes there
          const int64_t cut = in < kKaMinPart ? raw[k] - in : steps - in < kKaMinPart ? raw[k] - in + steps : raw[k];
          s_cut[k] = cut;
          if (k == 0) s_first = r0 + tid, s_begin = begin;
        }
    }
    carry += all;
  }
  __syncthreads();
  int64_t at = s_cut[0];
  const int64_t end = s_cut[1];
  int r = s_first;
  int64_t begin = s_begin;
  KaJoin join = {};
  float* parts = p.ws + (int64_t)kKaMaxCtas * (sizeof(KaJoin) / 4);
  bool first = true;

  uint8_t* ring = ka_smem + warp * S::kRing;
  const uint32_t ring_u = smem_u32(ring);
  float4* scales = reinterpret_cast<float4*>(ka_smem + S::kOffScale) + warp * S::kStages;
  float* s_qscale = reinterpret_cast<float*>(ka_smem + S::kOffRow);
  float* s_max = reinterpret_cast<float*>(ka_smem + S::kOffMax);
  float* s_den = s_max + kKaWarps * kKaRows;

  while (at < end) {
    // ---------------------------------------------------------- the next tile's steps [step0, step1)
    KaRequest rq = ka_request(p, r);
    while (at >= begin + (int64_t)rq.tiles * rq.steps * p.nk) {  // (ends: at < total, the last request's end)
      begin += (int64_t)rq.tiles * rq.steps * p.nk;
      rq = ka_request(p, ++r);
    }
    const int64_t item = (at - begin) / rq.steps;
    const int step0 = (int)(at - begin - item * rq.steps);
    const int step1 = (int)min((int64_t)rq.steps, step0 + (end - at));
    const int h = (int)(item / rq.tiles), tile = (int)(item - (int64_t)h * rq.tiles);
    const int tile_rows = (int)min((int64_t)kKaRows, (int64_t)rq.fresh * p.group - (int64_t)tile * kKaRows);
    const int64_t item_end = at - step0 + rq.steps;
    const int* table = p.table + (int64_t)r * p.width;
    const int my_steps = max(0, (step1 - step0 - warp + kKaWarps - 1) / kKaWarps);
    // the tokens that a row sees: those before its place behind the older ones
    auto sees = [&](int row) { return min(rq.held, rq.len - rq.fresh + (tile * kKaRows + row) / p.group + 1); };
    const int seen_by_all = sees(0);

    // ---------------------------------------------------------- copies
    // lane l looks up the blocks and scales of the warp's steps l, l + 32, ...
    int blk = -1;
    float4 sc;
    auto look_up = [&](int i0) {
      const int i = i0 + lane;
      blk = -1;
      sc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < my_steps) {
        const int token = (step0 + warp + kKaWarps * i) * kKaStep;
        const int b = token < rq.held ? table[token >> p.log_bs] : -1;
        if (b >= 0 && b < p.blocks) {
          blk = b;
          const int64_t bh = (int64_t)b * p.nk + h;
          const float v = fmaxf(p.vmax[bh] * (1.0f / 127.0f), 7.703719777548943e-34f);  // 2^-110 (keeps no NaN)
          const bool nan = !(p.vmax[bh] <= 3.4028234663852886e38f);
          sc.x = p.kmax[bh];
          sc.y = nan ? __uint_as_float(0x7FC00000u) : log2f(v);
          sc.z = nan ? 0.0f : __fdividef(1.0f, v);
          sc.w = 1.0f;
        }
      }
    };
    auto issue = [&](int i) {
      if (i < my_steps) {
        if ((i & 31) == 0) look_up(i);
        const int stage = i % S::kStages;
        const int b = __shfl_sync(~0u, blk, i & 31);
        if (lane == (i & 31)) scales[stage] = sc;
        if (b >= 0) {
          const int token = (step0 + warp + kKaWarps * i) * kKaStep;
          const int64_t base = ((((int64_t)b * p.nk + h) << p.log_bs) + (token & ((1 << p.log_bs) - 1))) * D;
          const uint32_t dst = ring_u + stage * S::kStage;
          const int8_t* k = p.kc + base + g * D;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int c = 0; c < S::kK16; ++c)
              cp_async16(dst + ((j * S::kK16 + c) * 32 + lane) * 16, k + j * 8 * D + 64 * c + 16 * t);
            if constexpr (S::kK8 != 0)
              cp_async_small<8>(dst + 2 * S::kK16 * 512 + (j * 32 + lane) * 8, k + j * 8 * D + 64 * S::kK16 + 8 * t);
          }
          const int8_t* v = p.vc + base + 2 * t * D;
          const uint32_t vd = dst + S::kKBytes;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int8_t* vr = v + ((u & 1) + 8 * (u >> 1)) * D;
#pragma unroll
            for (int c = 0; c < S::kV16; ++c) cp_async16(vd + ((u * S::kV16 + c) * 32 + lane) * 16, vr + 128 * c + 16 * g);
            if constexpr (S::kV8 != 0)
              cp_async_small<8>(vd + 4 * S::kV16 * 512 + (u * 32 + lane) * 8, vr + 128 * S::kV16 + 8 * g);
            if constexpr (S::kV4 != 0)
              cp_async_small<4>(vd + 4 * S::kV16 * 512 + 4 * S::kV8 * 256 + (u * 32 + lane) * 4,
                                vr + 128 * S::kV16 + 64 * S::kV8 + 4 * g);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) issue(i);

    // ---------------------------------------------------------- queries
    // 8 lanes to a row: its largest exponent, then fp16 (rows behind the tile's last: zeros)
    {
      const int row = tid >> 3, part = tid & 7;
      constexpr int kEach = D / 8;  // elements of a lane, in pairs
      uint32_t x[kEach / 2];
      const bool there = row < tile_rows;
      const int64_t idx = (int64_t)tile * kKaRows + row;
      const uint32_t* src = nullptr;
      if (there) {
        const int64_t i = idx / p.group;
        src = reinterpret_cast<const uint32_t*>(p.q + (rq.row0 + i) * p.ldq + ((int64_t)h * p.group + (idx - i * p.group)) * D) +
              part * (kEach / 2);
      }
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kEach / 2; ++j) {
        x[j] = there ? src[j] : 0u;
        top = max(top, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
      }
#pragma unroll
      for (int k = 1; k < 8; k *= 2) top = max(top, __shfl_xor_sync(~0u, top, k));
      // the exponent of 2^(14 - e), e that of the largest element (kept where both powers are normal numbers)
      const int e = min(max((int)(top >> 7) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      uint32_t* dst = reinterpret_cast<uint32_t*>(ka_smem + S::kOffQ + row * S::kQPitch) + part * (kEach / 2);
#pragma unroll
      for (int j = 0; j < kEach / 2; ++j) dst[j] = pack_half2(bf16lo(x[j]) * up, bf16hi(x[j]) * up);
      if (part == 0) s_qscale[row] = p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    }
    __syncthreads();
    // the operands of k-step s of a 64-wide chunk c: words 2 s and 2 s + 1 of a lane's 16 elements, rows g and g + 8
    const uint8_t* qrow = ka_smem + S::kOffQ + g * S::kQPitch;
    constexpr int kChunks = S::kK16 + S::kK8;
    uint32_t qa[S::kQRegs ? D / 16 : 1][4];
    auto load_q = [&](int chunk, int s, uint32_t (&a)[4]) {  // a wide chunk's lane holds 16 elements, the narrow one's 8
      const int off = chunk < S::kK16 ? chunk * 128 + 32 * t + 8 * s : S::kK16 * 128 + 16 * t + 8 * s;
      const uint2 x = *reinterpret_cast<const uint2*>(qrow + off), y = *reinterpret_cast<const uint2*>(qrow + 8 * S::kQPitch + off);
      a[0] = x.x, a[1] = y.x, a[2] = x.y, a[3] = y.y;
    };
    if constexpr (S::kQRegs) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int s = 0; s < (c < S::kK16 ? 4 : 2); ++s) load_q(c, s, qa[4 * c + s]);
    }
    const float qs0 = s_qscale[g], qs1 = s_qscale[g + 8];
    const int see0 = g < tile_rows ? sees(g) : 0x7FFFFFFF, see1 = g + 8 < tile_rows ? sees(g + 8) : 0x7FFFFFFF;

    // ---------------------------------------------------------- the steps
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, b0 = -kKaLift, b1 = -kKaLift, l0 = 0.0f, l1 = 0.0f;

    for (int i = 0; i < my_steps; ++i) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      const int stage = i % S::kStages;
      const uint8_t* sk = ring + stage * S::kStage;
      const float4 scale = scales[stage];
      float c[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.0f;
#pragma unroll
      for (int ch = 0; ch < S::kK16; ++ch) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 w = *reinterpret_cast<const uint4*>(sk + ((j * S::kK16 + ch) * 32 + lane) * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t x = ws[s] ^ 0x80808080u;
            if constexpr (S::kQRegs) {
              mma_f16(c[j], qa[4 * ch + s], codes_lo(x), codes_hi(x));
            } else {
              uint32_t a[4];
              load_q(ch, s, a);
              mma_f16(c[j], a, codes_lo(x), codes_hi(x));
            }
          }
        }
      }
      if constexpr (S::kK8 != 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 w = *reinterpret_cast<const uint2*>(sk + 2 * S::kK16 * 512 + (j * 32 + lane) * 8);
          const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t x = ws[s] ^ 0x80808080u;
            if constexpr (S::kQRegs) {
              mma_f16(c[j], qa[4 * S::kK16 + s], codes_lo(x), codes_hi(x));
            } else {
              uint32_t a[4];
              load_q(S::kK16, s, a);
              mma_f16(c[j], a, codes_lo(x), codes_hi(x));
            }
          }
        }
      }
      // scores in powers of two, the block's value scale among them
      const float f0 = qs0 * scale.x, f1 = qs1 * scale.x;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[j][0] = fmaf(c[j][0], f0, scale.y), c[j][1] = fmaf(c[j][1], f0, scale.y);
        c[j][2] = fmaf(c[j][2], f1, scale.y), c[j][3] = fmaf(c[j][3], f1, scale.y);
      }
      const int token = (step0 + warp + kKaWarps * i) * kKaStep;
      if (token + kKaStep > seen_by_all || scale.w == 0.0f) {  // (scale.w: there is no such block)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at_token = token + 8 * j + 2 * t + e;
            if (at_token >= see0 || scale.w == 0.0f) c[j][e] = -INFINITY;
            if (at_token >= see1 || scale.w == 0.0f) c[j][2 + e] = -INFINITY;
          }
      }
      float x0 = fmaxf(fmaxf(c[0][0], c[0][1]), fmaxf(c[1][0], c[1][1]));
      float x1 = fmaxf(fmaxf(c[0][2], c[0][3]), fmaxf(c[1][2], c[1][3]));
      if (__any_sync(~0u, x0 > m0 || x1 > m1)) {
        x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 1)), x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 2)), x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 2));
        x0 = fmaxf(x0, m0), x1 = fmaxf(x1, m1);
        const float a0 = x0 == m0 ? 1.0f : exp2_fast(m0 - x0), a1 = x1 == m1 ? 1.0f : exp2_fast(m1 - x1);
        m0 = x0, m1 = x1;
        b0 = (m0 == -INFINITY ? 0.0f : m0) - kKaLift, b1 = (m1 == -INFINITY ? 0.0f : m1) - kKaLift;
        l0 *= a0, l1 *= a1;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) o[k][0] *= a0, o[k][1] *= a0, o[k][2] *= a1, o[k][3] *= a1;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[j][0] = exp2_fast(c[j][0] - b0), c[j][1] = exp2_fast(c[j][1] - b0);
        c[j][2] = exp2_fast(c[j][2] - b1), c[j][3] = exp2_fast(c[j][3] - b1);
      }
      l0 = fmaf((c[0][0] + c[0][1]) + (c[1][0] + c[1][1]), scale.z, l0);
      l1 = fmaf((c[0][2] + c[0][3]) + (c[1][2] + c[1][3]), scale.z, l1);
      const uint32_t pa[4] = {pack_half2(c[0][0], c[0][1]), pack_half2(c[0][2], c[0][3]), pack_half2(c[1][0], c[1][1]),
                              pack_half2(c[1][2], c[1][3])};
      // four columns' operands out of a word of each of four tokens
      const uint8_t* sv = sk + S::kKBytes;
      auto columns = [&](float (*acc)[4], uint32_t wa, uint32_t wb, uint32_t wc, uint32_t wd) {
        const uint32_t x = __byte_perm(wa, wb, 0x5140) ^ 0x80808080u, y = __byte_perm(wc, wd, 0x5140) ^ 0x80808080u;
        mma_f16(acc[0], pa, codes_lo(x), codes_lo(y));
        mma_f16(acc[1], pa, codes_hi(x), codes_hi(y));
        const uint32_t z = __byte_perm(wa, wb, 0x7362) ^ 0x80808080u, w = __byte_perm(wc, wd, 0x7362) ^ 0x80808080u;
        mma_f16(acc[2], pa, codes_lo(z), codes_lo(w));
        mma_f16(acc[3], pa, codes_hi(z), codes_hi(w));
      };
#pragma unroll
      for (int ch = 0; ch < S::kV16; ++ch) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = *reinterpret_cast<const uint4*>(sv + ((u * S::kV16 + ch) * 32 + lane) * 16);
        columns(o + 16 * ch, w[0].x, w[1].x, w[2].x, w[3].x);
        columns(o + 16 * ch + 4, w[0].y, w[1].y, w[2].y, w[3].y);
        columns(o + 16 * ch + 8, w[0].z, w[1].z, w[2].z, w[3].z);
        columns(o + 16 * ch + 12, w[0].w, w[1].w, w[2].w, w[3].w);
      }
      if constexpr (S::kV8 != 0) {
        uint2 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = *reinterpret_cast<const uint2*>(sv + 4 * S::kV16 * 512 + (u * 32 + lane) * 8);
        columns(o + 16 * S::kV16, w[0].x, w[1].x, w[2].x, w[3].x);
        columns(o + 16 * S::kV16 + 4, w[0].y, w[1].y, w[2].y, w[3].y);
      }
      if constexpr (S::kV4 != 0) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          w[u] = *reinterpret_cast<const uint32_t*>(sv + 4 * S::kV16 * 512 + 4 * S::kV8 * 256 + (u * 32 + lane) * 4);
        columns(o + 16 * S::kV16 + 8 * S::kV8, w[0], w[1], w[2], w[3]);
      }
      __syncwarp();  // scales[stage] has been read by all
      issue(i + S::kStages - 1);
    }
    cp_async_wait<0>();

    // ---------------------------------------------------------- the four warps' sums
    l0 += __shfl_xor_sync(~0u, l0, 1), l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2), l1 += __shfl_xor_sync(~0u, l1, 2);
    if (t == 0) {
      s_max[warp * kKaRows + g] = m0, s_max[warp * kKaRows + g + 8] = m1;
      s_den[warp * kKaRows + g] = l0, s_den[warp * kKaRows + g + 8] = l1;
    }
    __syncthreads();
    float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kKaWarps; ++w) top0 = fmaxf(top0, s_max[w * kKaRows + g]), top1 = fmaxf(top1, s_max[w * kKaRows + g + 8]);
    const float a0 = m0 == top0 ? 1.0f : exp2_fast(m0 - top0), a1 = m1 == top1 ? 1.0f : exp2_fast(m1 - top1);
    {
      // columns: lane t of a wide chunk holds 32 successive ones, 16 in tile order from row 2 t, 16 from 2 t + 1
      float* mine = reinterpret_cast<float*>(ring);
      auto put = [&](int first_tile, int width, int d0) {
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < width; i += 4) {
            const int col = d0 + width * (2 * t + e) + i;
            *reinterpret_cast<float4*>(mine + g * S::kOPitch + col) =
                make_float4(o[first_tile + i][e] * a0, o[first_tile + i + 1][e] * a0, o[first_tile + i + 2][e] * a0, o[first_tile + i + 3][e] * a0);
            *reinterpret_cast<float4*>(mine + (g + 8) * S::kOPitch + col) =
                make_float4(o[first_tile + i][2 + e] * a1, o[first_tile + i + 1][2 + e] * a1, o[first_tile + i + 2][2 + e] * a1,
                            o[first_tile + i + 3][2 + e] * a1);
          }
      };
#pragma unroll
      for (int ch = 0; ch < S::kV16; ++ch) put(16 * ch, 16, 128 * ch);
      if constexpr (S::kV8 != 0) put(16 * S::kV16, 8, 128 * S::kV16);
      if constexpr (S::kV4 != 0) put(16 * S::kV16 + 8 * S::kV8, 4, 128 * S::kV16 + 64 * S::kV8);
    }
    __syncthreads();
    const bool whole = step0 == 0 && step1 == rq.steps;
    const int slot = 2 * (int)blockIdx.x + (first ? 0 : 1);
    {
      const int row = tid >> 3, part = tid & 7;
      float top = -INFINITY, den = 0.0f;
#pragma unroll
      for (int w = 0; w < kKaWarps; ++w) top = fmaxf(top, s_max[w * kKaRows + row]);
#pragma unroll
      for (int w = 0; w < kKaWarps; ++w) {
        const float m = s_max[w * kKaRows + row];
        den += s_den[w * kKaRows + row] * (m == top ? 1.0f : exp2_fast(m - top));
      }
      const float inv = den == 0.0f ? 0.0f : 1.0f / den;  // a row that sees nothing is 0
      const int64_t idx = (int64_t)tile * kKaRows + row, i = idx / p.group;
      uint16_t* out = p.o + (rq.row0 + i) * p.ldo + ((int64_t)h * p.group + (idx - i * p.group)) * D;
      float* part_at = parts + slot * ka_part_floats(D);
      for (int col = 4 * part; col < D; col += 32) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kKaWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(ka_smem + w * S::kRing + (row * S::kOPitch + col) * 4);
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        if (!whole) {
          *reinterpret_cast<float4*>(part_at + 2 * kKaRows + row * D + col) = v;
        } else if (row < tile_rows) {
          *reinterpret_cast<uint2*>(out + col) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        }
      }
      if (!whole && part == 0) part_at[row] = top, part_at[kKaRows + row] = den;
    }
    if (step0 == 0 && step1 < rq.steps) {
      join.parts = (int)((item_end - kKaMinPart) / share) - (int)blockIdx.x + 1;
      join.slot = slot;
      join.row0 = rq.row0;
      join.head = h;
      join.rows = tile_rows;
      join.tile = tile;
    }
    first = false;
    at += step1 - step0;
    __syncthreads();  // the rings and the rows' sums have been read
  }
  if (tid == 0) reinterpret_cast<KaJoin*>(p.ws)[blockIdx.x] = join;
}

// The parts of the tile that begins in CTA blockIdx.x of the launch before and goes on in the next ones, in
// order: four rows to a CTA (blockIdx.y), a warp each.
template <int D>
__global__ void __launch_bounds__(128) k_kv_attn_join(KvAttnParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const KaJoin join = reinterpret_cast<const KaJoin*>(p.ws)[blockIdx.x];
  const int lane = threadIdx.x & 31, row = 4 * blockIdx.y + (threadIdx.x >> 5);
  if (join.parts == 0 || row >= join.rows) return;
  const float* parts = p.ws + (int64_t)kKaMaxCtas * (sizeof(KaJoin) / 4);
  // the first part is where it says, the others are the first ones of the CTAs that follow
  auto at = [&](int k) { return parts + (int64_t)(k == 0 ? join.slot : 2 * ((int)blockIdx.x + k)) * ka_part_floats(D); };
  float top = -INFINITY;
  for (int k = lane; k < join.parts; k += 32) top = fmaxf(top, at(k)[row]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
  float v[D / 32], den = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < join.parts; ++k) {
    const float* part = at(k);
    const float m = part[row], a = m == top ? 1.0f : exp2_fast(m - top);
    den = fmaf(part[kKaRows + row], a, den);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) v[j] = fmaf(part[2 * kKaRows + row * D + 32 * j + lane], a, v[j]);
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  const int64_t idx = (int64_t)join.tile * kKaRows + row, i = idx / p.group;
  uint16_t* out = p.o + (join.row0 + i) * p.ldo + ((int64_t)join.head * p.group + (idx - i * p.group)) * D;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) out[32 * j + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j] * inv));
}

}  // namespace gbmlp
