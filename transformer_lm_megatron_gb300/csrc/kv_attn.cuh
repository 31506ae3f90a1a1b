// Attention of each request's new tokens over its cached keys and values (8-bit codes, a maximum
// for each block and head: kv_cache.cuh), for few new tokens.
//
//   O = softmax(scale Q K^T) V,  K = Kc Kmax / 127,  V = Vc Vmax / 127
//
// HBM bounds it: a code is read once and meets 4 * rows operations, rows = new tokens * query heads
// of a key head.  What counts is that every SM has reads in flight all the time and that a
// code becomes a matrix operand in few instructions:
//   - Work is counted in steps of 16 tokens, over all requests, heads and tiles of rows, and cut
//     into equal shares, one for each CTA that fits on the GPU, wherever that falls: a long request
//     spreads over all SMs, a ragged batch leaves none idle.  A tile that ends up with several
//     CTAs leaves its parts (fp32 sums, base and denominator of each row) in the workspace, and
//     k_kv_attn_join adds them up in order, so results do not change from run to run.
//   - Each warp takes every fourth step of a share, alone.  Its lanes read straight into registers the
//     very bytes that they feed to the tensor cores, so there is no barrier in the loop and no
//     transposition: reductions may run over d and over tokens in any order, so a lane's 16 bytes of
//     a key are operands of four successive MMAs, and its 16 bytes of four tokens' values those of eight.  A step's
//     registers are filled again as soon as they are used up; one bulk prefetch of a step's keys and one of its values,
//     two steps ahead, have brought them to L2 by then.  (A ring in shared memory took 378 us where this takes 276 for 64
//     requests of 12000 to 16384 tokens: twice the shared-memory traffic.  Four steps ahead fill the queues to HBM, which
//     every tile's first look-ups then wait behind: 58 us for 55 for one request of 131077.)
//   - Both products are taken transposed, S^T = K Q^T and O^T += V^T P^T: the codes are the operand with 16
//     rows, the query rows the one with 8, so that eight query rows waste nothing and more of them
//     (NT times 8) use a converted code again.  P^T changes places within a warp (movmatrix).
//   - Codes become fp16 exactly (1024 + (c + 128) by a byte permutation, minus 1152): 5 instructions
//     for 4 keys, 6 for 4 values.  mma.sync, not tcgen05: operands come from registers, where
//     the codes are converted, and there are as few as 8 rows where tcgen05 wants 128 by 16 out of shared memory.
//   - Queries go to fp16 with a power of two for each row that brings its largest element below
//     2^15: exact but for elements under 2^-29 of it.
//   - A block's value scale goes into the exponent: p' = exp2(s + log2(vscale) - base) is the operand of the second
//     product, rounded to fp16 (2^-11 of a weight where bf16 takes 2^-8), whatever the scales; the denominator adds
//     p' / vscale in fp32.  The base is the maximum of a row's first step less 10, and moves (and with it all sums so far)
//     only where a p' would pass 2^15.5: with random scores the first step's is nearly always near enough, where a running
//     maximum moves in half of a part's steps (68 us for 57 with 40 rows).  fp16 so holds a weight above
//     2^-24 of the largest in full precision, and below it to 2^-35 of the largest.  Where scales lie 2^100 apart see kKaFar.
// Measured (graph replay, inputs rotated; the bytes at the copy rate in brackets): 64 requests of 12000 to 16384 tokens,
// 8 key heads of 128, 64 query heads 276 us (275); one request of 131077 tokens 51 us (40); 48 of 100 to 16384 tokens 56 us
// (42); 8 of 1500 to 2048, 128 heads of 160 103 us (88).  What the shorter ones lose, 11 us, is the launch, a chain of three
// reads (lengths, table, codes) that nothing hides, the last warps' lag and the joining launch.  From 9 rows on the
// instructions bound it: 16 requests of 3000 to 9000 tokens, 4 key heads, 8 rows 26 us, 16 31 us, 40 57 us (14).
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace gbmlp {

constexpr int kKaWarps = 4;
constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaStep = 16;        // tokens of a step
constexpr int kKaWsRows = 19456;   // of the workspace, d + 2 floats each
constexpr int kKaMinPart = 8;      // steps: no tile is cut nearer than this to either end (24: 13 us for 6 with 137 tokens)
constexpr int kKaTileCost = 16;    // steps that beginning and ending a tile takes as long as (8: 64 us for 59 on a ragged batch)
constexpr float kKaLift = 10.0f;   // a row's base is that far below its first maximum
constexpr float kKaMost = 15.5f;   // p' is at most 2^15.5
constexpr float kKaLowest = -3.0e38f;
// 2^-100: of weights whose block's scale is that far below the tile's largest (a block of zeros beside values above 2^20, say),
// the denominator takes exp2(s - base) as the square of its root, which stays in fp32: p' may be 0 with weights that count.  Bases
// may lie as far apart, so every factor between two of them is taken as a square too.
constexpr float kKaFar = 7.888609052210118e-31f;
constexpr int kKaAhead = 2;        // how many of its steps ahead a warp asks for codes in L2
constexpr int kKaJoinWarps = 16;

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

// The workspace: two descriptors for each CTA, then two parts (bases, denominators, sums): of the tile that
// the CTA begins in the middle of, and of the one that it begins and another one goes on with.
struct KaJoin {
  int first, parts, row0, head, tile, rows, pad[2];  // the CTA that began the tile; 0 parts: there is no such tile
};
__host__ __device__ constexpr int64_t ka_part_floats(int rows, int d) { return (int64_t)rows * (d + 2); }
__host__ __device__ constexpr int ka_max_ctas(int rows, int d) {
  return (int)((int64_t)kKaWsRows * (d + 2) / (2 * (int64_t)(sizeof(KaJoin) / 4) + 2 * ka_part_floats(rows, d)));
}

// 16, 8 or 4 bytes that one lane of the SM reads, once.
__device__ __forceinline__ uint4 ld_once16(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_once8(const int8_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_once4(const int8_t* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const int8_t* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B: 16 x 16 by 16 x 8, fp16, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&b)[2]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}

// An 8 x 8 matrix of 16-bit elements, two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// Heads of size D, tiles of 8 NT rows.
template <int D, int NT>
struct KaShape {
  static constexpr int kRows = 8 * NT;
  // As many CTAs as leave a thread the registers that it needs: 64 long requests with heads of 128 take 276 us with 3, 287 us with 4
  // and spills; 16 query heads to a key head (32 requests of 4000 to 8000 tokens) 47 us with 2, 54 with 3 and spills; heads of 32
  // 49 us with 4, 51 with 3; heads of 64 68 us with 3, 70 with 4; heads of 192, 224 and 256 53, 62 and 67 us with 2, 57, 71 and
  // 82 with 3 and spills.  Tiles of 16 rows of heads of 224 and 256 need more than the 255 that a thread can have (they spill 76 and 312
  // bytes, with 1 CTA as with 2): 83 and 90 us with 16 query heads, where heads of 192 without spills take 67.
  static constexpr int kCtasPerSm = NT == 1 ? (D <= 32 ? 4 : D <= 160 ? 3 : 2) : 2;
  // Query operands in registers where they are 32 of them or fewer, else in shared memory (the 16 query heads: 47.3 us for 48.3).
  static constexpr bool kQRegs = NT * D <= 256;
  static constexpr int kK16 = D / 64, kK8 = D / 32 % 2; // key chunks: 16 bytes a lane over 64 d, 8 over 32
  static constexpr int kV16 = D / 128, kV8 = D / 64 % 2, kV4 = D / 32 % 2;  // value chunks: 16, 8, 4 bytes a lane
  // Steps that a warp works on at once: what a step costs whatever its size counts for small heads (heads of 32 49 us for
  // 62, of 64 68 for 71), not for 128 (276 us either way, 102 us become 108 for 160).
  static constexpr int kAtOnce = D <= 64 ? 2 : 1;
  // Each warp's largest value scale so far: in a register where there are more than 168 of them (40 rows 57.2 us for 59.2), else in
  // shared memory (heads of 160 102.4 us for 105.6).
  static constexpr bool kTopReg = NT > 1;
  static constexpr int kQPitch = 2 * D + 16;            // bytes of a query row
  static constexpr int kOPitch = D + 4;                 // floats of a row of sums
  static constexpr int kOffPlace = 0;                                 // KaPlace of 64 steps of each warp
  static constexpr int kOffQ = kOffPlace + kKaWarps * 64 * 16;
  static constexpr int kOffO = kOffQ + kRows * kQPitch;
  static constexpr int kOffRow = kOffO + kKaWarps * kRows * kOPitch * 4;  // query scale of each row
  static constexpr int kOffMax = kOffRow + kRows * 4;                 // [warps][rows] bases, denominators
  static constexpr int kOffTop = kOffMax + 2 * kKaWarps * kRows * 4;  // each warp's largest value scale in the tile so far
  static constexpr int kBytes = kOffTop + kKaWarps * 4;
};

// Where a step's tokens are, in units of 16 tokens of a head from the pools' beginnings (complemented if their
// block is not there: what it says is read all the same, and masked), and their scales.  vinv < 0: see kKaFar.
struct __align__(16) KaPlace {
  int unit;
  float kscale, vlog, vinv;
};

// A request as the work is counted: its rows, and its steps.
struct KaRequest {
  int row0, fresh, len, held, tiles, steps;  // held: the tokens that its table row has room for
  __device__ __forceinline__ int64_t weight(int nk) const { return (int64_t)tiles * nk * (steps + kKaTileCost); }
};
template <int ROWS>
__device__ __forceinline__ KaRequest ka_request(const KvAttnParams& p, int r) {
  KaRequest q;
  const int a = p.cu[r], b = p.cu[r + 1], len = p.lens[r];
  const int64_t most = (int64_t)p.width << p.log_bs;
  q.row0 = a;
  q.fresh = a >= 0 && b > a && b <= p.rows ? b - a : 0;
  q.len = max(0, len);
  q.held = (int)min((int64_t)q.len, most);
  q.tiles = (int)(((int64_t)q.fresh * p.group + ROWS - 1) / ROWS);
  q.steps = max(1, (int)(((int64_t)q.held + kKaStep - 1) / kKaStep));
  return q;
}

// The steps [step0, step1) of a tile that a CTA takes.
struct KaItem {
  KaRequest rq;
  int r, h, tile, step0, step1, my_steps;
  int64_t end;  // of the tile in the work
};

// a / b, a >= 0, b > 0: in 32 bits where they fit.
__device__ __forceinline__ int64_t ka_div(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int D, int NT>
__global__ void __launch_bounds__(kKaThreads, KaShape<D, NT>::kCtasPerSm) k_kv_attn(KvAttnParams p) {
  using S = KaShape<D, NT>;
  constexpr int ROWS = S::kRows;
  extern __shared__ __align__(16) uint8_t ka_smem[];
  __shared__ int64_t s_part[kKaWarps];
  __shared__ int64_t s_cut[2], s_begin;
  __shared__ int s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();

  // ------------------------------------------------------------ the share
  // (the requests in groups of 128: the first group's sums are kept, a further one's are worked out again)
  int64_t weight = 0, inc = 0, total = 0;
  int steps = 1;
  auto group_sums = [&](int r0) {  // weight, its inclusive sum, and the group's total
    weight = 0;
    if (r0 + tid < p.n) {
      const KaRequest q = ka_request<ROWS>(p, r0 + tid);
      weight = q.weight(p.nk);
      steps = q.steps;
    }
    inc = weight;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int64_t x = __shfl_up_sync(~0u, inc, k);
      if (lane >= k) inc += x;
    }
    if (lane == 31) s_part[warp] = inc;
    __syncthreads();
    int64_t all = 0;
    for (int k = 0; k < kKaWarps; ++k) {
      if (k < warp) inc += s_part[k];
      all += s_part[k];
    }
    return all;
  };
  if (p.n > kKaThreads) {
    for (int r = kKaThreads + tid; r < p.n; r += kKaThreads) total += ka_request<ROWS>(p, r).weight(p.nk);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(~0u, total, k);
    if (lane == 0) s_part[warp] = total;
    __syncthreads();
    total = 0;
    for (int k = 0; k < kKaWarps; ++k) total += s_part[k];
    __syncthreads();
  }
  total += group_sums(0);
  const int64_t share = max(ka_div(total + gridDim.x - 1, gridDim.x), (int64_t)kKaMinPart);
  const int64_t raw[2] = {min(total, share * blockIdx.x), min(total, share * (blockIdx.x + 1))};
  if (tid == 0) s_cut[0] = raw[0], s_cut[1] = raw[1], s_first = p.n, s_begin = total;
  __syncthreads();
  int64_t carry = 0;
  for (int r0 = 0;;) {
    const int64_t begin = carry + inc - weight;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (raw[k] >= begin && raw[k] < begin + weight) {
        // a tile's cost comes before its steps; a cut near an end of a tile goes there
        const int64_t ahead = raw[k] - begin;
        const int in = (int)(ahead - ka_div(ahead, steps + kKaTileCost) * (steps + kKaTileCost)), step = in - kKaTileCost;
        s_cut[k] = raw[k] + (step < kKaMinPart ? -in : steps - step < kKaMinPart ? steps - step : 0);
        if (k == 0) s_first = r0 + tid, s_begin = begin;
      }
    for (int k = 0; k < kKaWarps; ++k) carry += s_part[k];
    __syncthreads();
    r0 += kKaThreads;
    if (r0 >= p.n || carry > raw[1]) break;
    group_sums(r0);
  }
  int64_t at = s_cut[0];
  const int64_t end = s_cut[1];
  KaJoin* joins = reinterpret_cast<KaJoin*>(p.ws) + 2 * blockIdx.x;
  if (tid < 2) joins[tid].parts = 0;
  if (at >= end) return;
  float* parts = p.ws + 2 * (int64_t)gridDim.x * (sizeof(KaJoin) / 4);
  int64_t begin = s_begin;

  KaPlace* places = reinterpret_cast<KaPlace*>(ka_smem + S::kOffPlace) + warp * 64;
  float* s_qscale = reinterpret_cast<float*>(ka_smem + S::kOffRow);
  float* s_max = reinterpret_cast<float*>(ka_smem + S::kOffMax);
  float* s_den = s_max + kKaWarps * ROWS;
  float* s_o = reinterpret_cast<float*>(ka_smem + S::kOffO);
  uint32_t* s_top = reinterpret_cast<uint32_t*>(ka_smem + S::kOffTop);

  // The tile that `at` is in (at < end, so there is one).
  KaItem it;
  it.r = s_first;
  it.rq = ka_request<ROWS>(p, it.r);
  auto next_item = [&]() {
    while (at >= begin + it.rq.weight(p.nk)) {
      begin += it.rq.weight(p.nk);
      it.rq = ka_request<ROWS>(p, ++it.r);
    }
    const int whole = it.rq.steps + kKaTileCost;
    const int64_t item = ka_div(at - begin, whole);
    it.end = begin + (item + 1) * whole;
    it.h = (int)ka_div(item, it.rq.tiles);
    it.tile = (int)(item - (int64_t)it.h * it.rq.tiles);
    it.step0 = max(0, (int)(at - (it.end - it.rq.steps)));
    it.step1 = it.rq.steps - (int)max((int64_t)0, it.end - end);
    it.my_steps = max(0, (it.step1 - it.step0 - warp + kKaWarps - 1) / kKaWarps);
  };

  // ------------------------------------------------------------ reads
  constexpr int U = S::kAtOnce;
  // Lane l looks up the place of the warp's step i0 + l: `find` where the codes are, and asks for the block's
  // scales (and, at a tile's beginning, for the first few steps' codes in L2); `settle` waits for them.
  int found;
  float most_k, most_v;
  uint32_t top_so_far = 0;
  auto find = [&](int i0) {
    const int i = i0 + lane;
    found = ~0, most_k = most_v = 0.0f;
    if (i < it.my_steps) {
      const int token = (it.step0 + warp + kKaWarps * i) * kKaStep;
      const int b = token < it.rq.held ? p.table[(int64_t)it.r * p.width + (token >> p.log_bs)] : -1;
      if (b >= 0 && b < p.blocks) {
        const int64_t bh = (int64_t)b * p.nk + it.h;
        found = (int)(bh << (p.log_bs - 4)) + ((token & ((1 << p.log_bs) - 1)) >> 4);
        most_k = p.kmax[bh], most_v = p.vmax[bh];
        if (i < kKaAhead * U) {
          prefetch_l2(p.kc + (int64_t)found * (16 * D), 16 * D);
          prefetch_l2(p.vc + (int64_t)found * (16 * D), 16 * D);
        }
      }
    }
  };
  auto settle = [&](int i0) {
    // (a block of zeros has no scale: the smallest that another one can have, so that it moves the base last)
    const float v = fmaxf(most_v, kKvTiny) * (1.0f / 127.0f);
    const bool fine = most_v <= 3.4028234663852886e38f;
    // the largest scale that p' of these steps may meet in the base
    uint32_t top = __reduce_max_sync(~0u, fine ? __float_as_uint(v) : 0u);
    if (i0 > 0) top = max(top, S::kTopReg ? top_so_far : s_top[warp]);
    top_so_far = top;
    const bool far = v < __uint_as_float(top) * kKaFar;
    __syncwarp();  // the places that these take the slots of, and s_top, have been read
    places[(i0 + lane) & 63] =
        KaPlace{found, most_k, fine ? log2f(v) : __uint_as_float(0x7FC00000u), !fine ? 0.0f : far ? -1.0f : __fdividef(1.0f, v)};
    if (!S::kTopReg && lane == 0) s_top[warp] = top;
    __syncwarp();
  };
  auto offset = [&](int unit) { return (int64_t)max(unit, ~unit) * (16 * D); };
  // asks for the codes of steps i .. i + U - 1 in L2
  auto ahead = [&](int i) {
    if (i >= it.my_steps) return;
    if ((i & 31) == 0) find(i), settle(i);
    if (lane < 2 * U) prefetch_l2(((lane & 1) == 0 ? p.kc : p.vc) + offset(places[(i + (lane >> 1)) & 63].unit), 16 * D);
  };
  uint4 k16[U][S::kK16 ? S::kK16 : 1][2], v16[U][S::kV16 ? S::kV16 : 1][4];
  uint2 k8[U][2], v8[U][4];
  uint32_t v4[U][4];
  KaPlace place[U];
  int64_t off[U];
  auto load_keys = [&]() {
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int8_t* k = p.kc + off[x] + g * D + 16 * t;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int c = 0; c < S::kK16; ++c) k16[x][c][j] = ld_once16(k + j * 8 * D + 64 * c);
        if constexpr (S::kK8 != 0) k8[x][j] = ld_once8(k + j * 8 * D + 64 * S::kK16 - 8 * t);
      }
    }
  };
  auto load_values = [&]() {
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int8_t* v = p.vc + off[x] + 2 * t * D;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int8_t* row = v + ((u & 1) + 8 * (u >> 1)) * D;
#pragma unroll
        for (int c = 0; c < S::kV16; ++c) v16[x][c][u] = ld_once16(row + 128 * c + 16 * g);
        if constexpr (S::kV8 != 0) v8[x][u] = ld_once8(row + 128 * S::kV16 + 8 * g);
        if constexpr (S::kV4 != 0) v4[x][u] = ld_once4(row + 128 * S::kV16 + 64 * S::kV8 + 4 * g);
      }
    }
  };
  // 16 lanes to a query row, 8 rows at a time (those behind the tile's last: zeros)
  uint32_t qx[NT][D / 32];
  auto tile_rows_of = [&](const KaItem& x) { return (int)min((int64_t)ROWS, (int64_t)x.rq.fresh * p.group - (int64_t)x.tile * ROWS); };
  auto load_queries = [&]() {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int row = 8 * q + (tid >> 4), idx = it.tile * ROWS + row, i = idx / p.group;
      const bool there = row < tile_rows_of(it);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (it.rq.row0 + i) * p.ldq + ((int64_t)it.h * p.group + (idx - i * p.group)) * D);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) qx[q][j] = there ? src[16 * j + (tid & 15)] : 0u;
    }
  };
  auto begin_item = [&]() {
    next_item();
    load_queries();
    if (it.my_steps == 0) return;
    find(0);
#pragma unroll
    for (int x = 0; x < U; ++x) off[x] = offset(__shfl_sync(~0u, found, x));
    load_keys();
    load_values();
    settle(0);
#pragma unroll
    for (int x = 0; x < U; ++x) place[x] = places[x];
  };
  begin_item();

  while (true) {
    const int tile_rows = tile_rows_of(it);
    // the tokens that a row sees: those before its place behind the older ones
    auto sees = [&](int row) { return min(it.rq.held, it.rq.len - it.rq.fresh + (it.tile * ROWS + row) / p.group + 1); };
    // the warp's steps from here on have tokens that some row does not see
    const int from = sees(0) / kKaStep - it.step0 - warp, first_masked = from <= 0 ? 0 : (from + kKaWarps - 1) / kKaWarps;

    // ---------------------------------------------------------- queries
    // to fp16, by the largest element's exponent
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int row = 8 * q + (tid >> 4), part = tid & 15;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) top = max(top, max(qx[q][j] & 0x7FFFu, (qx[q][j] >> 16) & 0x7FFFu));
#pragma unroll
      for (int k = 1; k < 16; k *= 2) top = max(top, __shfl_xor_sync(~0u, top, k));
      // 2^(14 - e), e the exponent of the largest element (kept where both powers are normal numbers)
      const int e = min(max((int)(top >> 7) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      uint32_t* dst = reinterpret_cast<uint32_t*>(ka_smem + S::kOffQ + row * S::kQPitch);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) dst[16 * j + part] = pack_half2(bf16lo(qx[q][j]) * up, bf16hi(qx[q][j]) * up);
      if (part == 0) s_qscale[row] = p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    }
    __syncthreads();
    // the operands of k-steps s and s + 1 of a 64-wide chunk c (or the 32-wide one): elements 4 s .. 4 s + 7 of row g
    const uint8_t* qrow = ka_smem + S::kOffQ + g * S::kQPitch;
    auto load_q = [&](int chunk, int s, int nt, uint32_t (&x)[2], uint32_t (&y)[2]) {
      const int at_byte = chunk < S::kK16 ? chunk * 128 + 32 * t + 8 * s : S::kK16 * 128 + 16 * t + 8 * s;
      const uint4 v = *reinterpret_cast<const uint4*>(qrow + nt * 8 * S::kQPitch + at_byte);
      x[0] = v.x, x[1] = v.y, y[0] = v.z, y[1] = v.w;
    };
    uint32_t qb[S::kQRegs ? D / 16 : 2][NT][2];
    if constexpr (S::kQRegs) {
#pragma unroll
      for (int c = 0; c < S::kK16 + S::kK8; ++c)
#pragma unroll
        for (int s = 0; s < (c < S::kK16 ? 4 : 2); s += 2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) load_q(c, s, nt, qb[4 * c + s][nt], qb[4 * c + s + 1][nt]);
    }
    float qs[NT][2];
    int see[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + 2 * t + e;
        qs[nt][e] = s_qscale[row];
        see[nt][e] = row < tile_rows ? sees(row) : 0x7FFFFFFF;
      }

    // ---------------------------------------------------------- the steps
    float o[D / 16][NT][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
    float b[NT][2], l[NT][2];  // base, denominator
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) b[nt][e] = kKaLowest, l[nt][e] = 0.0f;

    for (int i = 0; i < it.my_steps; i += U) {
      KaPlace scale[U];
#pragma unroll
      for (int x = 0; x < U; ++x) scale[x] = place[x];
      ahead(i + kKaAhead * U);
      if (i + U < it.my_steps) {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          place[x] = places[(i + U + x) & 63];  // (behind the last step: a block that is not there)
          off[x] = offset(place[x].unit);
        }
      }
      float c[U][NT][4];
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) c[x][nt][0] = c[x][nt][1] = c[x][nt][2] = c[x][nt][3] = 0.0f;
      // two k-steps: a word each of the keys of tokens g and g + 8
      auto keys = [&](float (&acc)[NT][4], int chunk, int s, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        if constexpr (!S::kQRegs) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) load_q(chunk, s, nt, qb[0][nt], qb[1][nt]);
        }
        const int at_q = S::kQRegs ? 4 * chunk + s : 0;
        const uint32_t x = w0 ^ 0x80808080u, y = w1 ^ 0x80808080u, z = w2 ^ 0x80808080u, w = w3 ^ 0x80808080u;
        const uint32_t x0 = codes_lo(x), x1 = codes_hi(x), y0 = codes_lo(y), y1 = codes_hi(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], x0, y0, x1, y1, qb[at_q][nt]);
        const uint32_t z0 = codes_lo(z), z1 = codes_hi(z), w0h = codes_lo(w), w1h = codes_hi(w);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], z0, w0h, z1, w1h, qb[at_q + 1][nt]);
      };
#pragma unroll
      for (int ch = 0; ch < S::kK16; ++ch) {
#pragma unroll
        for (int x = 0; x < U; ++x)
          keys(c[x], ch, 0, k16[x][ch][0].x, k16[x][ch][1].x, k16[x][ch][0].y, k16[x][ch][1].y);
#pragma unroll
        for (int x = 0; x < U; ++x)
          keys(c[x], ch, 2, k16[x][ch][0].z, k16[x][ch][1].z, k16[x][ch][0].w, k16[x][ch][1].w);
      }
      if constexpr (S::kK8 != 0) {
#pragma unroll
        for (int x = 0; x < U; ++x) keys(c[x], S::kK16, 0, k8[x][0].x, k8[x][1].x, k8[x][0].y, k8[x][1].y);
      }
      if (i + U < it.my_steps) load_keys();
      // scores in powers of two, the block's value scale among them: token g + 8 (j / 2), row 2 t + j % 2
      bool grows = false;
#pragma unroll
      for (int x = 0; x < U; ++x) {
        grows |= scale[x].vinv < 0.0f;
        const int token = (it.step0 + warp + kKaWarps * (i + x)) * kKaStep;
        const bool masked = i + x >= first_masked || scale[x].unit < 0;  // (there is no such block)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) c[x][nt][j] = fmaf(c[x][nt][j], qs[nt][j & 1] * scale[x].kscale, scale[x].vlog);
          if (masked) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (token + g + 8 * (j >> 1) >= see[nt][j & 1] || scale[x].unit < 0) c[x][nt][j] = -INFINITY;
          }
          grows |= fmaxf(c[x][nt][0], c[x][nt][2]) - b[nt][0] > kKaMost || fmaxf(c[x][nt][1], c[x][nt][3]) - b[nt][1] > kKaMost;
        }
      }
      if (__any_sync(~0u, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float a[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(c[0][nt][e], c[0][nt][2 + e]);
#pragma unroll
            for (int x = 1; x < U; ++x) top = fmaxf(top, fmaxf(c[x][nt][e], c[x][nt][2 + e]));
#pragma unroll
            for (int k = 4; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
            top = fmaxf(top - kKaLift, b[nt][e]);
            const float half = exp2_fast(0.5f * (b[nt][e] - top));  // (see kKaFar)
            a[e] = half * half;
            l[nt][e] = l[nt][e] * half * half;
            b[nt][e] = top;
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k) o[k][nt][0] *= a[0], o[k][nt][1] *= a[1], o[k][nt][2] *= a[0], o[k][nt][3] *= a[1];
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
          if (scale[x].vinv >= 0.0f) continue;
          scale[x].vinv = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float half = exp2_fast(0.5f * (c[x][nt][j] - b[nt][j & 1] - scale[x].vlog));
              l[nt][j & 1] = fmaf(half, half, l[nt][j & 1]);
            }
        }
      }
      uint32_t pb[U][NT][2];
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float(&w)[4] = c[x][nt];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = exp2_fast(w[j] - b[nt][j & 1]);
          l[nt][0] = fmaf(w[0] + w[2], scale[x].vinv, l[nt][0]);
          l[nt][1] = fmaf(w[1] + w[3], scale[x].vinv, l[nt][1]);
          pb[x][nt][0] = transpose8(pack_half2(w[0], w[1]));
          pb[x][nt][1] = transpose8(pack_half2(w[2], w[3]));
        }
      // the operands of two MMAs, four d, out of a word of each of four tokens
      auto values = [&](const uint32_t (&pw)[NT][2], int tile, uint32_t wa, uint32_t wb, uint32_t wc, uint32_t wd) {
        const uint32_t x = __byte_perm(wa, wb, 0x5140) ^ 0x80808080u, y = __byte_perm(wc, wd, 0x5140) ^ 0x80808080u;
        const uint32_t x0 = codes_lo(x), x1 = codes_hi(x), y0 = codes_lo(y), y1 = codes_hi(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[tile][nt], x0, x1, y0, y1, pw[nt]);
        const uint32_t z = __byte_perm(wa, wb, 0x7362) ^ 0x80808080u, w = __byte_perm(wc, wd, 0x7362) ^ 0x80808080u;
        const uint32_t z0 = codes_lo(z), z1 = codes_hi(z), w0 = codes_lo(w), w1 = codes_hi(w);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(o[tile + 1][nt], z0, z1, w0, w1, pw[nt]);
      };
#pragma unroll
      for (int x = 0; x < U; ++x) {
#pragma unroll
        for (int ch = 0; ch < S::kV16; ++ch) {
          const uint4(&w)[4] = v16[x][ch];
          values(pb[x], 8 * ch, w[0].x, w[1].x, w[2].x, w[3].x);
          values(pb[x], 8 * ch + 2, w[0].y, w[1].y, w[2].y, w[3].y);
          values(pb[x], 8 * ch + 4, w[0].z, w[1].z, w[2].z, w[3].z);
          values(pb[x], 8 * ch + 6, w[0].w, w[1].w, w[2].w, w[3].w);
        }
        if constexpr (S::kV8 != 0) {
          const uint2(&w)[4] = v8[x];
          values(pb[x], 8 * S::kV16, w[0].x, w[1].x, w[2].x, w[3].x);
          values(pb[x], 8 * S::kV16 + 2, w[0].y, w[1].y, w[2].y, w[3].y);
        }
        if constexpr (S::kV4 != 0) values(pb[x], 8 * S::kV16 + 4 * S::kV8, v4[x][0], v4[x][1], v4[x][2], v4[x][3]);
      }
      if (i + U < it.my_steps) load_values();
    }

    // ---------------------------------------------------------- the next tile's first reads go ahead of this one's end
    const KaItem done = it;
    at = min(it.end, end);
    const bool more = at < end;
    if (more) begin_item();

    // ---------------------------------------------------------- the four warps' sums
    // lane (g, t) holds `width` successive d of rows 2 t and 2 t + 1, two of each tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 4; k < 32; k *= 2) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], k);
        if (g == 0) {
          s_max[warp * ROWS + 8 * nt + 2 * t + e] = b[nt][e];
          s_den[warp * ROWS + 8 * nt + 2 * t + e] = l[nt][e];
        }
      }
    auto put = [&](int first_tile, int width, int d0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < width; i += 4) {
            const float(&x)[4] = o[first_tile + i / 2][nt];
            const float(&y)[4] = o[first_tile + i / 2 + 1][nt];
            *reinterpret_cast<float4*>(s_o + (warp * ROWS + 8 * nt + 2 * t + e) * S::kOPitch + d0 + width * g + i) =
                make_float4(x[e], x[2 + e], y[e], y[2 + e]);
          }
    };
#pragma unroll
    for (int ch = 0; ch < S::kV16; ++ch) put(8 * ch, 16, 128 * ch);
    if constexpr (S::kV8 != 0) put(8 * S::kV16, 8, 128 * S::kV16);
    if constexpr (S::kV4 != 0) put(8 * S::kV16 + 4 * S::kV8, 4, 128 * S::kV16 + 64 * S::kV8);
    __syncthreads();
    const bool whole = done.step0 == 0 && done.step1 == done.rq.steps;
    const int which = done.step0 == 0 ? 1 : 0;
    float* part_at = parts + (2 * (int64_t)blockIdx.x + which) * ka_part_floats(ROWS, D);
    if (!whole && tid == 0) {
      // The first CTA is the last one whose cut is not behind the tile's beginning, the last one is the last whose
      // cut is before its end: see where cuts near a tile's ends go.
      const int64_t start = done.end - done.rq.steps - kKaTileCost;
      const int c0 = which ? (int)blockIdx.x : (int)ka_div(start + kKaTileCost + kKaMinPart - 1, share);
      joins[which] = KaJoin{c0, (int)ka_div(done.end - kKaMinPart, share) - c0 + 1, done.rq.row0, done.h, done.tile, tile_rows, {0, 0}};
    }
    // 16 lanes to a row
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int row = 8 * q + (tid >> 4), part = tid & 15;
      float top = kKaLowest, den = 0.0f, a[kKaWarps];
#pragma unroll
      for (int w = 0; w < kKaWarps; ++w) top = fmaxf(top, s_max[w * ROWS + row]);
#pragma unroll
      for (int w = 0; w < kKaWarps; ++w) {
        const float x = s_max[w * ROWS + row];
        const float half = exp2_fast(0.5f * (x - top));
        a[w] = half * half;
        den = fmaf(s_den[w * ROWS + row] * half, half, den);
      }
      const float inv = den == 0.0f ? 0.0f : 1.0f / den;  // a row that sees nothing is 0
      if (!whole && part == 0) part_at[row] = top, part_at[ROWS + row] = den;
      const int idx = done.tile * ROWS + row, i = idx / p.group;
      uint16_t* out = p.o + (done.rq.row0 + i) * p.ldo + ((int64_t)done.h * p.group + (idx - i * p.group)) * D;
#pragma unroll
      for (int col = 4 * part; col < D; col += 64) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kKaWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(s_o + (w * ROWS + row) * S::kOPitch + col);
          v.x = fmaf(x.x, a[w], v.x), v.y = fmaf(x.y, a[w], v.y), v.z = fmaf(x.z, a[w], v.z), v.w = fmaf(x.w, a[w], v.w);
        }
        if (!whole) {
          *reinterpret_cast<float4*>(part_at + 2 * ROWS + row * D + col) = v;
        } else if (row < tile_rows) {
          *reinterpret_cast<uint2*>(out + col) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        }
      }
    }
    if (!more) break;
    __syncthreads();  // the rows' sums and scales have been read
  }
}

// The parts of the tiles that several CTAs worked on.  CTA c of the launch before has one of each of its two; the rows
// of a tile go round the CTAs that worked on it.  A row's parts are shared out over 1 to 16 warps, each
// adds up its own in order, then the first one the others' sums.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kKaJoinWarps) k_kv_attn_join(KvAttnParams p) {
  constexpr int ROWS = 8 * NT;
  __shared__ float s_sum[kKaJoinWarps][D];
  __shared__ float s_top[kKaJoinWarps], s_den[kKaJoinWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const KaJoin* joins = reinterpret_cast<const KaJoin*>(p.ws) + 2 * blockIdx.x;
  const KaJoin both[2] = {joins[0], joins[1]};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* parts = p.ws + 2 * (int64_t)gridDim.x * (sizeof(KaJoin) / 4);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const KaJoin join = both[which];
    if (join.parts == 0) continue;
    auto at = [&](int k) { return parts + (2 * (int64_t)(join.first + k) + (k == 0 ? 1 : 0)) * ka_part_floats(ROWS, D); };
    const int split = join.parts > 8 ? 16 : join.parts > 4 ? 8 : join.parts > 2 ? 4 : 2;  // warps to a row
    const int at_once = kKaJoinWarps / split, mine = warp % split;
    for (int row0 = (int)blockIdx.x - join.first; row0 < join.rows; row0 += at_once * join.parts) {
      const int row = row0 + warp / split * join.parts;
      float v[D / 32], den = 0.0f, top = kKaLowest;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) v[j] = 0.0f;
      if (row < join.rows) {
#pragma unroll 4
        for (int k = mine; k < join.parts; k += split) {
          const float* part = at(k);
          const float x = part[row], y = part[ROWS + row];
          float z[D / 32];
#pragma unroll
          for (int j = 0; j < D / 32; ++j) z[j] = part[2 * ROWS + row * D + 32 * j + lane];
          const float now = fmaxf(top, x), ah = exp2_fast(0.5f * (top - now)), bh = exp2_fast(0.5f * (x - now));
          const float a = ah * ah, b = bh * bh;
          den = fmaf(y * bh, bh, den * ah * ah);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) v[j] = fmaf(z[j], b, v[j] * a);
          top = now;
        }
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) s_sum[warp][32 * j + lane] = v[j];
      if (lane == 0) s_top[warp] = top, s_den[warp] = den;
      __syncthreads();
      if (mine == 0 && row < join.rows) {
        float all = top;
        for (int w = 1; w < split; ++w) all = fmaxf(all, s_top[warp + w]);
        den = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) v[j] = 0.0f;
        for (int w = 0; w < split; ++w) {
          const float half = exp2_fast(0.5f * (s_top[warp + w] - all)), a = half * half;
          den = fmaf(s_den[warp + w] * half, half, den);
#pragma unroll
          for (int j = 0; j < D / 32; ++j) v[j] = fmaf(s_sum[warp + w][32 * j + lane], a, v[j]);
        }
        const float inv = den == 0.0f ? 0.0f : 1.0f / den;
        const int idx = join.tile * ROWS + row, i = idx / p.group;
        uint16_t* out = p.o + (join.row0 + i) * p.ldo + ((int64_t)join.head * p.group + (idx - i * p.group)) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) out[32 * j + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(v[j] * inv));
      }
      __syncthreads();
    }
  }
}

}  // namespace gbmlp
