// The key/value cache in 8 bits: which blocks a step's tokens go to, and the write.
//
// Blocks of bs = 16, 32 or 64 tokens, a maximum for each block and head:
//   Kc, Vc [blocks, nk, bs, d] int8, Kmax, Vmax [blocks, nk] fp32;  a code c stands for c * max / 127
//
// The maximum is kept, not max / 127: keys and values are bf16, so that products of a code with a maximum are exact in
// fp32 and a division rounded once decides every rounding to a code as exact arithmetic would.  New values are
// multiplied by 127 / max rounded up instead.  With significands a of x and b of max, 8 bits each, and x's exponent t below max's,
// x * 127 / max = 127 a / (b 2^t): a tie where 127 divides b (b = 254; 127 / max is then a power of two and the product
// exact) or where |x| = max / 2 (+-63.5, which goes to the even 64 as it does from a little above).  Everything else is at least
// 1 / (2 b 2^t) > 2^-(9 + t) from a tie, and the rounded factor moves the quotient, which is below 2^(8 - t), by less
// than 2^-(15 + t).  The same holds for a moved code c old / new = c a / (b 2^t), whose one rounding moves it by half of that.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace gbmlp {

constexpr int kKvMaxHead = 256;
constexpr int kKvMaxRequests = 4096;

// ---------------------------------------------------------------- block tables and slots
constexpr int kKvPlanThreads = 512;
constexpr int kKvPlanRows = 1024;  // rows of a CTA

enum KvPlanStatus : int { kKvNoBlocks = 1, kKvTableFull = 2, kKvNoRows = 4, kKvNegative = 8 };

struct KvPlanParams {
  int n, log_bs, width, n_free, rows;
  const int* add;
  const int* lens;
  int* table;  // [n, width]
  const int* free;
  const int* taken;
  int* lens_out;
  int* taken_out;
  int* cu;  // [n + 1]
  int* pos;
  int* slots;
  int* status;
};

// Inclusive sum over the CTA of a pair; `part` holds a pair for each warp.
__device__ __forceinline__ void kv_scan2(int64_t& a, int64_t& b, int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const int64_t x = __shfl_up_sync(~0u, a, k), y = __shfl_up_sync(~0u, b, k);
    if (lane >= k) a += x, b += y;
  }
  if (lane == 31) part[warp][0] = a, part[warp][1] = b;
  __syncthreads();
  for (int w = 0; w < warp; ++w) a += part[w][0], b += part[w][1];
}

// Every CTA adds up all n requests (a few thousand at most, in L2) and fills in 1024 rows:
// one launch, nothing handed from CTA to CTA, so what bounds it is that launch and a chain
// of four loads: 2.8 us for a step of 64 requests, 3.9 us for 500 prompts of 65,000 rows (5.5 us with 256 threads,
// which go over the requests twice).
__global__ void __launch_bounds__(kKvPlanThreads) k_kv_plan(KvPlanParams p) {
  extern __shared__ int kv_plan_smem[];
  int* s_cu = kv_plan_smem;           // [n + 1]
  int* s_first = kv_plan_smem + p.n + 1;  // [n]: new blocks of the requests before
  __shared__ int64_t part[kKvPlanThreads / 32][2];
  __shared__ int s_bad;
  grid_dependency_wait();
  grid_launch_dependents();
  if (threadIdx.x == 0) s_bad = 0;
  const int bs = 1 << p.log_bs;
  const int64_t taken = *p.taken;
  int64_t rows = 0, blocks = 0;
  int bad = taken < 0 ? kKvNoBlocks : 0;
  for (int r0 = 0; r0 < p.n; r0 += kKvPlanThreads) {
    const int r = r0 + (int)threadIdx.x;
    int64_t add = 0, more = 0;
    if (r < p.n) {
      add = p.add[r];
      int64_t old = p.lens[r];
      if (add < 0 || old < 0) bad |= kKvNegative, add = add < 0 ? 0 : add, old = old < 0 ? 0 : old;
      const int64_t need = (old + add + bs - 1) >> p.log_bs;
      if (need > p.width) bad |= kKvTableFull;
      more = need - ((old + bs - 1) >> p.log_bs);
    }
    int64_t a = add, b = more;
    __syncthreads();  // `part` and s_bad
    kv_scan2(a, b, part);
    if (r < p.n) {
      s_cu[r] = (int)(rows + a - add);
      s_first[r] = (int)(blocks + b - more);
    }
    for (int w = 0; w < kKvPlanThreads / 32; ++w) rows += part[w][0], blocks += part[w][1];
  }
  if (taken + blocks > p.n_free) bad |= kKvNoBlocks;
  if (rows > p.rows) bad |= kKvNoRows;
  if (threadIdx.x == 0) s_cu[p.n] = (int)rows;
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  if (blockIdx.x == 0) {
    for (int r = threadIdx.x; r <= p.n; r += kKvPlanThreads) {
      p.cu[r] = bad ? 0 : s_cu[r];
      if (r < p.n) p.lens_out[r] = p.lens[r] + (bad ? 0 : p.add[r]);
    }
    if (threadIdx.x == 0) {
      *p.taken_out = (int)(taken + (bad ? 0 : blocks));
      *p.status = bad;
    }
  }
  const int64_t t_end = min((int64_t)p.rows, ((int64_t)blockIdx.x + 1) * kKvPlanRows);
  for (int64_t t = (int64_t)blockIdx.x * kKvPlanRows + threadIdx.x; t < t_end; t += kKvPlanThreads) {
    int pos = 0, slot = -1;
    if (!bad && t < rows) {
      int lo = 0, hi = p.n - 1;  // the last request whose rows begin at t or before (the empty ones' end there too)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int old = p.lens[lo];
      pos = old + (int)(t - s_cu[lo]);
      const int b = pos >> p.log_bs, have = (int)(((int64_t)old + bs - 1) >> p.log_bs);
      int* cell = p.table + (int64_t)lo * p.width + b;
      const int block = b < have ? *cell : p.free[taken + s_first[lo] + b - have];
      if ((pos & (bs - 1)) == 0) *cell = block;  // a block that begins here is a new one
      const int64_t wide = (int64_t)block * bs + (pos & (bs - 1));  // (what the table says need not be a block)
      slot = wide == (int)wide ? (int)wide : -1;
    }
    p.pos[t] = pos;
    p.slots[t] = slot;
  }
}

// ---------------------------------------------------------------- the write
struct KvWriteParams {
  int64_t tokens, ld[2];  // rows' strides of K, V
  int nk, blocks, log_bs;
  int chunk;              // tokens among which a CTA looks for runs' beginnings: at most 64
  int span;               // of the 2 nk heads of keys and values, those that a CTA takes
  const int* slots;
  const uint16_t* x[2];
  int8_t* codes[2];
  float* most[2];
};

constexpr float kKvTiny = 8.271806125530277e-25f;  // 2^-80: blocks of smaller magnitudes hold zeros
constexpr float kKvRound = 12582912.0f;            // 1.5 * 2^23: added, the sum's low byte is the rounded code

// The four codes of fp32 products already rounded into kKvRound's last places.
__device__ __forceinline__ uint32_t kv_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

__device__ __forceinline__ uint32_t kv_codes4(uint32_t x01, uint32_t x23, float inv) {
  return kv_pack4(fmaf(bf16lo(x01), inv, kKvRound), fmaf(bf16hi(x01), inv, kKvRound), fmaf(bf16lo(x23), inv, kKvRound),
                  fmaf(bf16hi(x23), inv, kKvRound));
}

// round(code * from / to), from <= to.  `from` is taken 2^-8 times, so that no product leaves fp32 (127 times the largest bf16
// would): exact, as it is 2^-80 at least where there are codes but 0, and the quotient's 2^8 come back with the rounding's sum.
__device__ __forceinline__ uint32_t kv_move4(uint32_t codes, float from, float to) {
  from *= 0.00390625f;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fmaf(__fdiv_rn((float)(int8_t)(codes >> (8 * i)) * from, to), 256.0f, kKvRound);
  return kv_pack4(v[0], v[1], v[2], v[3]);
}

// The largest magnitude of N pieces, as an fp32's bits: magnitudes are in the order of their bits, a NaN above all.
template <int N>
__device__ __forceinline__ uint32_t kv_top(const uint4 (&v)[N]) {
  uint32_t top = 0;  // of the low and of the high elements
#pragma unroll
  for (int j = 0; j < N; ++j)
    for (const uint32_t w : {v[j].x, v[j].y, v[j].z, v[j].w}) top = __vmaxu2(top, w & 0x7FFF7FFFu);
  return max(top << 16, top & 0xFFFF0000u);
}

// A block's maximum with the new tokens' largest magnitude, and 127 / it.
struct KvScale {
  float now, inv;
  bool finite;
};
__device__ __forceinline__ KvScale kv_scale(uint32_t bits, float old) {
  KvScale s;
  bits = max(bits, __float_as_uint(old) & 0x7FFFFFFFu);
  s.finite = bits < 0x7F800000u;
  s.now = __uint_as_float(s.finite ? bits : 0x7FC00000u);  // a block with an infinity or a NaN reads as NaN
  s.inv = s.finite && s.now >= kKvTiny ? __fdiv_ru(127.0f, s.now) : 0.0f;
  return s;
}

__device__ __forceinline__ uint2 kv_codes8(uint4 x, const KvScale& s) {
  return s.finite ? make_uint2(kv_codes4(x.x, x.y, s.inv), kv_codes4(x.z, x.w, s.inv)) : make_uint2(0, 0);
}

// One CTA of bs / 8 warps for each `chunk` tokens and `span` heads of keys or values.  Tokens in slots next
// to each other in one block go together (a run, which begins where the token before is not in the slot
// before): their rows are read once, into registers (16 bytes a
// lane, always the same 8 elements of a head), their largest magnitude found, their codes written; the codes before them move
// only where the maximum grows.  Runs of a few tokens (64 pieces of 16 bytes at most: one to 16 tokens) a warp takes alone, the
// next one the next warp.  Every access is 16 or 8 bytes a lane and side by side.  Over few tokens a launch with
// a chain of two or three reads bounds it, over many HBM latency and the instructions of the codes alike: 7021 tokens of 8
// heads of 128 10.8 us (6.4 of bytes), 753 tokens of 128 heads of 160 20.1 us (13.6), a token 2.0 us, one for each of 130
// requests 4.5 us, one for each of 4000 49 us (254 MB of codes move there; 73 us with a CTA to each).  A kernel for each
// block size (rows and distances known) took 12.1 to 10.1 and 20.9 to 19.9 us.
// Of blocks of 64 tokens 5 CTAs of 8 warps are to fit, with 48 registers, for heads up to 128: 20,500 tokens of 1024 elements take
// 38 us for 43 without that bound with heads of 64 (which then spill 28 bytes), 31 for 34 with 96, 28 for 30 with 128, 46 either
// way with 32 (which spill too).  Other kernels are left the registers that they take, and spill up to 44 bytes: bound to 1024 threads an
// SM, heads of 224 in blocks of 16 and 32 took 21 us for 22 and 23, smaller heads up to 1 us more, the rest 1 us less or the same.
template <int D, int BS>
__global__ void __launch_bounds__(4 * BS, BS == 64 && D <= 128 ? 5 : 0) k_kv_write(KvWriteParams p) {
  constexpr int kRowPieces = D / 8;                      // 16-byte pieces of a row
  constexpr int kRows = 4 * BS / kRowPieces;             // rows at once
  constexpr int kPieces = (BS + kRows - 1) / kRows;      // of a lane
  __shared__ uint32_t s_most[2][BS / 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned spans = (2u * p.nk + p.span - 1) / p.span, rest = blockIdx.x / spans;
  const int head0 = (int)(blockIdx.x - rest * spans) * p.span, head1 = min(head0 + p.span, 2 * p.nk);
  const int64_t t0 = (int64_t)rest * p.chunk;
  const int cap = p.blocks * BS;
  const int row = (int)threadIdx.x / kRowPieces;
  const int column = ((int)threadIdx.x - row * kRowPieces) * 8;
  // of the chunk's tokens and a block's more: those that go on with a run, and of the chunk's: those that begin one
  uint32_t goes_on[4] = {0, 0, 0, 0}, begins[2] = {0, 0};
  int slots[2] = {-1, -1};
#pragma unroll
  for (int j = 0; j < BS / 16; ++j) {
    const int64_t t = t0 + 32 * j + lane;
    int s = -1, before = -2;
    if (32 * j >= p.chunk + BS) break;
    if (t < p.tokens) {
      s = p.slots[t];
      before = t > 0 ? p.slots[t - 1] : -2;
    }
    const bool there = s >= 0 && s < cap, on = there && (s & (BS - 1)) != 0 && before == s - 1;
    goes_on[j] = __ballot_sync(~0u, on);
    if (j < 2) {
      begins[j] = __ballot_sync(~0u, there && !on && 32 * j + lane < p.chunk);
      slots[j] = s;
    }
  }
  const uint64_t on_lo = goes_on[0] | (uint64_t)goes_on[1] << 32, on_hi = goes_on[2] | (uint64_t)goes_on[3] << 32;
  uint64_t leads = begins[0] | (uint64_t)begins[1] << 32, few = 0;
  auto length = [&](int at_chunk) {  // tokens of the run that begins there
    const uint64_t after = at_chunk == 63 ? on_hi : on_lo >> (at_chunk + 1) | on_hi << (63 - at_chunk);
    return ~after == 0 ? 65 : __ffsll((long long)~after);
  };
  auto slot_of = [&](int at_chunk) { return __shfl_sync(~0u, at_chunk < 32 ? slots[0] : slots[1], at_chunk & 31); };
  int turn = 0;
  while (leads != 0) {
    const int at_chunk = __ffsll((long long)leads) - 1, count = length(at_chunk);
    leads &= leads - 1;
    if (count * kRowPieces <= 64) {
      few |= 1ull << at_chunk;
      continue;
    }
    const int64_t t = t0 + at_chunk;
    const int slot = slot_of(at_chunk), off = slot & (BS - 1);
    const int last = row < kRows ? off + count : 0;  // (lanes that are left over have no rows)
    for (int head = head0; head < head1; ++head) {
      const int kv = head >= p.nk ? 1 : 0, h = kv ? head - p.nk : head;
      const int64_t ld = kv ? p.ld[1] : p.ld[0];
      const uint16_t* x = (kv ? p.x[1] : p.x[0]) + (int64_t)h * D + column;
      const int64_t bh = (int64_t)(slot / BS) * p.nk + h;
      float* most = (kv ? p.most[1] : p.most[0]) + bh;
      int8_t* codes = (kv ? p.codes[1] : p.codes[0]) + (bh * BS + row) * D + column;
      const float old = off > 0 ? *most : 0.0f;
      uint4 v[kPieces];
      const uint16_t* from = x + (t - off + row) * ld;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int at = row + j * kRows;
        v[j] = make_uint4(0, 0, 0, 0);
        if (at >= off && at < last) v[j] = *reinterpret_cast<const uint4*>(from);
        from += kRows * ld;
      }
      uint32_t bits = __reduce_max_sync(~0u, kv_top(v));
      if (lane == 0) s_most[turn][warp] = bits;
      __syncthreads();
      bits = __reduce_max_sync(~0u, s_most[turn][lane & (BS / 8 - 1)]);
      turn ^= 1;
      const KvScale sc = kv_scale(bits, old);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int at = row + j * kRows;
        if (at >= off && at < last)
          *reinterpret_cast<uint2*>(codes + j * kRows * D) = kv_codes8(v[j], sc);
      }
      if (off > 0 && sc.finite && sc.now != old && row < kRows) {
        for (int at = row; at < off; at += kRows) {
          uint2* to = reinterpret_cast<uint2*>(codes + (at - row) * D);
          const uint2 c = *to;
          *to = make_uint2(kv_move4(c.x, old, sc.now), kv_move4(c.y, old, sc.now));
        }
      }
      if (threadIdx.x == 0) *most = sc.now;
    }
  }
  for (int turn_of = warp; few != 0; few &= few - 1, ++turn_of) {
    const int at_chunk = __ffsll((long long)few) - 1, pieces = length(at_chunk) * kRowPieces;
    const int slot = slot_of(at_chunk), off = slot & (BS - 1);
    for (int head = head0 + turn_of % (BS / 8); head < head1; head += BS / 8) {
      const int kv = head >= p.nk ? 1 : 0, h = kv ? head - p.nk : head;
      const int64_t ld = kv ? p.ld[1] : p.ld[0];
      const uint16_t* x = (kv ? p.x[1] : p.x[0]) + (t0 + at_chunk) * ld + (int64_t)h * D;
      const int64_t bh = (int64_t)(slot / BS) * p.nk + h;
      float* most = (kv ? p.most[1] : p.most[0]) + bh;
      int8_t* codes = (kv ? p.codes[1] : p.codes[0]) + bh * BS * D;
      const float old = off > 0 ? *most : 0.0f;
      uint4 v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = lane + 32 * j, at = i / kRowPieces;
        v[j] = make_uint4(0, 0, 0, 0);
        if (i < pieces) v[j] = *reinterpret_cast<const uint4*>(x + at * ld + (i - at * kRowPieces) * 8);
      }
      const KvScale sc = kv_scale(__reduce_max_sync(~0u, kv_top(v)), old);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = lane + 32 * j;  // (a run's codes lie side by side)
        if (i < pieces) *reinterpret_cast<uint2*>(codes + off * D + i * 8) = kv_codes8(v[j], sc);
      }
      if (off > 0 && sc.finite && sc.now != old) {
        for (int i = lane; i < off * kRowPieces; i += 32) {
          uint2* to = reinterpret_cast<uint2*>(codes + i * 8);
          const uint2 c = *to;
          *to = make_uint2(kv_move4(c.x, old, sc.now), kv_move4(c.y, old, sc.now));
        }
      }
      __syncwarp();  // the maximum has been read by all
      if (lane == 0) *most = sc.now;
    }
  }
}

}  // namespace gbmlp
