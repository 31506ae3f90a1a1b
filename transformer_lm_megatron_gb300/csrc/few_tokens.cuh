// The gated block's products over its weights for few tokens (a batch of sequences, one
// token each, or a short one): every weight is read for a handful of rows, so HBM bounds
// them and what counts is that every SM streams weights all the time.
//
//   D^T[N, T] = W^T[N, K] X^T[K, T]     (bf16 operands, fp32 accumulator in TMEM)
//
// The weights are the MMA's M operand (128 weight columns, MN-major as stored, or in the
// backward 128 weight rows, K-major as stored: W^T below) and the
// tokens its N (16 to 64), so a tile holds no idle rows of 128 tokens: a k-block brings
// 16 KB of weights and 2 KB of activations at 16 tokens.  A cluster of 1 to 8 CTAs shares
// one tile's reduction: each takes a range of k-blocks and writes its fp32 partial, token
// by token, straight from TMEM into the shared memory of the CTA that finishes that token
// (distributed shared memory); after one cluster barrier every CTA adds what it was sent,
// in rank order, and writes its tokens' outputs (deterministic, no workspace).  Sent, the
// partials take one barrier and no remote reads: 2 us of a launch less than fetched.
//   kFtGates   W = [Ag | Au]: 64 columns of each half in a tile; Y = act(G) U (and G, U)
//   kFtOut     W = B: O = R + dropout(Z + b)
//   kFtDGates  W = B^T: dY, and dG = dY U act'(G), dU = dY act(G)
//   kFtDX      W = [Ag | Au]^T: dX = [dO +] dGU W
// The second launch of a pass fetches its first weights before it waits for the first one.
// One token at h 4096, ffn 16384: 64 us a pass, 93 % of the copy rate (59 us for the
// weights); 99 us with the GEMMs of 256 x 256 tiles, whose second product has few of them.
// 27 tokens at h 2048, ffn 5464: 19 us and 35 us (10 us for the weights; a launch takes
// 2.5 us to its first bytes and 2 us to join and write).
//
// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, 2..5 TMEM to shared memory; all six
// add and write the outputs.  Every wait is bounded (see gemm_tc.cuh).
#pragma once
#include <cstdint>
#include <cuda.h>

#include "block_math.cuh"
#include "gemm_tc.cuh"
#include "ptx.cuh"

namespace gbmlp {

constexpr int kFtThreads = 192;
constexpr int kFtTileW = 128;                       // weight columns of a tile (GATED: 64 of each half)
constexpr uint32_t kFtWBytes = kFtTileW * kBK * 2;  // 16 KB
constexpr int kFtMaxTokens = 64;                    // tokens of a CTA
constexpr int kFtMaxStages = 8;
constexpr int kFtMaxSplit = 8;

enum FewTokensKind : int { kFtGates = 0, kFtOut = 1, kFtDGates = 2, kFtDX = 3 };

struct FewTokensParams {
  int T, N, K;             // tokens; columns of the output (kFtGates, kFtDGates: of each half); reduction
  int split;               // CTAs of a cluster, each a share of the k-blocks
  int tpad;                // tokens of a tile, rounded up: 16, 32 or 64
  int stages;
  int per_log2;            // log2 of the tokens that one CTA of the cluster finishes
  int act;
  const uint16_t* bias;    // [N], kFtGates [2 N]; may be null
  const uint16_t* in;      // kFtOut, kFtDX: residual [T, N] (kFtDX: may be null); kFtDGates: [G | U] [T, 2 N]
  uint16_t* out;           // Y, O or dX [T, N]; kFtDGates: [dG | dU] [T, 2 N]
  uint16_t* GU;            // kFtGates: [T, 2 N] or null
  DropoutParams drop;
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// 8 consecutive values at `at`, summed over the `split` partials, `pitch` floats apart.
__device__ __forceinline__ void ft_sum8(const float* at, int split, int pitch, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int r = 0; r < split; ++r) {
    const float4 x = reinterpret_cast<const float4*>(at + r * pitch)[0], y = reinterpret_cast<const float4*>(at + r * pitch)[1];
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
}

__device__ __forceinline__ void st_bf16x8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// Grid tiles * token tiles * split, clusters of `split` CTAs.
template <int KIND>
__global__ void __launch_bounds__(kFtThreads, 2)
    k_few_tokens(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FewTokensParams p,
                 int* status) {
  constexpr bool GATED = KIND == kFtGates, W_MN = KIND == kFtGates || KIND == kFtOut;
  // The first launch of a pass waits before it touches its weights, which the launch before
  // it may have written.
  constexpr bool FIRST = KIND == kFtGates || KIND == kFtDGates;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t x_bytes = (uint32_t)p.tpad * kBK * 2;
  uint8_t* sW = smem;
  uint8_t* sX = smem + p.stages * kFtWBytes;
  __shared__ uint64_t full[kFtMaxStages], empty[kFtMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int token_tiles = (p.T + p.tpad - 1) / p.tpad;  // side by side, so that they share the weights' lines in L2
  const int rank = (int)(blockIdx.x % (unsigned)p.split), item = (int)(blockIdx.x / (unsigned)p.split);
  const int tile = item / token_tiles;
  const int n0 = tile * (GATED ? kFtTileW / 2 : kFtTileW);
  const int t0 = (item - tile * token_tiles) * p.tpad;
  const int num_kb = (p.K + kBK - 1) / kBK;
  const int kb0 = (int)((int64_t)num_kb * rank / p.split), kb1 = (int)((int64_t)num_kb * (rank + 1) / p.split);
  const uint32_t tmem_cols = p.tpad < 32 ? 32u : (uint32_t)p.tpad;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc<false>(&tmem_slot, tmem_cols);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_arrive_relaxed();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t issued[kFtMaxStages];
#pragma unroll
      for (int s = 0; s < kFtMaxStages; ++s) issued[s] = 0;
      auto weights = [&](int stage, int kb) {
        mbar_arrive_expect_tx(&full[stage], kFtWBytes + x_bytes);
        uint8_t* dst = sW + stage * kFtWBytes;
        if constexpr (!W_MN) {
          tma_load_2d(dst, &tmW, &full[stage], kb * kBK, n0, 0, false);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if constexpr (GATED)
              tma_load_3d(dst + j * kChunkBytes, &tmW, &full[stage], n0, j, kb * kBK);
            else
              tma_load_2d(dst + j * kChunkBytes, &tmW, &full[stage], n0 + 64 * j, kb * kBK, 0, false);
          }
        }
      };
      auto tokens = [&](int stage, int kb) {
        tma_load_2d(sX + stage * x_bytes, &tmX, &full[stage], kb * kBK, t0, 0, false);
      };
      // A pass's second weights are older than its first launch, which waited for all before
      // it: they may be fetched before this launch's wait.
      const int head = min(p.stages, kb1 - kb0);
      if constexpr (FIRST) grid_dependency_wait();
      for (int i = 0; i < head; ++i) weights(i, kb0 + i);
      if constexpr (!FIRST) grid_dependency_wait();
      for (int i = 0; i < head; ++i) tokens(i, kb0 + i);
      int stage = head == p.stages ? 0 : head;
      uint32_t phase = head == p.stages ? 1 : 0;
#pragma unroll
      for (int s = 0; s < kFtMaxStages; ++s) issued[s] = s < head ? 1 : 0;
      for (int kb = kb0 + head; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1)) {
          record_status(status, kStatusTimeout, 21);
          break;
        }
        weights(stage, kb);
        tokens(stage, kb);
#pragma unroll
        for (int s = 0; s < kFtMaxStages; ++s) issued[s] += s == stage ? 1 : 0;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // every copy has landed before the memory is used for anything else
#pragma unroll
      for (int s = 0; s < kFtMaxStages; ++s)
        if (issued[s] > 0 && !mbar_wait(&full[s], (issued[s] - 1) & 1)) record_status(status, kStatusTimeout, 22);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc = make_idesc_bf16(kFtTileW, p.tpad, W_MN, false);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase)) {
          record_status(status, kStatusTimeout, 23);
          break;
        }
        tc_fence_after();
        const uint32_t w = smem_u32(sW + stage * kFtWBytes), x = smem_u32(sX + stage * x_bytes);
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, W_MN ? make_sdesc_sw128(w + kk * 2048, kChunkBytes, 1024) : make_sdesc_sw128(w + kk * 32, 16, 1024),
                    make_sdesc_sw128(x + kk * 32, 16, 1024), idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      umma_commit(&acc_full);
    }
    __syncwarp();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  // This CTA's partial to the CTAs that finish its tokens: slot [rank][token of that CTA]
  // of their `sent` (beside the ring, which a slower CTA still uses).
  const int rows = min(p.tpad, p.T - t0), per = 1 << p.per_log2;
  float* sent = reinterpret_cast<float*>(smem + (p.split > 1 ? p.stages * (kFtWBytes + x_bytes) : 0));
  if (p.split > 1) cluster_wait();  // every CTA of the cluster has begun
  if (warp >= 2) {
    if (!mbar_wait(&acc_full, 0)) record_status(status, kStatusTimeout, 24);
    tc_fence_after();
    const int quarter = warp & 3;
    const uint32_t mine = smem_u32(sent) + (uint32_t)((rank << p.per_log2) * kFtTileW + quarter * 32 + lane) * 4;
    for (int c = 0; c < rows; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int t = c + j;
        if (t < rows)
          st_cluster_f32(mapa_shared(mine + (uint32_t)(t & (per - 1)) * (kFtTileW * 4), (uint32_t)(t >> p.per_log2)),
                         __uint_as_float(r[j]));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (p.split > 1) cluster_sync();
  // The outputs of this CTA's tokens, 8 columns an item.
  const int first = rank << p.per_log2, mine = min(per, rows - first);
  constexpr int kItems = (GATED ? kFtTileW / 2 : kFtTileW) / 8;  // of a token
  for (int i = threadIdx.x; i < mine * kItems; i += kFtThreads) {
    const int t = i / kItems, c = (i - t * kItems) * 8, col = n0 + c;
    if (col >= p.N) continue;
    const int64_t row = t0 + first + t;
    const float* at = sent + t * kFtTileW + c;
    const int pitch = per * kFtTileW;
    float v[8];
    ft_sum8(at, p.split, pitch, v);
    if constexpr (GATED) {
      float u[8];
      ft_sum8(at + kFtTileW / 2, p.split, pitch, u);
      if (p.bias != nullptr) {
        float bg[8], bu[8];
        ld_bf16x8(p.bias + col, bg);
        ld_bf16x8(p.bias + p.N + col, bu);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] += bg[j];
          u[j] += bu[j];
        }
      }
      if (p.GU != nullptr) {
        st_bf16x8(p.GU + row * 2 * p.N + col, v);
        st_bf16x8(p.GU + row * 2 * p.N + p.N + col, u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (p.act == kActSilu ? silu_f(v[j]) : gelu_gate_f(v[j])) * u[j];
    } else if constexpr (KIND == kFtDGates) {
      float g[8], u[8], du[8];
      const int64_t place = row * 2 * p.N + col;
      ld_bf16x8(p.in + place, g);
      ld_bf16x8(p.in + place + p.N, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float value, slope;
        if (p.act == kActSilu)
          silu_both_f(g[j], value, slope);
        else
          gelu_both_f(g[j], value, slope);
        du[j] = v[j] * value;
        v[j] = v[j] * u[j] * slope;
      }
      st_bf16x8(p.out + place, v);
      st_bf16x8(p.out + place + p.N, du);
      continue;
    } else if constexpr (KIND == kFtDX) {
      if (p.in != nullptr) {
        float res[8];
        ld_bf16x8(p.in + row * p.N + col, res);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += res[j];
      }
    } else {
      float bb[8] = {0, 0, 0, 0, 0, 0, 0, 0}, res[8];
      if (p.bias != nullptr) ld_bf16x8(p.bias + col, bb);
      ld_bf16x8(p.in + row * p.N + col, res);
      const uint32_t keep = p.drop.thr == 0 ? 0xffu : dropout_keep8(p.drop, row, col);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = res[j] + (((keep >> j) & 1u) ? (v[j] + bb[j]) * p.drop.scale : 0.0f);
    }
    st_bf16x8(p.out + row * p.N + col, v);
  }
  // (No CTA touches another's memory after the barrier.)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<false>(tmem, tmem_cols);
  }
}

}  // namespace gbmlp
