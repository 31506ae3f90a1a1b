// The gated block's forward for few tokens (a batch of sequences, one token each): both
// products read every weight once for a handful of rows, so HBM bounds them and what
// counts is that every SM streams weights all the time.
//
//   D^T[N, T] = W^T[N, K] X^T[K, T]     (bf16 operands, fp32 accumulator in TMEM)
//
// The weights are the MMA's M operand (128 weight columns, MN-major as stored) and the
// tokens its N (16 to 128), so a tile holds no idle rows of 128 tokens: a k-block brings
// 16 KB of weights and 2 KB of activations at 16 tokens.  A cluster of 1 to 8 CTAs shares
// one tile's reduction: each takes a range of k-blocks, leaves its fp32 partial
// [tokens, 128] in shared memory, and adds the partials of its share of the outputs from
// all CTAs through distributed shared memory, in rank order (deterministic, no
// workspace).  Two CTAs to an SM: one streams while the other starts or ends.
//   GATED  W = [Ag | Au]: 64 columns of each half in a tile; Y = act(G) U (and G, U)
//   else   W = B: 128 columns; O = R + dropout(Z + b)
// The second launch fetches its first weights before it waits for the first one's Y.
// The GEMM of gemm_tc.cuh took 162 us for one token at h 4096, ffn 16384 (its second
// product has 16 tiles, one to an SM, and 59 us is the weights' time at the copy rate).
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
constexpr int kFtMaxTokens = 128;                   // tokens of a CTA
constexpr int kFtMaxStages = 8;
constexpr int kFtMaxSplit = 8;

struct FewTokensParams {
  int T, N, K;             // tokens; columns of the output (GATED: of each half); reduction
  int split;               // CTAs of a cluster, each a share of the k-blocks
  int tpad;                // tokens of a tile, rounded up: 16, 32, 64 or 128
  int stages;
  int act;
  const uint16_t* bias;    // [N], GATED [2 N]; may be null
  const uint16_t* R;       // residual [T, N]
  uint16_t* out;           // Y or O [T, N]
  uint16_t* GU;            // GATED: [T, 2 N] or null
  DropoutParams drop;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// 8 consecutive values of the partial at `at` (a shared-memory address valid in every CTA
// of the cluster), summed over the CTAs in rank order.
__device__ __forceinline__ void ft_sum8(uint32_t at, int split, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int r = 0; r < split; ++r) {
    const uint32_t a = mapa_shared(at, r);
    const float4 x = ld_cluster_f4(a), y = ld_cluster_f4(a + 16);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
}

__device__ __forceinline__ void st_bf16x8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// Grid (tiles * split, token tiles), clusters of (split, 1, 1).
template <bool GATED>
__global__ void __launch_bounds__(kFtThreads, 2)
    k_few_tokens(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FewTokensParams p,
                 int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t x_bytes = (uint32_t)p.tpad * kBK * 2;
  uint8_t* sW = smem;
  uint8_t* sX = smem + p.stages * kFtWBytes;
  __shared__ uint64_t full[kFtMaxStages], empty[kFtMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (unsigned)p.split), tile = (int)(blockIdx.x / (unsigned)p.split);
  const int n0 = tile * (GATED ? kFtTileW / 2 : kFtTileW);
  const int t0 = (int)blockIdx.y * p.tpad;
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
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (GATED)
            tma_load_3d(dst + j * kChunkBytes, &tmW, &full[stage], n0, j, kb * kBK);
          else
            tma_load_2d(dst + j * kChunkBytes, &tmW, &full[stage], n0 + 64 * j, kb * kBK, 0, false);
        }
      };
      auto tokens = [&](int stage, int kb) {
        tma_load_2d(sX + stage * x_bytes, &tmX, &full[stage], kb * kBK, t0, 0, false);
      };
      // The second product's weights are older than the first launch, which waited for
      // all before it: they may be fetched before this launch's wait.  The first
      // product's may be what the launch before it wrote.
      const int head = min(p.stages, kb1 - kb0);
      if constexpr (GATED) grid_dependency_wait();
      for (int i = 0; i < head; ++i) weights(i, kb0 + i);
      if constexpr (!GATED) grid_dependency_wait();
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
      const uint32_t idesc = make_idesc_bf16(kFtTileW, p.tpad, true, false);
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
          umma_bf16(tmem, make_sdesc_sw128(w + kk * 2048, kChunkBytes, 1024), make_sdesc_sw128(x + kk * 32, 16, 1024), idesc,
                    (kb != kb0 || kk != 0) ? 1u : 0u);
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
  // This CTA's partial [tokens, 128] in fp32, over the ring, once its last MMA has read it
  // and (the producer's last waits) its last copy has landed.
  if (!mbar_wait(&acc_full, 0)) record_status(status, kStatusTimeout, 24);
  tc_fence_after();
  __syncthreads();
  float* partial = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quarter = warp & 3;
    for (int c = 0; c < p.tpad; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < p.tpad) partial[(c + j) * kFtTileW + quarter * 32 + lane] = __uint_as_float(r[j]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (p.split > 1) cluster_sync();
  // The outputs, 8 columns an item, dealt out to the cluster's threads.
  const int rows = min(p.tpad, p.T - t0);
  const uint32_t base = smem_u32(partial);
  constexpr int kItems = (GATED ? kFtTileW / 2 : kFtTileW) / 8;  // of a token
  for (int i = rank * kFtThreads + (int)threadIdx.x; i < rows * kItems; i += p.split * kFtThreads) {
    const int t = i / kItems, c = (i - t * kItems) * 8, col = n0 + c;
    if (col >= p.N) continue;
    const int64_t row = t0 + t;
    const uint32_t at = base + (uint32_t)(t * kFtTileW + c) * 4;
    float v[8];
    ft_sum8(at, p.split, v);
    if constexpr (GATED) {
      float u[8];
      ft_sum8(at + kFtTileW / 2 * 4, p.split, u);
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
    } else {
      float bb[8] = {0, 0, 0, 0, 0, 0, 0, 0}, res[8];
      if (p.bias != nullptr) ld_bf16x8(p.bias + col, bb);
      ld_bf16x8(p.R + row * p.N + col, res);
      const uint32_t keep = p.drop.thr == 0 ? 0xffu : dropout_keep8(p.drop, row, col);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = res[j] + (((keep >> j) & 1u) ? (v[j] + bb[j]) * p.drop.scale : 0.0f);
    }
    st_bf16x8(p.out + row * p.N + col, v);
  }
  if (p.split > 1) cluster_sync();  // the peers have read this CTA's partial
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<false>(tmem, tmem_cols);
  }
}

}  // namespace gbmlp
