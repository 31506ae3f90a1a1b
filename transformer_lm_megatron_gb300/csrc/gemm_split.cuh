// The gated block's GEMMs of few tiles: one tile to a cluster of 2 to 4 CTA pairs that
// share its reduction.
//
// A GEMM of, say, 30 tiles of 256 x 256 keeps 60 of 152 SMs busy in k_gemm_bf16_tc,
// whatever its reduction.  Here a cluster of `split` pairs takes one tile: pair q the
// k-blocks [num_kb q / split, num_kb (q + 1) / split), with the same operand tiles, TMA
// copies and cta_group::2 MMAs as there.  Each CTA then leaves its fp32 partial [128, 256]
// in its shared memory (the ring, free by then), and the CTAs that hold the same rows
// share them out, add the partials in pair order through distributed shared memory and
// write the epilogue's result with whole rows of coalesced 16-byte accesses.  The order
// of additions is fixed by the shape; no memory outside the CTAs is used.
// 1317 tokens, h 1032 from a reduction of 5488 (30 tiles, 86 k-blocks): 29 us of main
// loop and epilogue in k_gemm_bf16_tc, of which 22 are the k-blocks; the pass that it is
// part of (the input gradient at ffn 2744) takes 40 us for 53.  It is bounded by what a
// tile costs besides its k-blocks (first bytes, the exchange of partials, the outputs).
#pragma once
#include <cstdint>
#include <cuda.h>

#include "few_tokens.cuh"
#include "gemm_tc.cuh"

namespace gbmlp {

constexpr int kGsThreads = 320;    // warps 0 TMA producer, 1 TMEM owner and MMA issuer, 2..9 TMEM to shared memory
constexpr int kGsStages = 6;
constexpr int kGsPitch = kBN + 4;  // floats: rows 16 bytes off each other's banks
constexpr uint32_t kGsStageBytes = kABytes + (kBN / 2) * kBK * 2;
constexpr int kGsMaxSplit = 4;
constexpr int kGsBatch = 4;        // items of a thread whose inputs are fetched together
constexpr size_t kGsSmemBytes = (size_t)kGsStages * kGsStageBytes + 1024;
static_assert(kBM * kGsPitch * 4 <= kGsStages * kGsStageBytes, "the partial fits the ring");

// 8 consecutive values of the partial at `at`, summed over the CTAs of the cluster that
// hold the same rows, in pair order.
__device__ __forceinline__ void gs_sum8(uint32_t at, int split, uint32_t half, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 2
  for (int r = 0; r < split; ++r) {
    const uint32_t a = mapa_shared(at, 2 * r + half);
    const float4 x = ld_cluster_f4(a), y = ld_cluster_f4(a + 16);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float (&v)[8]) {
  v[0] = bf16lo(q.x), v[1] = bf16hi(q.x), v[2] = bf16lo(q.y), v[3] = bf16hi(q.y);
  v[4] = bf16lo(q.z), v[5] = bf16hi(q.z), v[6] = bf16lo(q.w), v[7] = bf16hi(q.w);
}

// One item of the epilogue is 8 columns of one row.  What it reads from global memory is
// fetched for several items before the first is worked on: a = the residual, or G, and b = U.
__device__ __forceinline__ void gs_fetch(const EpiParams& ep, int64_t row, int col, int N, uint4& a, uint4& b) {
  if (ep.kind == kEpiDGlu) {
    const uint16_t* p = ep.in0 + row * 2 * N + col;
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + N);
  } else if (ep.kind == kEpiDropRes || (ep.kind == kEpiResAdd && ep.in0 != nullptr)) {
    a = *reinterpret_cast<const uint4*>(ep.in0 + row * ep.ld + col);
  }
}

// v = the item's sums.
__device__ __forceinline__ void gs_epilogue(const EpiParams& ep, int64_t row, int col, int N, const uint4& a,
                                            const uint4& b, float (&v)[8]) {
  const int64_t off = row * ep.ld + col;
  float x[8];
  switch (ep.kind) {
    case kEpiDropRes: {
      float bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (ep.bias != nullptr) ld_bf16x8(ep.bias + col, bias);
      unpack_bf16x8(a, x);
      const uint32_t keep = ep.drop.thr == 0 ? 0xffu : dropout_keep8(ep.drop, row, col);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x[j] + (((keep >> j) & 1u) ? (v[j] + bias[j]) * ep.drop.scale : 0.0f);
      st_bf16x8(ep.out0 + off, v);
      break;
    }
    case kEpiResAdd:
      if (ep.in0 != nullptr) {
        unpack_bf16x8(a, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += x[j];
      }
      st_bf16x8(ep.out0 + off, v);
      break;
    case kEpiDGlu: {
      float g[8], u[8], dg[8], du[8];
      const int64_t at = row * 2 * N + col;
      unpack_bf16x8(a, g);
      unpack_bf16x8(b, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float value, slope;
        if (ep.act == kActSilu)
          silu_both_f(g[j], value, slope);
        else
          gelu_both_f(g[j], value, slope);
        dg[j] = v[j] * u[j] * slope;
        du[j] = v[j] * value;
      }
      st_bf16x8(ep.out0 + at, dg);
      st_bf16x8(ep.out0 + at + N, du);
      break;
    }
    default: {  // kEpiF32Store, kEpiF32Add
      float4* p = reinterpret_cast<float4*>(ep.g_out + off);
      float4 s = make_float4(v[0], v[1], v[2], v[3]), t = make_float4(v[4], v[5], v[6], v[7]);
      if (ep.kind == kEpiF32Add) {
        const float4 c = p[0], d = p[1];
        s.x += c.x, s.y += c.y, s.z += c.z, s.w += c.w;
        t.x += d.x, t.y += d.y, t.z += d.z, t.w += d.w;
      }
      p[0] = s;
      p[1] = t;
    }
  }
}

// The gate's item: 8 columns of G (v) and U of one row.
__device__ __forceinline__ void gs_glu(const EpiParams& ep, int64_t row, int col, int N, float (&v)[8], float (&u)[8]) {
  if (ep.bias != nullptr) {
    float bg[8], bu[8];
    ld_bf16x8(ep.bias + col, bg);
    ld_bf16x8(ep.bias + N + col, bu);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] += bg[j];
      u[j] += bu[j];
    }
  }
  if (ep.out0 != nullptr) {
    st_bf16x8(ep.out0 + row * 2 * N + col, v);
    st_bf16x8(ep.out0 + row * 2 * N + N + col, u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (ep.act == kActSilu ? silu_f(v[j]) : gelu_gate_f(v[j])) * u[j];
  st_bf16x8(ep.out1 + row * N + col, v);
}

// Operand layouts and GATED as for k_gemm_bf16_tc.  Grid tiles * 2 * split, clusters of
// 2 * split CTAs; late_wait as there; tile t is row block t % num_m, column block t / num_m.
template <bool A_MN, bool B_MN, int GATED>
__global__ void __launch_bounds__(kGsThreads, 1)
    k_gemm_split(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, int M, int N, int K,
                 EpiParams ep, int split, int num_m, int late_wait, int* status) {
  constexpr int kTileN = GATED == kGatedFwd ? kBN / 2 : kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kGsStages * kABytes;
  __shared__ uint64_t full[kGsStages], empty[kGsStages], acc_full;
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), leader = rank & ~1u, half = rank & 1u;
  const int q = (int)(rank >> 1);
  const int tile = (int)(blockIdx.x / (unsigned)(2 * split));
  const int m0 = (tile % num_m) * 2 * kBM + (int)half * kBM, n0 = (tile / num_m) * kTileN;
  const int num_kb = (K + kBK - 1) / kBK;
  const int kb0 = (int)((int64_t)num_kb * q / split), kb1 = (int)((int64_t)num_kb * (q + 1) / split);
  const uint16_t pair_mask = (uint16_t)(3u << leader);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc<true>(&tmem_slot, kBN);
    tmem_relinquish<true>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every barrier of the cluster is initialised
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (!late_wait) grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t issued[kGsStages];
#pragma unroll
      for (int s = 0; s < kGsStages; ++s) issued[s] = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1)) {
          record_status(status, kStatusTimeout, 31);
          ok = false;
          break;
        }
        const int k0 = kb * kBK;
        uint8_t* a_dst = sA + stage * kABytes;
        uint8_t* b_dst = sB + stage * (kGsStageBytes - kABytes);
        // both CTAs' copies complete on the even CTA's barrier, which expects both
        const uint32_t bar = mapa_shared(smem_u32(&full[stage]), leader);
        if (half == 0) mbar_arrive_expect_tx(&full[stage], 2 * kGsStageBytes);
        if constexpr (A_MN) {
#pragma unroll
          for (int j = 0; j < kBM / 64; ++j)
            tma_load_2d_pair(a_dst + j * kChunkBytes, &tmA, bar, m0 + 64 * j, k0, 0, false);
        } else {
          tma_load_2d_pair(a_dst, &tmA, bar, k0, m0, 0, false);
        }
        if constexpr (GATED == kGatedFwd) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_3d_pair(b_dst + j * kChunkBytes, &tmB, bar, n0 + 64 * j, (int)half, k0);
        } else if constexpr (B_MN) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_2d_pair(b_dst + j * kChunkBytes, &tmB, bar, n0 + (int)half * (kBN / 2) + 64 * j, k0, 0, false);
        } else {
          tma_load_2d_pair(b_dst, &tmB, bar, k0, n0 + (int)half * (kBN / 2), 0, false);
        }
#pragma unroll
        for (int s = 0; s < kGsStages; ++s) issued[s] += s == stage ? 1 : 0;
        if (++stage == kGsStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // Every copy has landed before the ring is used for anything else, or left.
      if (half == 0) {
#pragma unroll
        for (int s = 0; s < kGsStages; ++s)
          if (issued[s] > 0 && !mbar_wait_cluster(&full[s], (issued[s] - 1) & 1)) record_status(status, kStatusTimeout, 32);
      } else if (!ok) {
        // they complete on the even CTA's barrier: after a failure give them time (bounded)
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(10000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && half == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = make_idesc_bf16(2 * kBM, kBN, A_MN, B_MN);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait_cluster(&full[stage], phase)) {
          record_status(status, kStatusTimeout, 33);
          break;
        }
        tc_fence_after();
        const uint32_t a_base = smem_u32(sA + stage * kABytes);
        const uint32_t b_base = smem_u32(sB + stage * (kGsStageBytes - kABytes));
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
          const uint64_t adesc = A_MN ? make_sdesc_sw128(a_base + kk * 2048, kChunkBytes, 1024)
                                      : make_sdesc_sw128(a_base + kk * 32, 16, 1024);
          const uint64_t bdesc = B_MN ? make_sdesc_sw128(b_base + kk * 2048, kChunkBytes, 1024)
                                      : make_sdesc_sw128(b_base + kk * 32, 16, 1024);
          umma_bf16_pair(tmem, adesc, bdesc, idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
        }
        umma_commit_pair(&empty[stage], pair_mask);
        if (++stage == kGsStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      umma_commit_pair(&acc_full, pair_mask);
    }
    __syncwarp();
  }
  // The CTA's partial [128, 256] in fp32, over the ring: the commit that acc_full waits for
  // follows the pair's last MMA, and that its last copies.
  if (!mbar_wait_cluster(&acc_full, 0)) record_status(status, kStatusTimeout, 34);
  tc_fence_after();
  __syncthreads();
  float* partial = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quarter = warp & 3, c_begin = ((warp - 2) >> 2) * (kBN / 2);
    float* mine = partial + (quarter * 32 + lane) * kGsPitch;
#pragma unroll 1
    for (int c = c_begin; c < c_begin + kBN / 2; c += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(mine + c + 4 * j) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    }
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();
  // This CTA's share of the rows, 8 columns an item, kGsBatch items of a thread at a time.
  const int r_begin = kBM * q / split, r_end = min(kBM * (q + 1) / split, M - m0);
  constexpr int kItems = kTileN / 8;
  const int items = max(r_end - r_begin, 0) * kItems;
  const uint32_t base = smem_u32(partial);
  for (int i0 = threadIdx.x; i0 < items; i0 += kGsBatch * kGsThreads) {
    uint4 a[kGsBatch], b[kGsBatch];
    if constexpr (GATED != kGatedFwd) {
#pragma unroll
      for (int k = 0; k < kGsBatch; ++k) {
        const int i = i0 + k * kGsThreads, col = n0 + (i % kItems) * 8;
        if (i < items && col < N) gs_fetch(ep, (int64_t)m0 + r_begin + i / kItems, col, N, a[k], b[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kGsBatch; ++k) {
      const int i = i0 + k * kGsThreads, r = r_begin + i / kItems, c = (i % kItems) * 8, col = n0 + c;
      if (i >= items || col >= N) continue;
      const uint32_t at = base + (uint32_t)(r * kGsPitch + c) * 4;
      float v[8];
      gs_sum8(at, split, half, v);
      if constexpr (GATED == kGatedFwd) {
        float u[8];
        gs_sum8(at + kTileN * 4, split, half, u);
        gs_glu(ep, (int64_t)m0 + r, col, N, v, u);
      } else {
        gs_epilogue(ep, (int64_t)m0 + r, col, N, a[k], b[k], v);
      }
    }
  }
  cluster_sync();  // the peers have read this CTA's partial, and the pair's MMAs its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<true>(tmem, kBN);
  }
  if (late_wait) grid_dependency_wait();
}

}  // namespace gbmlp
