// Host side of the gated block's forward for few tokens: the shape of the launches.
// Included by gb_mlp.cu inside its anonymous namespace.
#pragma once

// Up to this many tokens the forward's two products take the few-token launches, beyond
// them the GEMMs with shared-out reductions.  Measured, few-token / GEMM (us, both products):
// G, U and the gate: 48 tokens at h 4096, ffn 16384 69 / 75, 96 tokens 79 / 80, 160 tokens
// 124 / 96; h 2048, ffn 5464 27 / 34, 36 / 39, 46 / 39.  O: 48 tokens 69 / 76 and 27 / 29,
// 96 tokens 80 / 82 and 36 / 35, 160 tokens 96 / 93 and 39 / 35.
constexpr int kFewTokensGates = 128;
constexpr int kFewTokensOut = 64;

template <bool GATED>
int launch_few_tokens(DeviceState* st, const uint16_t* W, const uint16_t* X, FewTokensParams p, cudaStream_t s,
                      int trace_kind) {
  p.tpad = 16;
  while (p.tpad < p.T && p.tpad < kFtMaxTokens) p.tpad *= 2;
  const int tiles = (p.N + (GATED ? 64 : 128) - 1) / (GATED ? 64 : 128), num_kb = (p.K + kBK - 1) / kBK;
  const int token_tiles = (p.T + p.tpad - 1) / p.tpad;
  // A stage is 16 KB of weights and 128 bytes a token; two CTAs to an SM share its 227 KB.
  const int stage_bytes = (int)kFtWBytes + p.tpad * kBK * 2;
  p.stages = (int)(110 * 1024 / stage_bytes);
  if (p.stages > kFtMaxStages) p.stages = kFtMaxStages;
  const int smem = p.stages * stage_bytes + 1024;
  // CTAs share a tile's reduction until two to an SM are at work, each with 4 k-blocks or more.
  int64_t split = 2 * (int64_t)st->sms / ((int64_t)tiles * token_tiles);
  if (split > num_kb / 4) split = num_kb / 4;
  p.split = split < 1 ? 1 : split > kFtMaxSplit ? kFtMaxSplit : (int)split;
  CUtensorMap mW, mX;
  int rc = GATED ? make_half_map(&mW, W, p.N, p.K, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
                 : make_map(&mW, W, p.N, p.K, p.N, 64, kBK);
  if (!rc) rc = make_map(&mX, X, p.K, p.T, p.K, kBK, (uint32_t)p.tpad);
  if (rc) return rc;
  auto kern = k_few_tokens<GATED>;
  bool& ready = st->few_attr[GATED ? 1 : 0];
  if (!ready) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 111 * 1024);
    if (e != cudaSuccess) return fail(MLP_ECUDA, "cudaFuncSetAttribute (few tokens): %s", cudaGetErrorString(e));
    ready = true;
  }
  const int ts = trace_pre(s);
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)(tiles * p.split), (unsigned)token_tiles), dim3(kFtThreads),
                                      (size_t)smem, s, (unsigned)p.split, 1, mW, mX, p, st->status);
  trace_post(ts, s, trace_kind, p.T, p.N, p.K);
  return launch_check(e, "few-token product");
}
