// Host side of the gated block's products for few tokens: the shape of the launches.
// Included by gb_mlp.cu inside its anonymous namespace.
#pragma once

// Shared memory of a CTA: half of an SM's.
constexpr int kFtSmem = 110 * 1024;

// Whether a product of the gated block over `weight_bytes` of weights takes the few-token
// launch rather than the GEMMs of 256 x 256 tiles: where its tokens fit one tile of 64, and
// beyond while the weights, read from L2 once for each 64 tokens, stay under a limit: for a
// pass's first product (G, U and the gate, or dG and dU) of up to 512 tokens 64 MB, for its
// second (O, or dX, with `cols` columns) 96 MB where its outputs are those of a tile for a
// quarter of the SMs or less (with more, the GEMMs fill the SMs).  Measured, few-token / GEMM
// (us of a pass, the other product alike):
//   both   48 tokens, h 4096, ffn 16384 66 / 77; h 2048, ffn 5464 21 / 36
//   first  200 tokens, h 1024, ffn 4096 18 / 21; 192 tokens, h 2048, ffn 5464 34 / 31; 1600
//          tokens, h 640, ffn 1280 24 / 19; backward: 256 tokens, h 1024, ffn 4096 22 / 25, h
//          376, ffn 4752 17 / 20; 1024 tokens, h 376, ffn 4752 47 / 37
//   second 400 tokens, h 1024, ffn 4096 23 / 29; 192 tokens, h 4096, ffn 16384 109 / 92; 1600
//          tokens, h 1032, ffn 2744 53 / 44; backward: 128 tokens, h 2048, ffn 5464 28 / 37;
//          512 tokens, h 376, ffn 4752 24 / 34; 1024 tokens, h 1024, ffn 4096 43 / 40
//          and by the outputs, in tiles of 256 x 256: 8 (1024 tokens, h 512, ffn 1024) 16 / 20;
//          8 (2048, 256, 2048) 20 / 26; 24 (2048, 768, 1536) 27 / 29; 32 (4096, 512, 1024)
//          25 / 26; 35 (1500, 1536, 640) 23 / 27; 40 (1024, 2560, 512) 31 / 28; 40 (4096, 640,
//          1144) 37 / 32; 47 (3000, 1024, 512) 28 / 24; 64 (65536, 64, 256) 59 / 48; backward: 8
//          (1024, 512, 1024) 20 / 26; 35 (1500, 1536, 640) 26 / 28; 40 (1024, 2560, 512) 33 / 28;
//          64 (65536, 64, 256) 75 / 58
bool few_tokens_first(int T, int64_t weight_bytes) {
  return T <= 64 || (T <= 512 && (T + 63) / 64 * weight_bytes <= 64ll << 20);
}
bool few_tokens_second(const DeviceState* st, int T, int cols, int64_t weight_bytes) {
  return T <= 64 || ((int64_t)T * cols <= (int64_t)(st->sms / 4) << 16 && (T + 63) / 64 * weight_bytes <= 96ll << 20);
}

template <int KIND>
int launch_few_tokens(DeviceState* st, const uint16_t* W, const uint16_t* X, FewTokensParams p, cudaStream_t s,
                      int trace_kind) {
  constexpr bool GATED = KIND == kFtGates, W_MN = KIND == kFtGates || KIND == kFtOut;
  p.tpad = 16;
  while (p.tpad < p.T && p.tpad < kFtMaxTokens) p.tpad *= 2;
  const int tiles = (p.N + (GATED ? 64 : 128) - 1) / (GATED ? 64 : 128), num_kb = (p.K + kBK - 1) / kBK;
  const int token_tiles = (p.T + p.tpad - 1) / p.tpad;
  // CTAs share a tile's reduction until two to an SM are at work, each with 4 k-blocks or
  // more.  A stage is 16 KB of weights and 128 bytes a token; two CTAs share an SM's 227 KB,
  // with three stages each or more beside what they are sent (a CTA by itself leaves its
  // sums in its own ring).  27 tokens at h 2048, ffn 5464: 19 us; with CTAs for 1.25 or 1.5
  // to an SM 1 us more, with three small CTAs to an SM (two stages each) 13 us more.
  const int rows = p.T < p.tpad ? p.T : p.tpad, stage_bytes = (int)kFtWBytes + p.tpad * kBK * 2;
  int64_t split = 2 * (int64_t)st->sms / ((int64_t)tiles * token_tiles);
  if (split > num_kb / 4) split = num_kb / 4;
  p.split = split < 1 ? 1 : split > kFtMaxSplit ? kFtMaxSplit : (int)split;
  int sent_bytes;
  for (;; --p.split) {
    p.per_log2 = 0;
    while ((p.split << p.per_log2) < rows) ++p.per_log2;
    sent_bytes = p.split > 1 ? (p.split << p.per_log2) * kFtTileW * 4 : 0;
    p.stages = (kFtSmem - sent_bytes) / stage_bytes;
    if (p.split == 1 || p.stages >= 3) break;
  }
  if (p.stages > kFtMaxStages) p.stages = kFtMaxStages;
  const int smem = p.stages * stage_bytes + sent_bytes + 1024;
  CUtensorMap mW, mX;
  int rc = GATED ? make_half_map(&mW, W, p.N, p.K, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
           : W_MN ? make_map(&mW, W, p.N, p.K, p.N, 64, kBK)
                  : make_map(&mW, W, p.K, p.N, p.K, kBK, kFtTileW);
  if (!rc) rc = make_map(&mX, X, p.K, p.T, p.K, kBK, (uint32_t)p.tpad);
  if (rc) return rc;
  auto kern = k_few_tokens<KIND>;
  {
    std::lock_guard<std::mutex> lock(g_setup_mu);
    bool& ready = st->few_attr[KIND];
    if (!ready) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFtSmem + 1024);
      if (e != cudaSuccess) return fail(MLP_ECUDA, "cudaFuncSetAttribute (few tokens): %s", cudaGetErrorString(e));
      ready = true;
    }
  }
  const int ts = trace_pre(s);
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)(tiles * token_tiles * p.split)), dim3(kFtThreads),
                                      (size_t)smem, s, (unsigned)p.split, 1, mW, mX, p, st->status);
  trace_post(ts, s, trace_kind, p.T, p.N, p.K);
  return launch_check(e, "few-token product");
}
