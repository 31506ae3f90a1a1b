// Host side of the key/value cache: argument checks and launches.  Included by gb_mlp.cu
// inside its anonymous namespace.
#pragma once

static_assert(kKaWsRows == KV_ATTN_WS_ROWS, "the header's workspace");

// Blocks of bs tokens, `blocks` of them, for nk heads of size d.
int check_kv_cache(const char* what, int nk, int d, int bs, int blocks) {
  if (nk <= 0 || nk > 65536) return fail(MLP_EINVAL, "%s: nk = %d must be in [1, 65536]", what, nk);
  if (d <= 0 || d % 32 != 0) return fail(MLP_EINVAL, "%s: head size d = %d must be a positive multiple of 32", what, d);
  if (d > kKvMaxHead) return fail(MLP_EUNSUPPORTED, "%s: head size d = %d is above %d", what, d, kKvMaxHead);
  if (bs != 16 && bs != 32 && bs != 64) return fail(MLP_EINVAL, "%s: blocks of %d tokens: 16, 32 or 64 are taken", what, bs);
  if (blocks <= 0 || (int64_t)blocks * bs >= (int64_t)1 << 31)
    return fail(MLP_EINVAL, "%s: %d blocks of %d tokens: at least one, and fewer than 2^31 tokens", what, blocks, bs);
  return MLP_OK;
}

int kv_log2(int bs) { return bs == 16 ? 4 : bs == 32 ? 5 : 6; }

int check_kv_table(const char* what, int n, int width, int bs) {
  if (n <= 0 || n > kKvMaxRequests) return fail(MLP_EINVAL, "%s: n = %d requests must be in [1, %d]", what, n, kKvMaxRequests);
  if (width <= 0 || (int64_t)width * bs >= (int64_t)1 << 31)
    return fail(MLP_EINVAL, "%s: a table of %d blocks of %d tokens: at least one, and fewer than 2^31 tokens", what, width, bs);
  return MLP_OK;
}

// Pointers to 4-byte elements.
int check_kv_words(const char* what, std::initializer_list<std::pair<const char*, const void*>> ptrs) {
  for (const auto& p : ptrs) {
    if (p.second == nullptr) return fail(MLP_EINVAL, "%s: %s is NULL", what, p.first);
    if ((reinterpret_cast<uintptr_t>(p.second) & 3) != 0) return fail(MLP_EALIGN, "%s: %s is not 4-byte aligned", what, p.first);
  }
  return MLP_OK;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// Rows of `wide` 2-byte elements, lda and ldb apart, that may have elements in common.  (Slices of one buffer's rows do not:
// their distance, less whole rows of it, leaves each the room that it takes.)
bool overlap_rows(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t wide) {
  if (!overlap(a, 2 * ((rows - 1) * lda + wide), b, 2 * ((rows - 1) * ldb + wide))) return false;
  const int64_t pitch = std::gcd(lda, ldb);
  int64_t apart = ((intptr_t)b - (intptr_t)a) / 2 % pitch;
  if (apart < 0) apart += pitch;
  return apart < wide || pitch - apart < wide;
}

template <int D>
int launch_kv_write_t(KvWriteParams& p, int64_t ctas, cudaStream_t s) {
  const int ts = trace_pre(s);
  auto kern = p.log_bs == 4 ? k_kv_write<D, 16> : p.log_bs == 5 ? k_kv_write<D, 32> : k_kv_write<D, 64>;
  const cudaError_t e = launch_kernel(kern, dim3((unsigned)ctas), dim3(4 << p.log_bs), 0, s, 1, 1, p);
  trace_post(ts, s, kTraceKvWrite, p.tokens, 2 * (int64_t)p.nk * D, 0);
  return launch_check(e, "cache write");
}

int launch_kv_write(const DeviceState* st, KvWriteParams& p, int d, cudaStream_t s) {
  // A CTA for each token and head gives a step's single tokens the most CTAs at once.  Of more than two loads of CTAs,
  // each takes up to a block's tokens, so that prompts have no CTAs that find no run beginning, and then several heads, which
  // know where their tokens go.  (753 tokens of 128 heads: 20.1 us; 22.7 with twice as many CTAs, 22.1 with half.)
  const int64_t heads = 2 * (int64_t)p.nk, full = (int64_t)st->sms * (512 >> p.log_bs);
  p.chunk = 1;
  while (p.chunk < 1 << p.log_bs && p.tokens * heads >= full * p.chunk) p.chunk *= 2;
  const int64_t chunks = (p.tokens + p.chunk - 1) / p.chunk;
  p.span = (int)std::max<int64_t>(1, std::min<int64_t>(chunks * heads / full, 8));
  const int64_t ctas = chunks * ((heads + p.span - 1) / p.span);
  if (ctas >= (int64_t)1 << 31) return fail(MLP_EUNSUPPORTED, "kv_write: %lld tokens of %d heads are too many for a launch", (long long)p.tokens, p.nk);
  switch (d / 32) {
    case 1: return launch_kv_write_t<32>(p, ctas, s);
    case 2: return launch_kv_write_t<64>(p, ctas, s);
    case 3: return launch_kv_write_t<96>(p, ctas, s);
    case 4: return launch_kv_write_t<128>(p, ctas, s);
    case 5: return launch_kv_write_t<160>(p, ctas, s);
    case 6: return launch_kv_write_t<192>(p, ctas, s);
    case 7: return launch_kv_write_t<224>(p, ctas, s);
    default: return launch_kv_write_t<256>(p, ctas, s);
  }
}

template <int D, int NT>
int launch_kv_attn_t(DeviceState* st, const KvAttnParams& p, cudaStream_t s) {
  auto kern = k_kv_attn<D, NT>;
  constexpr int smem = KaShape<D, NT>::kBytes;
  int ctas;
  {
    std::lock_guard<std::mutex> lock(g_setup_mu);
    int& per_sm = st->kv_per_sm[D / 32 - 1][NT - 1];
    if (per_sm == 0) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      int n = 0;
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kKaThreads, smem);
      if (e != cudaSuccess || n < 1) return fail(MLP_ECUDA, "cache attention: %s", cudaGetErrorString(e));
      per_sm = n;
    }
    ctas = std::min(per_sm * st->sms, ka_max_ctas(8 * NT, D));
  }
  int ts = trace_pre(s);
  cudaError_t e = launch_kernel(kern, dim3(ctas), dim3(kKaThreads), smem, s, 1, 1, p);
  trace_post(ts, s, kTraceKvAttn, p.rows, (int64_t)p.nq * D, 0);
  const int rc = launch_check(e, "cache attention");
  // (a table of fewer steps than two parts have: no tile is cut)
  if (rc || (((int64_t)p.width << p.log_bs) + kKaStep - 1) / kKaStep < 2 * kKaMinPart) return rc;
  ts = trace_pre(s);
  e = launch_kernel(k_kv_attn_join<D, NT>, dim3(ctas), dim3(32 * kKaJoinWarps), 0, s, 1, 1, p);
  trace_post(ts, s, kTraceKvJoin, ctas, D, 0);
  return launch_check(e, "cache attention, joining");
}

template <int D>
int launch_kv_attn_d(DeviceState* st, const KvAttnParams& p, cudaStream_t s) {
  // Tiles of 8, 16 or, where the sums fit in registers, 24 rows, for a request's rows on average, unused ones
  // of the buffer among them (the header says what those cost).  A tile of 24 takes
  // 5/4 of the time of one of 16 (16 requests of 3000 to 9000 tokens: 17 us and 21 us a tile, 31 us a call with
  // 16 rows; with 40 rows 65 us in tiles of 16, 57 us in tiles of 24; with 32 48 us and 57 us).
  const int64_t rows = (p.rows + p.n - 1) / p.n * p.group;
  if (rows <= 8) return launch_kv_attn_t<D, 1>(st, p, s);
  if constexpr (D <= 128) {
    if ((rows + 23) / 24 * 5 < (rows + 15) / 16 * 4) return launch_kv_attn_t<D, 3>(st, p, s);
  }
  return launch_kv_attn_t<D, 2>(st, p, s);
}

int launch_kv_attn(DeviceState* st, const KvAttnParams& p, int d, cudaStream_t s) {
  switch (d / 32) {
    case 1: return launch_kv_attn_d<32>(st, p, s);
    case 2: return launch_kv_attn_d<64>(st, p, s);
    case 3: return launch_kv_attn_d<96>(st, p, s);
    case 4: return launch_kv_attn_d<128>(st, p, s);
    case 5: return launch_kv_attn_d<160>(st, p, s);
    case 6: return launch_kv_attn_d<192>(st, p, s);
    case 7: return launch_kv_attn_d<224>(st, p, s);
    default: return launch_kv_attn_d<256>(st, p, s);
  }
}
