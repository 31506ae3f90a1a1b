// Host side of the head norms with position rotation: argument checks, the share of a
// warp, and the launches.  Included by gb_mlp.cu inside its anonymous namespace.
#pragma once

// The rotation and the norm as the entry points take them.
struct QkRopeArgs {
  int rot, interleaved, n_axes, s0, s1, s2;
  float eps;
  const uint16_t* wq;
  const uint16_t* wk;
  const int32_t* pos;
  const float* inv_freq;
};

// One [tokens, heads, d] tensor: rows of `heads` vectors, `ld` elements apart.
int check_qk_rows(const char* what, const char* name, const void* p, int64_t ld, int heads, int d) {
  if (p == nullptr) return fail(MLP_EINVAL, "%s: %s is NULL", what, name);
  if (!aligned16(p)) return fail(MLP_EALIGN, "%s: %s is not 16-byte aligned", what, name);
  if (ld < (int64_t)heads * d || ld % 8 != 0)
    return fail(MLP_EINVAL, "%s: the row stride of %s (%lld) must be a multiple of 8 and at least heads * d = %lld", what,
                name, (long long)ld, (long long)heads * d);
  return MLP_OK;
}

int check_qk_rope(const char* what, int64_t tokens, int nq, int nk, int d, const QkRopeArgs& r) {
  if (tokens <= 0 || tokens >= (int64_t)1 << 31) return fail(MLP_EINVAL, "%s: tokens = %lld out of range", what, (long long)tokens);
  if (nq <= 0 || nk <= 0 || nq > 65536 || nk > 65536)
    return fail(MLP_EINVAL, "%s: nq = %d and nk = %d must be in [1, 65536]", what, nq, nk);
  if (d <= 0 || d % 8 != 0) return fail(MLP_EINVAL, "%s: head size d = %d must be a positive multiple of 8", what, d);
  if (d > kQkMaxHead) return fail(MLP_EUNSUPPORTED, "%s: head size d = %d is above %d", what, d, kQkMaxHead);
  if (r.rot <= 0 || r.rot > d || r.rot % 8 != 0)
    return fail(MLP_EINVAL, "%s: rot = %d must be a multiple of 8 in [8, d = %d]", what, r.rot, d);
  if (r.interleaved != 0 && r.interleaved != 1) return fail(MLP_EINVAL, "%s: interleaved = %d not in {0, 1}", what, r.interleaved);
  const int s[3] = {r.s0, r.s1, r.s2};
  if (r.n_axes < 1 || r.n_axes > 3) return fail(MLP_EINVAL, "%s: n_axes = %d not in [1, 3]", what, r.n_axes);
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || (i >= r.n_axes && s[i] != 0))
      return fail(MLP_EINVAL, "%s: section %d = %d of %d axes", what, i, s[i], r.n_axes);
    sum += s[i];
  }
  if (sum != r.rot / 2)
    return fail(MLP_EINVAL, "%s: the sections (%d, %d, %d) must add up to rot / 2 = %d pairs", what, r.s0, r.s1, r.s2, r.rot / 2);
  if (!(r.eps >= 0.0f)) return fail(MLP_EINVAL, "%s: eps = %g must be >= 0", what, (double)r.eps);
  if ((r.wq == nullptr) != (r.wk == nullptr)) return fail(MLP_EINVAL, "%s: wq and wk must both be given or both be NULL", what);
  if (r.wq != nullptr && (!aligned16(r.wq) || !aligned16(r.wk)))
    return fail(MLP_EALIGN, "%s: wq and wk must be 16-byte aligned", what);
  if (r.pos == nullptr || r.inv_freq == nullptr) return fail(MLP_EINVAL, "%s: pos or inv_freq is NULL", what);
  if ((reinterpret_cast<uintptr_t>(r.pos) & 3) != 0 || (reinterpret_cast<uintptr_t>(r.inv_freq) & 3) != 0)
    return fail(MLP_EALIGN, "%s: pos and inv_freq must be 4-byte aligned", what);
  return MLP_OK;
}

void fill_qk_rope(QkRopeParams* p, int64_t tokens, int nq, int nk, int d, const QkRopeArgs& r) {
  p->tokens = tokens;
  p->nq = nq;
  p->nk = nk;
  p->d = d;
  p->rot = r.rot;
  p->axis1 = r.s0;
  p->axis2 = r.s0 + r.s1;
  p->eps = r.eps;
  p->wq = r.wq;
  p->wk = r.wk;
  p->pos = r.pos;
  p->inv_freq = r.inv_freq;
}

// The steps of a token, and the grid: a step for each warp, at most ctas_per_sm CTAs an SM.
unsigned plan_qk_rope(const DeviceState* st, QkRopeParams* p, int vec, int ctas_per_sm) {
  const int hpw = 32 / (p->d / (2 * vec));
  p->steps_q = (p->nq + hpw - 1) / hpw;
  p->steps_k = (p->nk + hpw - 1) / hpw;
  const int64_t ctas = (p->tokens * (p->steps_q + p->steps_k) + kQkWarps - 1) / kQkWarps;
  const int64_t most = (int64_t)st->sms * ctas_per_sm;
  return (unsigned)(ctas < most ? ctas : most);
}

bool qk_wide(int d, int rot) { return d % 16 == 0 && rot % 16 == 0; }  // vectors of 8 elements, else 4

template <int VEC, bool INTER, bool NORM, bool BWD>
int launch_qk_t(DeviceState* st, QkRopeParams& p, cudaStream_t s, unsigned* ctas) {
  auto kern = k_qk_norm_rope<VEC, INTER, NORM, BWD>;
  constexpr int smem = QkSmem<VEC, BWD, NORM>::kBytes;
  int ctas_per_sm;
  {
    std::lock_guard<std::mutex> lock(g_setup_mu);
    int& per_sm = st->qk_per_sm[(VEC == 8 ? 8 : 0) + (INTER ? 4 : 0) + (NORM ? 2 : 0) + (BWD ? 1 : 0)];
    if (per_sm == 0) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      int n = 0;
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kQkThreads, smem);
      if (e != cudaSuccess || n < 1) return fail(MLP_ECUDA, "head norms and rotation: %s", cudaGetErrorString(e));
      per_sm = n < kQkMaxPerSm ? n : kQkMaxPerSm;
    }
    ctas_per_sm = per_sm;
  }
  *ctas = plan_qk_rope(st, &p, VEC, ctas_per_sm);
  const int ts = trace_pre(s);
  const cudaError_t e = launch_kernel(kern, dim3(*ctas), dim3(kQkThreads), smem, s, 1, 1, p);
  trace_post(ts, s, BWD ? kTraceQkRopeBwd : kTraceQkRope, p.tokens, (int64_t)(p.nq + p.nk) * p.d, 0);
  return launch_check(e, "head norms and rotation");
}

template <bool BWD>
int launch_qk(DeviceState* st, QkRopeParams& p, int interleaved, cudaStream_t s, unsigned* ctas) {
  const bool norm = p.wq != nullptr;
  if (qk_wide(p.d, p.rot)) {
    if (interleaved) return norm ? launch_qk_t<8, true, true, BWD>(st, p, s, ctas) : launch_qk_t<8, true, false, BWD>(st, p, s, ctas);
    return norm ? launch_qk_t<8, false, true, BWD>(st, p, s, ctas) : launch_qk_t<8, false, false, BWD>(st, p, s, ctas);
  }
  if (interleaved) return norm ? launch_qk_t<4, true, true, BWD>(st, p, s, ctas) : launch_qk_t<4, true, false, BWD>(st, p, s, ctas);
  return norm ? launch_qk_t<4, false, true, BWD>(st, p, s, ctas) : launch_qk_t<4, false, false, BWD>(st, p, s, ctas);
}

int launch_qk_rope(DeviceState* st, QkRopeParams p, int interleaved, cudaStream_t s) {
  unsigned ctas = 0;
  return launch_qk<false>(st, p, interleaved, s, &ctas);
}

int launch_qk_rope_bwd(DeviceState* st, QkRopeParams p, int interleaved, float* dwq, float* dwk, int accumulate,
                       cudaStream_t s) {
  unsigned ctas = 0;
  const int rc = launch_qk<true>(st, p, interleaved, s, &ctas);
  if (rc || p.wq == nullptr) return rc;
  const int ts = trace_pre(s);
  const cudaError_t e = launch_kernel(k_qk_dw, dim3((2 * p.d + 31) / 32), dim3(1024), 0, s, 1, 1, (const float*)p.ws,
                                      (int)ctas, p.d, dwq, dwk, accumulate);
  trace_post(ts, s, kTraceQkDw, ctas, 2 * p.d, 0);
  return launch_check(e, "head norm weight gradients");
}
