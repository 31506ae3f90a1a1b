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

// The share of a warp: one token's heads, or fewer while that leaves warps idle.
unsigned plan_qk_rope(const DeviceState* st, QkRopeParams* p, int vec, int ctas_per_sm) {
  const int hpw = 32 / (p->d / (2 * vec)), heads = p->nq + p->nk;
  const int64_t warps = (int64_t)st->sms * ctas_per_sm * kQkWarps;
  const int steps = (heads + hpw - 1) / hpw;  // a warp's steps over one token
  int64_t units = warps / p->tokens;
  if (units < 1) units = 1;
  if (units > steps) units = steps;
  p->heads_per_unit = (int)((steps + units - 1) / units) * hpw;
  p->units = (heads + p->heads_per_unit - 1) / p->heads_per_unit;
  const int64_t ctas = (p->tokens * p->units + kQkWarps - 1) / kQkWarps;
  return (unsigned)(ctas < (int64_t)st->sms * ctas_per_sm ? ctas : (int64_t)st->sms * ctas_per_sm);
}

bool qk_wide(int d, int rot) { return d % 16 == 0 && rot % 16 == 0; }  // vectors of 8 elements, else 4

int launch_qk_rope(DeviceState* st, QkRopeParams p, int interleaved, cudaStream_t s) {
  const int vec = qk_wide(p.d, p.rot) ? 8 : 4;
  const unsigned grid = plan_qk_rope(st, &p, vec, 4);
  const bool norm = p.wq != nullptr;
  const int ts = trace_pre(s);
  cudaError_t e;
#define GB_QK(V_, I_, N_) e = launch_kernel(k_qk_norm_rope<V_, I_, N_>, dim3(grid), dim3(kQkThreads), 0, s, 1, 1, p)
  if (vec == 8) {
    if (interleaved) { if (norm) GB_QK(8, true, true); else GB_QK(8, true, false); }
    else { if (norm) GB_QK(8, false, true); else GB_QK(8, false, false); }
  } else {
    if (interleaved) { if (norm) GB_QK(4, true, true); else GB_QK(4, true, false); }
    else { if (norm) GB_QK(4, false, true); else GB_QK(4, false, false); }
  }
#undef GB_QK
  trace_post(ts, s, kTraceQkRope, p.tokens, (int64_t)(p.nq + p.nk) * p.d, 0);
  return launch_check(e, "head norms and rotation");
}

int launch_qk_rope_bwd(DeviceState* st, QkRopeParams p, int interleaved, float* dwq, float* dwk, int accumulate,
                       cudaStream_t s) {
  const int vec = qk_wide(p.d, p.rot) ? 8 : 4;
  const unsigned grid = plan_qk_rope(st, &p, vec, 4);
  const bool norm = p.wq != nullptr;
  const int ts = trace_pre(s);
  cudaError_t e;
#define GB_QK(V_, I_, N_) e = launch_kernel(k_qk_norm_rope_bwd<V_, I_, N_>, dim3(grid), dim3(kQkThreads), 0, s, 1, 1, p)
  if (vec == 8) {
    if (interleaved) { if (norm) GB_QK(8, true, true); else GB_QK(8, true, false); }
    else { if (norm) GB_QK(8, false, true); else GB_QK(8, false, false); }
  } else {
    if (interleaved) { if (norm) GB_QK(4, true, true); else GB_QK(4, true, false); }
    else { if (norm) GB_QK(4, false, true); else GB_QK(4, false, false); }
  }
#undef GB_QK
  trace_post(ts, s, kTraceQkRopeBwd, p.tokens, (int64_t)(p.nq + p.nk) * p.d, 0);
  int rc = launch_check(e, "head norms and rotation backward");
  if (rc || !norm) return rc;
  const int tw = trace_pre(s);
  e = launch_kernel(k_qk_dw, dim3((2 * p.d + 31) / 32), dim3(1024), 0, s, 1, 1, (const float*)p.ws, (int)grid, p.d, dwq,
                    dwk, accumulate);
  trace_post(tw, s, kTraceQkDw, grid, 2 * p.d, 0);
  return launch_check(e, "head norm weight gradients");
}
