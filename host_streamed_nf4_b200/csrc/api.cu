// api.cu -- the C ABI of libhsnf4.so: argument validation, error reporting,
// the NF4 codebook, and the launch sequences of the LoRA linear.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <memory>
#include <mutex>
#include <new>

#include "internal.h"

namespace hsnf4 {

// ---------------------------------------------------------------- errors

static thread_local char t_detail[512] = "";
static thread_local int t_status = HSNF4_OK;

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_detail, sizeof t_detail, fmt, ap);
  va_end(ap);
  t_status = status;
  return status;
}

int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return HSNF4_OK;
  return fail(HSNF4_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

static std::atomic<int> g_fault{kFaultNone};

bool take_fault(FaultSite site) {
  int expected = site;
  return g_fault.compare_exchange_strong(expected, kFaultNone);
}

// ---------------------------------------------------------------- codebook
// NormalFloat-4, the "nf4" type of the Poros API reference: the 16 float32
// values of the data type as QLoRA (Dettmers et al. 2023) prints them in its
// Appendix E, as IEEE-754 bit patterns, code 0 (-1) up to code 15 (+1).  They
// are standard-normal quantiles at evenly spaced probabilities plus an exact
// zero, normalised to [-1, 1] (the paper's "4-bit NormalFloat Quantization").

static const uint32_t kNf4Bits[16] = {
    0xbf800000u, 0xbf3239b1u, 0xbf066b30u, 0xbeca32a0u, 0xbe91a24du, 0xbe3d353fu,
    0xbdba7871u, 0x00000000u, 0x3da2faffu, 0x3e24cae3u, 0x3e7c04ddu, 0x3ead033au,
    0x3ee1a4b8u, 0x3f1007abu, 0x3f3913b3u, 0x3f800000u,
};

const Nf4Codebook& codebook() {
  static const Nf4Codebook cb = [] {
    Nf4Codebook c;
    memcpy(c.v, kNf4Bits, sizeof c.v);
    return c;
  }();
  return cb;
}

}  // namespace hsnf4

using namespace hsnf4;

// ---------------------------------------------------------------- C ABI

extern "C" {

const char* hsnf4_status_string(int status) {
  switch (status) {
    case HSNF4_OK: return "ok";
    case HSNF4_ERR_INVALID: return "invalid argument";
    case HSNF4_ERR_OOM: return "buffer too small";
    case HSNF4_ERR_CUDA: return "CUDA error";
    case HSNF4_ERR_TIMEOUT: return "timed out";
    case HSNF4_ERR_STATE: return "protocol misuse";
    case HSNF4_ERR_DEVICE: return "device wait gave up";
    default: return "unknown status";
  }
}

int hsnf4_last_error(char* buf, size_t n) {
  if (buf && n) {
    strncpy(buf, t_detail, n - 1);
    buf[n - 1] = 0;
  }
  return t_status;
}

int hsnf4_device_status(void* stream, uint32_t* flags) {
  if (!flags) return fail(HSNF4_ERR_INVALID, "hsnf4_device_status: flags is NULL");
  int rc = cuda_status(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)),
                       "hsnf4_device_status: cudaStreamSynchronize");
  if (rc) return rc;
  uint32_t f = 0, fr = 0, fm = 0, fa = 0;
  rc = cuda_status(read_gemm_flags(&f), "hsnf4_device_status: read flags");
  if (!rc) rc = cuda_status(read_rank_flags(&fr), "hsnf4_device_status: read flags");
  if (!rc) rc = cuda_status(read_merge_flags(&fm), "hsnf4_device_status: read flags");
  if (!rc) rc = cuda_status(read_attn_flags(&fa), "hsnf4_device_status: read flags");
  if (rc) return rc;
  f |= fr | fm | fa;
  *flags = f;
  if (f) return fail(HSNF4_ERR_DEVICE, "a kernel wait gave up (flags 0x%x)", f);
  return HSNF4_OK;
}

int hsnf4_selftest_stall(void* stream) {
  return cuda_status(launch_selftest_stall(static_cast<cudaStream_t>(stream)),
                     "hsnf4_selftest_stall launch");
}

int hsnf4_inject_fault(const char* site) {
  if (!site || !*site) {
    g_fault.store(kFaultNone);
    return HSNF4_OK;
  }
  if (!strcmp(site, "copy_enqueue")) {
    g_fault.store(kFaultCopyEnqueue);
    return HSNF4_OK;
  }
  if (!strcmp(site, "event_record")) {
    g_fault.store(kFaultEventRecord);
    return HSNF4_OK;
  }
  return fail(HSNF4_ERR_INVALID, "hsnf4_inject_fault: unknown site '%s'", site);
}

int nf4_codebook(float* out) {
  if (!out) return fail(HSNF4_ERR_INVALID, "nf4_codebook: out is NULL");
  memcpy(out, codebook().v, sizeof(float) * 16);
  return HSNF4_OK;
}

static int check_nf4_shape(const char* fn, int64_t n_out, int64_t k_in) {
  if (n_out < 1 || k_in < 1 || k_in % 64 != 0)
    return fail(HSNF4_ERR_INVALID,
                "%s: need n_out >= 1 and k_in a positive multiple of 64 (got n_out=%lld, "
                "k_in=%lld)",
                fn, (long long)n_out, (long long)k_in);
  if (n_out > (int64_t(1) << 31) || k_in > (int64_t(1) << 31))
    return fail(HSNF4_ERR_INVALID, "%s: dimension too large", fn);
  return HSNF4_OK;
}

static int check_ptrs(const char* fn, std::initializer_list<std::pair<const void*, const char*>> ps) {
  for (auto& p : ps) {
    if (!p.first) return fail(HSNF4_ERR_INVALID, "%s: %s is NULL", fn, p.second);
    if (!aligned16(p.first))
      return fail(HSNF4_ERR_INVALID, "%s: %s is not 16-byte aligned", fn, p.second);
  }
  return HSNF4_OK;
}

int nf4_quantize_pack(const void* w_bf16, int64_t n_out, int64_t k_in, void* codes,
                      float* absmax, void* stream) {
  int rc = check_nf4_shape("nf4_quantize_pack", n_out, k_in);
  if (rc) return rc;
  rc = check_ptrs("nf4_quantize_pack", {{w_bf16, "w_bf16"}, {codes, "codes"}, {absmax, "absmax"}});
  if (rc) return rc;
  return cuda_status(launch_nf4_quantize(w_bf16, n_out, k_in, codes, absmax,
                                         static_cast<cudaStream_t>(stream)),
                     "nf4_quantize_pack launch");
}

int nf4_dequant(const void* codes, const float* absmax, int64_t n_out, int64_t k_in,
                void* w_bf16_out, void* stream) {
  int rc = check_nf4_shape("nf4_dequant", n_out, k_in);
  if (rc) return rc;
  rc = check_ptrs("nf4_dequant", {{codes, "codes"}, {absmax, "absmax"}, {w_bf16_out, "w_bf16_out"}});
  if (rc) return rc;
  return cuda_status(launch_nf4_dequant(codes, absmax, n_out, k_in, w_bf16_out,
                                        static_cast<cudaStream_t>(stream)),
                     "nf4_dequant launch");
}

// ---------------------------------------------------------------- LoRA linear

static int r_padded(int r) { return (r + 15) / 16 * 16; }

static int check_weight(const char* fn, int i, const hsnf4_nf4_weight& W) {
  if (W.n_out < 64 || W.n_out % 64 || W.k_in < 64 || W.k_in % 64)
    return fail(HSNF4_ERR_INVALID,
                "%s: problem %d: n_out and k_in must be positive multiples of 64 (got %lld x %lld)",
                fn, i, (long long)W.n_out, (long long)W.k_in);
  if (W.n_out > (1 << 30) || W.k_in > (1 << 30))
    return fail(HSNF4_ERR_INVALID, "%s: problem %d: weight dimension too large", fn, i);
  if (W.format == HSNF4_BASE_NF4)
    return check_ptrs(fn, {{W.codes, "W.codes"}, {W.absmax, "W.absmax"}});
  if (W.format == HSNF4_BASE_BF16) {
    if (W.absmax)
      return fail(HSNF4_ERR_INVALID, "%s: problem %d: a BF16 base weight takes absmax = NULL",
                  fn, i);
    return check_ptrs(fn, {{W.codes, "W.codes (bf16 weight)"}});
  }
  return fail(HSNF4_ERR_INVALID, "%s: problem %d: unknown base format %d", fn, i, W.format);
}

// one base format per group (the fused GEMM reads all its problems one way)
static int check_one_format(const char* fn, int n, const int32_t* formats) {
  for (int i = 1; i < n; ++i)
    if (formats[i] != formats[0])
      return fail(HSNF4_ERR_INVALID, "%s: problem %d has base format %d, problem 0 has %d; a "
                  "group takes one format", fn, i, formats[i], formats[0]);
  return HSNF4_OK;
}

static int check_dropout(const char* fn, int i, float p) {
  if (!(p >= 0.0f && p < 1.0f))
    return fail(HSNF4_ERR_INVALID, "%s: problem %d: dropout_p must be in [0, 1) (got %g)", fn, i,
                static_cast<double>(p));
  return HSNF4_OK;
}

static int check_group(const char* fn, int n, int64_t T, int r, float alpha) {
  if (n < 1 || n > 8)
    return fail(HSNF4_ERR_INVALID, "%s: 1..8 problems per call (got %d)", fn, n);
  if (T < 1 || T > 32768)
    return fail(HSNF4_ERR_INVALID, "%s: T must be in [1, 32768] (got %lld)", fn, (long long)T);
  if (r < 8 || r > 64 || r % 8)
    return fail(HSNF4_ERR_INVALID, "%s: rank must be a multiple of 8 in [8, 64] (got %d)", fn, r);
  if (!isfinite(alpha)) return fail(HSNF4_ERR_INVALID, "%s: alpha is not finite", fn);
  return HSNF4_OK;
}

// Workspace layout of a forward group:
//   [s*t bf16 [T, r_pad] per problem][t fp32 [T, r] per problem without t_save]
//   [X_d bf16 [T, k_in] per problem with dropout]
//   [projection partials][GEMM split-K partial tiles]
// Nothing in it needs clearing between calls: every byte a call reads was
// written earlier in the same call, except the GEMM's K-split arrival words,
// which each launch tags with a fresh 56-bit value (a word holding any other
// value counts as no arrivals).
struct FwdLayout {
  size_t zs[8], tscratch[8], xd[8], prj, gemm, total;
};

static void fwd_layout(const hsnf4_lora_fwd_args* p, int n, int64_t T, int r, FwdLayout* L) {
  const int rp = r_padded(r);
  size_t off = 0;
  for (int i = 0; i < n; ++i) {
    L->zs[i] = off;
    off += round_up(static_cast<size_t>(T) * rp * 2, 256);
  }
  for (int i = 0; i < n; ++i) {
    L->tscratch[i] = off;
    if (!p[i].t_save) off += round_up(static_cast<size_t>(T) * r * 4, 256);
  }
  for (int i = 0; i < n; ++i) {
    L->xd[i] = off;
    if (p[i].dropout_p > 0.0f) off += round_up(static_cast<size_t>(T) * p[i].W.k_in * 2, 256);
  }
  ProjectDesc pd[8];
  GemmProblemDesc gd[8];
  for (int i = 0; i < n; ++i) {
    // with dropout the projection reads this problem's own X_d: a distinct
    // input, as the launch will see it (only equality of inputs matters here)
    const void* z = p[i].dropout_p > 0.0f ? reinterpret_cast<const void*>(uintptr_t(16) * (i + 1))
                                          : p[i].X;
    pd[i] = {z, p[i].W.k_in, p[i].A, true, nullptr, nullptr};
    gd[i] = {p[i].W.codes, p[i].W.absmax, p[i].W.n_out, p[i].W.k_in, p[i].X, p[i].B, nullptr,
             p[i].Y, p[i].W.format == HSNF4_BASE_BF16};
  }
  L->prj = off;
  off += project_workspace_bytes(pd, n, T, r);
  L->gemm = off;
  off += gemm_workspace_bytes(kGemmFwd, gd, n, T, r);
  L->total = off;
}

// Workspace layout of a backward group:
//   [s*u bf16 [T, r_pad] per problem][u fp32 [T, r] per problem]
//   [u and t as two bf16 parts each, 4 x [T, r_pad] per problem: the
//    adapter-gradient operands]
//   [X_d bf16 [T, k_in] and its keep-mask bytes [T, k_in / 8] per problem
//    with dropout]
//   [projection partials][GEMM split-K partial tiles]
// As for the forward, nothing in it needs clearing between calls.
struct BwdLayout {
  size_t su[8], u[8], parts[8], xd[8], bits[8], prj, gemm, total;
};

static void bwd_layout(const hsnf4_lora_bwd_args* p, int n, int64_t T, int r, BwdLayout* L) {
  const int rp = r_padded(r);
  size_t off = 0;
  for (int i = 0; i < n; ++i) {
    L->su[i] = off;
    off += round_up(static_cast<size_t>(T) * rp * 2, 256);
  }
  for (int i = 0; i < n; ++i) {
    L->u[i] = off;
    off += round_up(static_cast<size_t>(T) * r * 4, 256);
  }
  for (int i = 0; i < n; ++i) {
    L->parts[i] = off;
    off += 4 * round_up(static_cast<size_t>(T) * rp * 2, 256);
  }
  for (int i = 0; i < n; ++i) {
    L->xd[i] = off;
    if (p[i].dropout_p > 0.0f) off += round_up(static_cast<size_t>(T) * p[i].W.k_in * 2, 256);
    L->bits[i] = off;
    if (p[i].dropout_p > 0.0f) off += round_up(static_cast<size_t>(T) * p[i].W.k_in / 8, 256);
  }
  ProjectDesc pd[8];
  GemmProblemDesc gd[8];
  for (int i = 0; i < n; ++i) {
    pd[i] = {p[i].dY, p[i].W.n_out, p[i].B, false, nullptr, nullptr};
    gd[i] = {p[i].W.codes, p[i].W.absmax, p[i].W.n_out, p[i].W.k_in, p[i].dY, p[i].A, nullptr,
             p[i].dX, p[i].W.format == HSNF4_BASE_BF16};
  }
  L->prj = off;
  off += project_workspace_bytes(pd, n, T, r);
  L->gemm = off;
  off += gemm_workspace_bytes(kGemmDx, gd, n, T, r);
  L->total = off;
}

size_t lora_group_fwd_workspace(const hsnf4_lora_fwd_args* probs, int n, int64_t T, int r) {
  if (!probs || n < 1 || n > 8 || T < 1 || r < 1) return 0;
  FwdLayout L;
  fwd_layout(probs, n, T, r, &L);
  return L.total;
}

int hsnf4_gemm_plan(int mode, const int64_t* n_out, const int64_t* k_in, int n, int64_t T,
                    int r, hsnf4_gemm_plan_info* out) {
  if (!n_out || !k_in || !out)
    return fail(HSNF4_ERR_INVALID, "hsnf4_gemm_plan: NULL argument");
  if (mode != 0 && mode != 1)
    return fail(HSNF4_ERR_INVALID, "hsnf4_gemm_plan: mode %d (0 forward, 1 dX)", mode);
  if (n < 1 || n > 8 || T < 1 || r < 1 || r > 64)
    return fail(HSNF4_ERR_INVALID, "hsnf4_gemm_plan: n=%d T=%lld r=%d", n, (long long)T, r);
  GemmProblemDesc d[8] = {};
  for (int i = 0; i < n; ++i) {
    if (n_out[i] < 64 || k_in[i] < 64 || n_out[i] % 64 || k_in[i] % 64)
      return fail(HSNF4_ERR_INVALID, "hsnf4_gemm_plan: problem %d: %lld x %lld", i,
                  (long long)n_out[i], (long long)k_in[i]);
    d[i].n_out = n_out[i];
    d[i].k_in = k_in[i];
  }
  const int rc = check_gemm_tokens(mode == 0 ? kGemmFwd : kGemmDx, T, r);
  if (rc) return rc;
  return gemm_plan_info(mode == 0 ? kGemmFwd : kGemmDx, d, n, T, r, out);
}

size_t lora_group_bwd_workspace(const hsnf4_lora_bwd_args* probs, int n, int64_t T, int r) {
  if (!probs || n < 1 || n > 8 || T < 1 || r < 1) return 0;
  BwdLayout L;
  bwd_layout(probs, n, T, r, &L);
  return L.total;
}

static int check_workspace(const char* fn, void* ws, size_t have, size_t need) {
  if (have < need)
    return fail(HSNF4_ERR_OOM, "%s: workspace too small: need %zu bytes, given %zu", fn, need,
                have);
  if (need && !ws) return fail(HSNF4_ERR_INVALID, "%s: workspace is NULL", fn);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(HSNF4_ERR_INVALID, "%s: workspace must be 256-byte aligned", fn);
  return HSNF4_OK;
}

int lora_group_fwd(const hsnf4_lora_fwd_args* probs, int n, int64_t T, int r, float alpha,
                   void* workspace, size_t ws_bytes, void* stream) {
  static const char* fn = "lora_group_fwd";
  if (!probs) return fail(HSNF4_ERR_INVALID, "%s: probs is NULL", fn);
  int rc = check_group(fn, n, T, r, alpha);
  if (!rc) rc = check_gemm_tokens(kGemmFwd, T, r);
  if (rc) return rc;
  for (int i = 0; i < n; ++i) {
    const hsnf4_lora_fwd_args& p = probs[i];
    rc = check_weight(fn, i, p.W);
    if (!rc) rc = check_ptrs(fn, {{p.X, "X"}, {p.A, "A"}, {p.B, "B"}, {p.Y, "Y"}});
    if (!rc && p.t_save && !aligned16(p.t_save))
      rc = fail(HSNF4_ERR_INVALID, "%s: problem %d: t_save misaligned", fn, i);
    if (!rc) rc = check_dropout(fn, i, p.dropout_p);
    if (rc) return rc;
  }
  {
    int32_t formats[8];
    for (int i = 0; i < n; ++i) formats[i] = probs[i].W.format;
    rc = check_one_format(fn, n, formats);
    if (rc) return rc;
  }
  FwdLayout L;
  fwd_layout(probs, n, T, r, &L);
  rc = check_workspace(fn, workspace, ws_bytes, L.total);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const float s = alpha / static_cast<float>(r);
  ProjectDesc pd[8];
  GemmProblemDesc gd[8];
  DropDesc dd[8];
  int nd = 0;
  for (int i = 0; i < n; ++i) {
    const hsnf4_lora_fwd_args& p = probs[i];
    float* t_out = p.t_save ? p.t_save : reinterpret_cast<float*>(ws + L.tscratch[i]);
    // with dropout the adapter branch reads X_d = dropout(X); the base reads X
    const void* xl = p.X;
    if (p.dropout_p > 0.0f) {
      xl = ws + L.xd[i];
      dd[nd++] = {p.X, ws + L.xd[i], nullptr, nullptr, p.W.k_in, p.dropout_p, p.dropout_seed,
                  p.dropout_offset};
    }
    pd[i] = {xl, p.W.k_in, p.A, true, t_out, ws + L.zs[i]};
    gd[i] = {p.W.codes, p.W.absmax, p.W.n_out, p.W.k_in, p.X, p.B, ws + L.zs[i], p.Y,
             p.W.format == HSNF4_BASE_BF16};
  }
  if (nd) {
    rc = cuda_status(launch_dropout_apply(dd, nd, T, st), "lora_group_fwd: dropout launch");
    if (rc) return rc;
  }
  rc = cuda_status(launch_lora_project_group(pd, n, T, r, s, ws + L.prj, st),
                   "lora_group_fwd: projection launch");
  if (rc) return rc;
  return launch_lora_gemm_group(kGemmFwd, gd, n, T, r, ws + L.gemm, L.total - L.gemm, st);
}

int lora_group_bwd(const hsnf4_lora_bwd_args* probs, int n, int64_t T, int r, float alpha,
                   void* workspace, size_t ws_bytes, void* stream) {
  static const char* fn = "lora_group_bwd";
  if (!probs) return fail(HSNF4_ERR_INVALID, "%s: probs is NULL", fn);
  int rc = check_group(fn, n, T, r, alpha);
  if (!rc) rc = check_gemm_tokens(kGemmDx, T, r);
  if (rc) return rc;
  for (int i = 0; i < n; ++i) {
    const hsnf4_lora_bwd_args& p = probs[i];
    rc = check_weight(fn, i, p.W);
    if (!rc)
      rc = check_ptrs(fn, {{p.X, "X"}, {p.t_save, "t_save"}, {p.A, "A"}, {p.B, "B"},
                           {p.dY, "dY"}, {p.dX, "dX"}, {p.dA, "dA"}, {p.dB, "dB"}});
    if (!rc) rc = check_dropout(fn, i, p.dropout_p);
    if (rc) return rc;
  }
  {
    int32_t formats[8];
    for (int i = 0; i < n; ++i) formats[i] = probs[i].W.format;
    rc = check_one_format(fn, n, formats);
    if (rc) return rc;
  }
  BwdLayout L;
  bwd_layout(probs, n, T, r, &L);
  rc = check_workspace(fn, workspace, ws_bytes, L.total);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const float s = alpha / static_cast<float>(r);
  ProjectDesc pd[8];
  GemmProblemDesc gd[8];
  GradDesc grd[16];
  DropDesc dd[8], da[8];
  int nd = 0;
  for (int i = 0; i < n; ++i) {
    const hsnf4_lora_bwd_args& p = probs[i];
    float* u = reinterpret_cast<float*>(ws + L.u[i]);
    const bool drop = p.dropout_p > 0.0f;
    // with dropout: X_d recomputed from the forward's (seed, offset) feeds
    // dA; the GEMM's rank-r slice is zero and the masked adapter term of dX
    // is added after it
    const void* xl = drop ? static_cast<const void*>(ws + L.xd[i]) : p.X;
    if (drop) {
      // the apply pass records the keep mask; the dX pass reads it back
      dd[nd] = {p.X, ws + L.xd[i], nullptr, nullptr, p.W.k_in, p.dropout_p, p.dropout_seed,
                p.dropout_offset, ws + L.bits[i]};
      da[nd] = {nullptr, p.dX, u, p.A, p.W.k_in, p.dropout_p, p.dropout_seed, p.dropout_offset,
                ws + L.bits[i]};
      ++nd;
    }
    // u and the forward's t as two bf16 parts each: the gradient kernel's operands
    const size_t part = round_up(static_cast<size_t>(T) * r_padded(r) * 2, 256);
    uint8_t* u_hi = ws + L.parts[i];
    uint8_t* u_lo = u_hi + part;
    uint8_t* t_hi = u_lo + part;
    uint8_t* t_lo = t_hi + part;
    pd[i] = {p.dY, p.W.n_out, p.B, false, u, ws + L.su[i], drop, u_hi, u_lo, p.t_save, t_hi,
             t_lo};
    gd[i] = {p.W.codes, p.W.absmax, p.W.n_out, p.W.k_in, p.dY, p.A, ws + L.su[i], p.dX,
             p.W.format == HSNF4_BASE_BF16};
    grd[2 * i] = {p.dY, p.W.n_out, t_hi, t_lo, p.dB, true};  // dB = s dY^T t    [n_out, r]
    grd[2 * i + 1] = {xl, p.W.k_in, u_hi, u_lo, p.dA, false};  // dA = s u^T X(_d) [r, k_in]
  }
  if (nd) {
    rc = cuda_status(launch_dropout_apply(dd, nd, T, st), "lora_group_bwd: dropout launch");
    if (rc) return rc;
  }
  rc = cuda_status(launch_lora_project_group(pd, n, T, r, s, ws + L.prj, st),
                   "lora_group_bwd: projection launch");
  if (rc) return rc;
  // The adapter gradients need only u, t, X and dY: they run before the dX
  // GEMM, while the dY the projection has just read (and X) are still in L2,
  // instead of after the GEMM has streamed the base through it.
  rc = cuda_status(launch_lora_grad_group(grd, 2 * n, T, r, s, st),
                   "lora_group_bwd: gradient launch");
  if (rc) return rc;
  rc = launch_lora_gemm_group(kGemmDx, gd, n, T, r, ws + L.gemm, L.total - L.gemm, st);
  if (rc) return rc;
  if (nd)
    rc = cuda_status(launch_dx_dropout_add(da, nd, T, r, s, st),
                     "lora_group_bwd: dropout dX launch");
  return rc;
}

int lora_merge(const hsnf4_nf4_weight* W, const void* A, const void* B, int r, float alpha,
               void* W_out, void* stream) {
  static const char* fn = "lora_merge";
  if (!W) return fail(HSNF4_ERR_INVALID, "%s: W is NULL", fn);
  int rc = check_weight(fn, 0, *W);
  if (rc) return rc;
  if (r < 8 || r > 64 || r % 8)
    return fail(HSNF4_ERR_INVALID, "%s: rank must be a multiple of 8 in [8, 64] (got %d)", fn, r);
  if (!isfinite(alpha)) return fail(HSNF4_ERR_INVALID, "%s: alpha is not finite", fn);
  rc = check_ptrs(fn, {{A, "A"}, {B, "B"}, {W_out, "W_out"}});
  if (rc) return rc;
  if (W_out == W->codes) return fail(HSNF4_ERR_INVALID, "%s: W_out aliases the base", fn);
  return cuda_status(launch_lora_merge(W->codes, W->absmax, W->format == HSNF4_BASE_BF16,
                                       W->n_out, W->k_in, A, B, r,
                                       alpha / static_cast<float>(r), W_out,
                                       static_cast<cudaStream_t>(stream)),
                     "lora_merge launch");
}

int lora_dropout_apply(const void* X, int64_t T, int64_t k_in, float p, uint64_t seed,
                       uint64_t offset, void* X_d, void* stream) {
  static const char* fn = "lora_dropout_apply";
  int rc = check_nf4_shape(fn, T, k_in);
  if (!rc) rc = check_dropout(fn, 0, p);
  if (!rc) rc = check_ptrs(fn, {{X, "X"}, {X_d, "X_d"}});
  if (rc) return rc;
  DropDesc d = {X, X_d, nullptr, nullptr, k_in, p, seed, offset};
  return cuda_status(launch_dropout_apply(&d, 1, T, static_cast<cudaStream_t>(stream)),
                     "lora_dropout_apply launch");
}

// ---------------------------------------------------------------- decoder glue

static int check_rows(const char* fn, int64_t T, int64_t n) {
  if (T < 1 || n < 8 || n % 8 || T > (int64_t(1) << 31) || n > (int64_t(1) << 30))
    return fail(HSNF4_ERR_INVALID, "%s: need T >= 1 and n a positive multiple of 8 (got T=%lld, "
                "n=%lld)", fn, (long long)T, (long long)n);
  return HSNF4_OK;
}

static int check_elems(const char* fn, int64_t n) {
  if (n < 8 || n % 8)
    return fail(HSNF4_ERR_INVALID, "%s: need a positive multiple of 8 elements (got %lld)", fn,
                (long long)n);
  return HSNF4_OK;
}

static int check_opt(const char* fn, const void* p, const char* name) {
  if (p && !aligned16(p)) return fail(HSNF4_ERR_INVALID, "%s: %s is not 16-byte aligned", fn, name);
  return HSNF4_OK;
}

int decoder_rmsnorm_fwd(const void* xa, const void* xb, const void* g, void* h_out, void* y,
                        int64_t T, int64_t n, float eps, void* stream) {
  static const char* fn = "decoder_rmsnorm_fwd";
  int rc = check_rows(fn, T, n);
  if (!rc) rc = check_ptrs(fn, {{xa, "xa"}, {g, "g"}, {y, "y"}});
  if (!rc) rc = check_opt(fn, xb, "xb");
  if (!rc && xb) rc = check_ptrs(fn, {{h_out, "h_out"}});
  if (!rc && !(eps >= 0.0f)) rc = fail(HSNF4_ERR_INVALID, "%s: eps must be >= 0", fn);
  if (rc) return rc;
  return cuda_status(launch_rmsnorm_fwd(xa, xb, g, h_out, y, T, n, eps,
                                        static_cast<cudaStream_t>(stream)),
                     "decoder_rmsnorm_fwd launch");
}

int decoder_rmsnorm_bwd(const void* x, const void* g, const void* dy1, const void* dy2,
                        const void* dy3, const void* dres, void* dx, int64_t T, int64_t n,
                        float eps, void* stream) {
  static const char* fn = "decoder_rmsnorm_bwd";
  int rc = check_rows(fn, T, n);
  if (!rc) rc = check_ptrs(fn, {{x, "x"}, {g, "g"}, {dy1, "dy1"}, {dx, "dx"}});
  if (!rc) rc = check_opt(fn, dy2, "dy2");
  if (!rc) rc = check_opt(fn, dy3, "dy3");
  if (!rc) rc = check_opt(fn, dres, "dres");
  if (!rc && !(eps >= 0.0f)) rc = fail(HSNF4_ERR_INVALID, "%s: eps must be >= 0", fn);
  if (rc) return rc;
  return cuda_status(launch_rmsnorm_bwd(x, g, dy1, dy2, dy3, dres, dx, T, n, eps,
                                        static_cast<cudaStream_t>(stream)),
                     "decoder_rmsnorm_bwd launch");
}

int decoder_swiglu_fwd(const void* a, const void* b, void* m, int64_t n, void* stream) {
  static const char* fn = "decoder_swiglu_fwd";
  int rc = check_elems(fn, n);
  if (!rc) rc = check_ptrs(fn, {{a, "a"}, {b, "b"}, {m, "m"}});
  if (rc) return rc;
  return cuda_status(launch_silu_mul_fwd(a, b, m, n, static_cast<cudaStream_t>(stream)),
                     "decoder_swiglu_fwd launch");
}

int decoder_swiglu_bwd(const void* a, const void* b, const void* dm, void* da, void* db, int64_t n,
                       void* stream) {
  static const char* fn = "decoder_swiglu_bwd";
  int rc = check_elems(fn, n);
  if (!rc) rc = check_ptrs(fn, {{a, "a"}, {b, "b"}, {dm, "dm"}, {da, "da"}, {db, "db"}});
  if (rc) return rc;
  return cuda_status(launch_silu_mul_bwd(a, b, dm, da, db, n, static_cast<cudaStream_t>(stream)),
                     "decoder_swiglu_bwd launch");
}

int decoder_add(const void* x, const void* y, void* out, int64_t n, void* stream) {
  static const char* fn = "decoder_add";
  int rc = check_elems(fn, n);
  if (!rc) rc = check_ptrs(fn, {{x, "x"}, {y, "y"}, {out, "out"}});
  if (rc) return rc;
  return cuda_status(launch_add(x, y, out, n, static_cast<cudaStream_t>(stream)),
                     "decoder_add launch");
}

static int check_attn(const char* fn, int64_t T, int H, int KV) {
  if (T < 1 || T > 32768 || H < 1 || KV < 1 || H % KV)
    return fail(HSNF4_ERR_INVALID, "%s: need 1 <= T <= 32768 and H a multiple of KV (got T=%lld, "
                "H=%d, KV=%d)", fn, (long long)T, H, KV);
  return HSNF4_OK;
}

int decoder_attention_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                          int64_t T, int H, int KV, void* stream) {
  static const char* fn = "decoder_attention_fwd";
  int rc = check_attn(fn, T, H, KV);
  if (!rc) rc = check_ptrs(fn, {{q, "q"}, {k, "k"}, {v, "v"}, {o, "o"}, {lse, "lse"}});
  if (rc) return rc;
  return cuda_status(launch_attention_fwd(q, k, v, o, lse, T, H, KV, 1.0f / sqrtf(128.0f),
                                          static_cast<cudaStream_t>(stream)),
                     "decoder_attention_fwd launch");
}

size_t decoder_attention_scratch_bytes(int64_t T, int H) {
  if (T < 1 || H < 1) return 0;
  // row dots [H, T] (rounded up to 64 floats), then fp32 dK, dV partials [2H][T][128]
  return (static_cast<size_t>(T) * H + 63) / 64 * 64 * 4 + static_cast<size_t>(T) * H * 2 * 128 * 4;
}

int decoder_attention_bwd(const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* dout, void* dq, void* dk, void* dv,
                          float* scratch, int64_t T, int H, int KV, void* stream) {
  static const char* fn = "decoder_attention_bwd";
  int rc = check_attn(fn, T, H, KV);
  if (!rc)
    rc = check_ptrs(fn, {{q, "q"}, {k, "k"}, {v, "v"}, {o, "o"}, {lse, "lse"}, {dout, "dout"},
                         {dq, "dq"}, {dk, "dk"}, {dv, "dv"}, {scratch, "scratch"}});
  if (rc) return rc;
  return cuda_status(launch_attention_bwd(q, k, v, o, lse, dout, dq, dk, dv, scratch, T, H, KV,
                                          1.0f / sqrtf(128.0f), static_cast<cudaStream_t>(stream)),
                     "decoder_attention_bwd launch");
}

// ---------------------------------------------------------------- rotary positions

// A strided matrix of bf16 rows: `rows` rows of `width` elements, `stride`
// elements apart.
struct Rows {
  const void* p;
  int64_t stride, width, rows;
  const char* name;
};

// Whether two of them share a byte.  Rows of one stride may interleave (the
// columns of a fused tensor); of different strides, meeting byte ranges count
// as shared.
static bool rows_meet(const Rows& a, const Rows& b) {
  if (!a.rows || !b.rows || !a.width || !b.width) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + 2 * static_cast<uintptr_t>((a.rows - 1) * a.stride + a.width);
  const uintptr_t eb = pb + 2 * static_cast<uintptr_t>((b.rows - 1) * b.stride + b.width);
  if (ea <= pb || eb <= pa) return false;
  if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
  const uintptr_t pitch = 2 * static_cast<uintptr_t>(a.stride);
  const uintptr_t off = pa >= pb ? (pa - pb) % pitch : (pitch - (pb - pa) % pitch) % pitch;
  return off < 2 * static_cast<uintptr_t>(b.width) ||
         off + 2 * static_cast<uintptr_t>(a.width) > pitch;
}

static int check_disjoint(const char* fn, const Rows& out, std::initializer_list<Rows> others) {
  for (const Rows& r : others)
    if (rows_meet(out, r))
      return fail(HSNF4_ERR_INVALID, "%s: %s overlaps %s", fn, out.name, r.name);
  return HSNF4_OK;
}

// *stride (0: the row itself) of rows of `width` elements
static int check_stride(const char* fn, const char* name, int64_t* stride, int64_t width) {
  if (*stride == 0) *stride = width;
  if (*stride < width || *stride % 8 || *stride > (int64_t(1) << 30))
    return fail(HSNF4_ERR_INVALID,
                "%s: %s must be a multiple of 8, at least the row of %lld elements and at most "
                "2^30 (got %lld)", fn, name, (long long)width, (long long)*stride);
  return HSNF4_OK;
}

static int rope_call(const char* fn, bool backward, const hsnf4_rope* R, const int32_t* pos,
                     int64_t T, int H, int KV, const void* q, int64_t qs, const void* k,
                     int64_t ks, void* qo, int64_t qos, void* ko, int64_t kos, void* stream) {
  if (!R) return fail(HSNF4_ERR_INVALID, "%s: rope is NULL", fn);
  if (R->head_dim < 16 || R->head_dim > 256 || R->head_dim % 8 || R->rot_dim < 16 ||
      R->rot_dim > R->head_dim || R->rot_dim % 16)
    return fail(HSNF4_ERR_INVALID, "%s: need head_dim a multiple of 8 in [16, 256] and rot_dim a "
                "multiple of 16 in [16, head_dim] (got %d, %d)", fn, R->head_dim, R->rot_dim);
  if (R->n_axes < 1 || R->n_axes > 8)
    return fail(HSNF4_ERR_INVALID, "%s: n_axes must be in [1, 8] (got %d)", fn, R->n_axes);
  if (R->pairing != HSNF4_ROPE_HALF && R->pairing != HSNF4_ROPE_ADJACENT)
    return fail(HSNF4_ERR_INVALID, "%s: unknown pairing %d", fn, R->pairing);
  if (!isfinite(R->scale)) return fail(HSNF4_ERR_INVALID, "%s: scale is not finite", fn);
  for (int i = 0; i < R->rot_dim / 2; ++i) {
    if (!isfinite(R->inv_freq[i]))
      return fail(HSNF4_ERR_INVALID, "%s: inv_freq[%d] is not finite", fn, i);
    if (R->axis[i] >= R->n_axes)
      return fail(HSNF4_ERR_INVALID, "%s: axis[%d] = %d of %d axes", fn, i, R->axis[i], R->n_axes);
  }
  if (T < 1 || T > (int64_t(1) << 30) || H < 1 || KV < 0 || H > 1024 || KV > 1024)
    return fail(HSNF4_ERR_INVALID, "%s: need 1 <= T <= 2^30, 1 <= H <= 1024 and 0 <= KV <= 1024 "
                "(got T=%lld, H=%d, KV=%d)", fn, (long long)T, H, KV);
  int rc = check_ptrs(fn, {{q, backward ? "dq" : "q"}, {qo, backward ? "dq_out" : "q_out"}});
  if (!rc && KV) rc = check_ptrs(fn, {{k, backward ? "dk" : "k"}, {ko, backward ? "dk_out" : "k_out"}});
  if (!rc && !pos) rc = fail(HSNF4_ERR_INVALID, "%s: pos is NULL", fn);
  if (!rc && (reinterpret_cast<uintptr_t>(pos) & 3))
    rc = fail(HSNF4_ERR_INVALID, "%s: pos is not 4-byte aligned", fn);
  if (!rc && !KV && (k || ko)) rc = fail(HSNF4_ERR_INVALID, "%s: k given with KV = 0", fn);
  const int64_t wq = static_cast<int64_t>(H) * R->head_dim,
                wk = static_cast<int64_t>(KV) * R->head_dim;
  if (!rc) rc = check_stride(fn, backward ? "dq_stride" : "q_stride", &qs, wq);
  if (!rc) rc = check_stride(fn, backward ? "dq_out_stride" : "q_out_stride", &qos, wq);
  if (!rc && KV) rc = check_stride(fn, backward ? "dk_stride" : "k_stride", &ks, wk);
  if (!rc && KV) rc = check_stride(fn, backward ? "dk_out_stride" : "k_out_stride", &kos, wk);
  if (rc) return rc;
  const Rows rq = {q, qs, wq, T, backward ? "dq" : "q"};
  const Rows rk = {k, ks, wk, KV ? T : 0, backward ? "dk" : "k"};
  const Rows rqo = {qo, qos, wq, T, backward ? "dq_out" : "q_out"};
  const Rows rko = {ko, kos, wk, KV ? T : 0, backward ? "dk_out" : "k_out"};
  // pos as one row of 16-bit words
  const Rows rp = {pos, 0, 2 * R->n_axes * T, 1, "pos"};
  const bool q_in_place = q == qo && qs == qos, k_in_place = k == ko && ks == kos;
  if (!q_in_place) rc = check_disjoint(fn, rqo, {rq});
  if (!rc) rc = check_disjoint(fn, rqo, {rk, rko, rp});
  if (!rc && !k_in_place) rc = check_disjoint(fn, rko, {rk});
  if (!rc) rc = check_disjoint(fn, rko, {rq, rp});
  if (rc) return rc;
  const RopeTensors t = {{q, k}, {qo, ko}, {qs, ks}, {qos, kos}, pos};
  return cuda_status(launch_rope(*R, t, T, H, KV, backward, static_cast<cudaStream_t>(stream)),
                     backward ? "decoder_rope_bwd launch" : "decoder_rope_fwd launch");
}

int decoder_rope_fwd(const hsnf4_rope* rope, const int32_t* pos, int64_t T, int H, int KV,
                     const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                     void* stream) {
  return rope_call("decoder_rope_fwd", false, rope, pos, T, H, KV, q, q_stride, k, k_stride,
                   q_out, q_out_stride, k_out, k_out_stride, stream);
}

int decoder_rope_bwd(const hsnf4_rope* rope, const int32_t* pos, int64_t T, int H, int KV,
                     const void* dq, int64_t dq_stride, const void* dk, int64_t dk_stride,
                     void* dq_out, int64_t dq_out_stride, void* dk_out, int64_t dk_out_stride,
                     void* stream) {
  return rope_call("decoder_rope_bwd", true, rope, pos, T, H, KV, dq, dq_stride, dk, dk_stride,
                   dq_out, dq_out_stride, dk_out, dk_out_stride, stream);
}

// ---------------------------------------------------------------- packed attention

static int check_packed_sizes(const char* fn, int64_t Tq, int64_t Tk, int n_seq, int H, int KV,
                              int d) {
  const int64_t most = int64_t(1) << 24;
  if (Tq < 1 || Tk < 1 || Tq > most || Tk > most || n_seq < 1 || n_seq > 65535 || H < 1 ||
      H > 1024 || KV < 1 || H % KV)
    return fail(HSNF4_ERR_INVALID, "%s: need 1 <= Tq, Tk <= 2^24, 1 <= n_seq <= 65535 and H <= "
                "1024 a multiple of KV (got Tq=%lld, Tk=%lld, n_seq=%d, H=%d, KV=%d)", fn,
                (long long)Tq, (long long)Tk, n_seq, H, KV);
  if (d != 64 && d != 128)
    return fail(HSNF4_ERR_INVALID, "%s: head_dim must be 64 or 128 (got %d)", fn, d);
  return HSNF4_OK;
}

// checks *a and fills its zero strides
static int check_packed(const char* fn, hsnf4_packed_attention* a) {
  int rc = check_packed_sizes(fn, a->Tq, a->Tk, a->n_seq, a->H, a->KV, a->head_dim);
  if (!rc) rc = check_ptrs(fn, {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}});
  if (rc) return rc;
  const std::pair<const int32_t*, const char*> cus[] = {{a->cu_q, "cu_q"}, {a->cu_k, "cu_k"}};
  for (auto& c : cus) {
    if (!c.first) return fail(HSNF4_ERR_INVALID, "%s: %s is NULL", fn, c.second);
    if (reinterpret_cast<uintptr_t>(c.first) & 3)
      return fail(HSNF4_ERR_INVALID, "%s: %s is not 4-byte aligned", fn, c.second);
  }
  if (a->causal != 0 && a->causal != 1)
    return fail(HSNF4_ERR_INVALID, "%s: causal must be 0 or 1 (got %d)", fn, a->causal);
  if (!(isfinite(a->scale) && a->scale > 0.0f))
    return fail(HSNF4_ERR_INVALID, "%s: scale must be finite and > 0 (got %g)", fn,
                static_cast<double>(a->scale));
  const int64_t wq = static_cast<int64_t>(a->H) * a->head_dim,
                wk = static_cast<int64_t>(a->KV) * a->head_dim;
  rc = check_stride(fn, "q_stride", &a->q_stride, wq);
  if (!rc) rc = check_stride(fn, "k_stride", &a->k_stride, wk);
  if (!rc) rc = check_stride(fn, "v_stride", &a->v_stride, wk);
  return rc;
}

// the cumulative lengths, as one row of 16-bit words
static Rows cu_rows(const hsnf4_packed_attention& a, const int32_t* cu, const char* name) {
  return {cu, 0, 2 * (static_cast<int64_t>(a.n_seq) + 1), 1, name};
}

int decoder_attention_packed_fwd(const hsnf4_packed_attention* args, void* o, int64_t o_stride,
                                 float* lse, void* stream) {
  static const char* fn = "decoder_attention_packed_fwd";
  if (!args) return fail(HSNF4_ERR_INVALID, "%s: a is NULL", fn);
  hsnf4_packed_attention a = *args;
  int rc = check_packed(fn, &a);
  if (!rc) rc = check_ptrs(fn, {{o, "o"}, {lse, "lse"}});
  const int64_t wq = static_cast<int64_t>(a.H) * a.head_dim,
                wk = static_cast<int64_t>(a.KV) * a.head_dim;
  if (!rc) rc = check_stride(fn, "o_stride", &o_stride, wq);
  if (rc) return rc;
  const Rows q = {a.q, a.q_stride, wq, a.Tq, "q"}, k = {a.k, a.k_stride, wk, a.Tk, "k"},
             v = {a.v, a.v_stride, wk, a.Tk, "v"}, ro = {o, o_stride, wq, a.Tq, "o"},
             rl = {lse, 0, 2 * a.H * a.Tq, 1, "lse"}, cq = cu_rows(a, a.cu_q, "cu_q"),
             ck = cu_rows(a, a.cu_k, "cu_k");
  rc = check_disjoint(fn, ro, {q, k, v, rl, cq, ck});
  if (!rc) rc = check_disjoint(fn, rl, {q, k, v, cq, ck});
  if (rc) return rc;
  return cuda_status(launch_packed_fwd(a, o, o_stride, lse, static_cast<cudaStream_t>(stream)),
                     "decoder_attention_packed_fwd launch");
}

size_t decoder_attention_packed_workspace(int64_t Tq, int64_t Tk, int n_seq, int H, int KV,
                                          int head_dim) {
  if (check_packed_sizes("decoder_attention_packed_workspace", Tq, Tk, n_seq, H, KV, head_dim))
    return 0;
  return packed_workspace_bytes(Tq, Tk, n_seq, H, KV, head_dim);
}

int decoder_attention_packed_bwd(const hsnf4_packed_attention* args, const void* o,
                                 int64_t o_stride, const float* lse, const void* dout,
                                 int64_t dout_stride, void* dq, int64_t dq_stride, void* dk,
                                 int64_t dk_stride, void* dv, int64_t dv_stride, void* workspace,
                                 size_t ws_bytes, void* stream) {
  static const char* fn = "decoder_attention_packed_bwd";
  if (!args) return fail(HSNF4_ERR_INVALID, "%s: a is NULL", fn);
  hsnf4_packed_attention a = *args;
  int rc = check_packed(fn, &a);
  if (!rc)
    rc = check_ptrs(fn, {{o, "o"}, {lse, "lse"}, {dout, "dout"}, {dq, "dq"}, {dk, "dk"},
                         {dv, "dv"}});
  const int64_t wq = static_cast<int64_t>(a.H) * a.head_dim,
                wk = static_cast<int64_t>(a.KV) * a.head_dim;
  if (!rc) rc = check_stride(fn, "o_stride", &o_stride, wq);
  if (!rc) rc = check_stride(fn, "dout_stride", &dout_stride, wq);
  if (!rc) rc = check_stride(fn, "dq_stride", &dq_stride, wq);
  if (!rc) rc = check_stride(fn, "dk_stride", &dk_stride, wk);
  if (!rc) rc = check_stride(fn, "dv_stride", &dv_stride, wk);
  if (rc) return rc;
  const size_t need = packed_workspace_bytes(a.Tq, a.Tk, a.n_seq, a.H, a.KV, a.head_dim);
  rc = check_workspace(fn, workspace, ws_bytes, need);
  if (rc) return rc;
  const Rows in[] = {{a.q, a.q_stride, wq, a.Tq, "q"},
                     {a.k, a.k_stride, wk, a.Tk, "k"},
                     {a.v, a.v_stride, wk, a.Tk, "v"},
                     {o, o_stride, wq, a.Tq, "o"},
                     {dout, dout_stride, wq, a.Tq, "dout"},
                     {lse, 0, 2 * a.H * a.Tq, 1, "lse"},
                     cu_rows(a, a.cu_q, "cu_q"),
                     cu_rows(a, a.cu_k, "cu_k"),
                     {workspace, 0, static_cast<int64_t>(need / 2), 1, "workspace"}};
  constexpr int kIn = sizeof in / sizeof in[0];  // the last of them is written too
  const Rows out[] = {{dq, dq_stride, wq, a.Tq, "dq"},
                      {dk, dk_stride, wk, a.Tk, "dk"},
                      {dv, dv_stride, wk, a.Tk, "dv"}};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if ((rc = check_disjoint(fn, out[i], {r}))) return rc;
    for (int j = 0; j < i; ++j)
      if ((rc = check_disjoint(fn, out[i], {out[j]}))) return rc;
  }
  for (int j = 0; j + 1 < kIn; ++j)
    if ((rc = check_disjoint(fn, in[kIn - 1], {in[j]}))) return rc;
  const PackedBwd b = {o, lse, dout, dq, dk, dv, o_stride, dout_stride, dq_stride, dk_stride,
                       dv_stride};
  return cuda_status(launch_packed_bwd(a, b, workspace, static_cast<cudaStream_t>(stream)),
                     "decoder_attention_packed_bwd launch");
}

// ---------------------------------------------------------------- gradient norm

size_t lora_grad_table_bytes(int n) { return n < 1 || n > 65536 ? 0 : grad_table_bytes(n); }

int lora_grad_plan(const hsnf4_grad* grads, int n, void* table, size_t table_bytes,
                   hsnf4_grad_plan* plan, void* stream) {
  static const char* fn = "lora_grad_plan";
  if (!grads || !plan) return fail(HSNF4_ERR_INVALID, "%s: %s is NULL", fn, grads ? "plan" : "grads");
  if (n < 1 || n > 65536)
    return fail(HSNF4_ERR_INVALID, "%s: 1..65536 tensors (got %d)", fn, n);
  int rc = check_ptrs(fn, {{table, "table"}});
  if (rc) return rc;
  if (table_bytes < grad_table_bytes(n))
    return fail(HSNF4_ERR_OOM, "%s: table too small: need %zu bytes, given %zu", fn,
                grad_table_bytes(n), table_bytes);
  // byte ranges: every out against every other range, but its own g in place
  struct Range {
    uintptr_t a, b;
    int i;
    bool out;
  };
  std::unique_ptr<Range[]> r(new (std::nothrow) Range[2 * static_cast<size_t>(n)]);
  if (!r) return fail(HSNF4_ERR_OOM, "%s: no host memory", fn);
  int m = 0;
  int64_t elements = 0;
  for (int i = 0; i < n; ++i) {
    const hsnf4_grad& g = grads[i];
    if (g.dtype != HSNF4_F32 && g.dtype != HSNF4_BF16 && g.dtype != HSNF4_F16)
      return fail(HSNF4_ERR_INVALID, "%s: tensor %d has unknown type %d", fn, i, g.dtype);
    if (g.n < 0 || g.n > (int64_t(1) << 40))
      return fail(HSNF4_ERR_INVALID, "%s: tensor %d has %lld elements", fn, i, (long long)g.n);
    if (!g.n) continue;
    const uintptr_t size = g.dtype == HSNF4_F32 ? 4 : 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g.g), o = reinterpret_cast<uintptr_t>(g.out);
    if (!a || !o || a % size || o % size)
      return fail(HSNF4_ERR_INVALID, "%s: tensor %d is NULL or not aligned to its element", fn, i);
    elements += g.n;
    r[m++] = {a, a + size * static_cast<uintptr_t>(g.n), i, a == o};
    if (a != o) r[m++] = {o, o + size * static_cast<uintptr_t>(g.n), i, true};
  }
  // the table is written now, and later calls trust its addresses
  const uintptr_t ta = reinterpret_cast<uintptr_t>(table), tb = ta + grad_table_bytes(n);
  for (int j = 0; j < m; ++j)
    if (r[j].a < tb && ta < r[j].b)
      return fail(HSNF4_ERR_INVALID, "%s: the table overlaps tensor %d", fn, r[j].i);
  // in order of their starts, a range that is written meets another exactly
  // when it meets the furthest-reaching range before it, or the furthest
  // written one does
  std::sort(r.get(), r.get() + m, [](const Range& x, const Range& y) {
    return x.a != y.a ? x.a < y.a : x.i < y.i;
  });
  int far = -1, far_out = -1;  // furthest end so far, of any range and of a written one
  for (int j = 0; j < m; ++j) {
    const int hit = r[j].out ? far : far_out;
    if (hit >= 0 && r[hit].b > r[j].a)
      return fail(HSNF4_ERR_INVALID, "%s: tensors %d and %d overlap where one is written", fn,
                  r[hit].i, r[j].i);
    if (far < 0 || r[j].b > r[far].b) far = j;
    if (r[j].out && (far_out < 0 || r[j].b > r[far_out].b)) far_out = j;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  rc = cuda_status(cudaStreamIsCapturing(st, &cap), "lora_grad_plan: cudaStreamIsCapturing");
  if (rc) return rc;
  if (cap != cudaStreamCaptureStatusNone)
    return fail(HSNF4_ERR_STATE, "%s: the table cannot be filled during stream capture", fn);
  int64_t chunks = 0;
  rc = cuda_status(fill_grad_table(grads, n, table, &chunks, st), "lora_grad_plan: table copy");
  if (rc) return rc;
  *plan = {table, chunks, elements, n, 0};
  return HSNF4_OK;
}

size_t lora_grad_workspace(const hsnf4_grad_plan* plan) {
  return plan ? grad_workspace_bytes(plan->chunks) : 0;
}

static int grad_call(const char* fn, const hsnf4_grad_plan* plan, float max_norm, bool scale,
                     float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (!plan || !plan->table || plan->n < 1 || plan->chunks < 0)
    return fail(HSNF4_ERR_INVALID, "%s: plan is NULL or was not filled by lora_grad_plan", fn);
  if (!(max_norm >= 0.0f))
    return fail(HSNF4_ERR_INVALID, "%s: max_norm must be >= 0 (got %g)", fn,
                static_cast<double>(max_norm));
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3))
    return fail(HSNF4_ERR_INVALID, "%s: norm is NULL or not 4-byte aligned", fn);
  const size_t need = grad_workspace_bytes(plan->chunks);
  int rc = check_workspace(fn, ws, ws_bytes, need);
  if (rc) return rc;
  const int64_t table_bytes = static_cast<int64_t>(grad_table_bytes(plan->n));
  const Rows rw = {ws, 0, static_cast<int64_t>(need / 2), 1, "workspace"}, rn = {norm, 0, 2, 1, "norm"},
             rt = {plan->table, 0, table_bytes / 2, 1, "the plan's table"};
  rc = check_disjoint(fn, rw, {rt, rn});
  if (!rc) rc = check_disjoint(fn, rn, {rt});
  if (rc) return rc;
  return cuda_status(launch_grad_norm(plan->table, plan->n, plan->chunks, max_norm, scale, norm,
                                      ws, static_cast<cudaStream_t>(stream)),
                     scale ? "lora_grad_clip launch" : "lora_grad_norm launch");
}

int lora_grad_norm(const hsnf4_grad_plan* plan, float* norm, void* workspace, size_t ws_bytes,
                   void* stream) {
  return grad_call("lora_grad_norm", plan, 0.0f, false, norm, workspace, ws_bytes, stream);
}

int lora_grad_clip(const hsnf4_grad_plan* plan, float max_norm, float* norm, void* workspace,
                   size_t ws_bytes, void* stream) {
  return grad_call("lora_grad_clip", plan, max_norm, true, norm, workspace, ws_bytes, stream);
}

static hsnf4_lora_fwd_args one_fwd(const hsnf4_nf4_weight* W, const void* X, const void* A,
                                   const void* B, void* Y, float* t_save) {
  hsnf4_lora_fwd_args a;
  memset(&a, 0, sizeof a);  // no dropout
  a.W = *W;
  a.X = X;
  a.A = A;
  a.B = B;
  a.Y = Y;
  a.t_save = t_save;
  return a;
}

size_t lora_linear_fwd_workspace(int64_t T, int64_t n_out, int64_t k_in, int r) {
  hsnf4_nf4_weight W = {nullptr, nullptr, n_out, k_in, HSNF4_BASE_NF4, 0};
  hsnf4_lora_fwd_args a = one_fwd(&W, nullptr, nullptr, nullptr, nullptr, nullptr);
  return lora_group_fwd_workspace(&a, 1, T, r);
}

size_t lora_linear_bwd_workspace(int64_t T, int64_t n_out, int64_t k_in, int r) {
  hsnf4_lora_bwd_args a;
  memset(&a, 0, sizeof a);
  a.W.n_out = n_out;
  a.W.k_in = k_in;
  return lora_group_bwd_workspace(&a, 1, T, r);
}

int lora_linear_fwd(const hsnf4_nf4_weight* W, const void* X, int64_t T, const void* A,
                    const void* B, int r, float alpha, void* Y, float* t_save, void* workspace,
                    size_t ws_bytes, void* stream) {
  if (!W) return fail(HSNF4_ERR_INVALID, "lora_linear_fwd: W is NULL");
  hsnf4_lora_fwd_args a = one_fwd(W, X, A, B, Y, t_save);
  return lora_group_fwd(&a, 1, T, r, alpha, workspace, ws_bytes, stream);
}

int lora_linear_bwd(const hsnf4_nf4_weight* W, const void* X, const float* t_save, int64_t T,
                    const void* A, const void* B, int r, float alpha, const void* dY, void* dX,
                    float* dA, float* dB, void* workspace, size_t ws_bytes, void* stream) {
  if (!W) return fail(HSNF4_ERR_INVALID, "lora_linear_bwd: W is NULL");
  hsnf4_lora_bwd_args a;
  memset(&a, 0, sizeof a);  // no dropout
  a.W = *W;
  a.X = X;
  a.t_save = t_save;
  a.A = A;
  a.B = B;
  a.dY = dY;
  a.dX = dX;
  a.dA = dA;
  a.dB = dB;
  return lora_group_bwd(&a, 1, T, r, alpha, workspace, ws_bytes, stream);
}

}  // extern "C"
