// C ABI of libwhtq: argument validation, then dispatch to the kernels.
// Every check runs before the first HIP call, so an error status means
// nothing was enqueued.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>
#include <vector>

#include "../../include/whtq.h"
#include "kv_attn.hpp"
#include "launch.hpp"
#include "logprob.hpp"
#include "qk_norm.hpp"

namespace whtq {

hipError_t launch_stream_probe(const void* src, int64_t in_bytes, void* dst, int64_t out_bytes, hipStream_t s);
hipError_t launch_wht(int logn, int din, int dout, const void* x, void* y, int64_t rows, int64_t ldx,
                      int64_t ldy, const uint32_t* sbits, int sign_mode, float scale, hipStream_t s);
hipError_t launch_rht_quant(int logn, int din, int bits, int logg, const void* w, int64_t rows,
                            int64_t ldw, const uint32_t* sb, uint8_t* codes, uint16_t* scales,
                            hipStream_t s);
hipError_t launch_rht_dequant(int logn, int dout, int bits, int logg, const uint8_t* codes,
                              const uint16_t* scales, int64_t rows, const uint32_t* sb, void* out,
                              int64_t ldo, hipStream_t s);
hipError_t launch_rht_gemv(int logn, int bits, int logg, const void* x, int64_t tokens, int64_t ldx,
                           const uint8_t* codes, const uint16_t* scales, int64_t rows, const uint32_t* sb,
                           void* y, int64_t ldy, hipStream_t s);
hipError_t launch_qwha(const void* x, int64_t tokens, int64_t d_in, int64_t ldx, const int32_t* row_ptr,
                       const int32_t* col_idx, const void* vals, int val_dt, int64_t d_out, int64_t nnz,
                       void* y, int64_t ldy, const void* plan, int64_t plan_bytes, hipStream_t s);
int64_t qwha_fwd_plan_bytes(int64_t tokens, int64_t d_out, int64_t nnz);
hipError_t launch_qwha_fwd_plan(int64_t tokens, const int32_t* row_ptr, int64_t d_out, int64_t nnz, void* plan,
                                int64_t plan_bytes, hipStream_t s);
hipError_t launch_qwha_bwd_input(const void* dy, int64_t tokens, int64_t lddy, int64_t d_out,
                                 const int32_t* t_row_ptr, const int32_t* t_col_idx, const void* t_vals,
                                 int val_dt, int64_t d_in, int64_t nnz, void* dx, int64_t lddx, hipStream_t s);
int64_t qwha_dc_workspace_bytes(int64_t tokens, int64_t d_in, int64_t nnz);
hipError_t launch_qwha_dc(const void* x, int64_t ldx, const void* dy, int64_t lddy, int64_t tokens, int64_t d_in,
                          int64_t d_out, const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz,
                          float* dc, void* workspace, hipStream_t s);
hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t s);
hipError_t launch_permute(const void* vals, int val_dt, const int32_t* perm, int64_t nnz, void* out,
                          hipStream_t s);
hipError_t launch_harp_gen(const void* x, void* y, int xdt, int64_t tokens, int d, int64_t ldx, int64_t ldy,
                           const uint32_t* sbits, int precondition, const int32_t* radices, int n_stages,
                           const void* blocks, int bdt, hipStream_t s);
hipError_t launch_harp_build(const void* params, int pdt, const float* scales, int64_t d, const int32_t* radices,
                             int n_stages, const float* mixers, void* blocks, int bdt, hipStream_t s);
hipError_t launch_harp(const void* x, void* y, int dt, int64_t tokens, int64_t ldx, int64_t ldy,
                       const uint32_t* sbits, int precondition, const void* blocks, int bdt, hipStream_t s);
hipError_t launch_qi_sub(const void* w, int wdt, int64_t ldw, float* f, int64_t ldf, int64_t rows, int64_t n,
                         hipStream_t s);
hipError_t launch_qi_gram(const float* z, int64_t T, int64_t n, float* g, float beta, hipStream_t s);
hipError_t launch_qi_fg(const float* f, int64_t ldf, int64_t rows, int64_t n, const float* g, float* p,
                        hipStream_t s);
hipError_t launch_qi_qform(const float* f, int64_t ldf, const float* p, int64_t rows, int64_t n, float* err,
                           hipStream_t s);
hipError_t launch_qi_select(const float* f, int64_t ldf, int64_t rows, int n, const int32_t* row_ptr,
                            int32_t* col_idx, hipStream_t s);
hipError_t launch_qi_refine(const float* g, int64_t n, const float* p, int64_t rows, const int32_t* row_ptr,
                            const int32_t* col_idx, float* vals, hipStream_t s);

hipError_t launch_kv_gather(const KvCache& c, int dim, int dt, bool int4, int64_t tokens, const int64_t* slots,
                            int64_t capacity, void* ko, const int64_t* ks, void* vo, const int64_t* vs,
                            hipStream_t s);
hipError_t launch_kv_step(const KvAttnArgs& a, int dim, int dt, bool int4, int nq, hipStream_t s);
hipError_t launch_kv_join(const KvAttnArgs& a, int dim, int dt, bool int4, hipStream_t s);
hipError_t launch_kv_chunk(const KvAttnArgs& a, int dim, int dt, bool int4, int waves, hipStream_t s);
int kv_step_unit(int dim, bool int4, bool whole);
int64_t qk_norm_split(QkArgs& a, int dim, int cus);
hipError_t launch_qk_norm(const QkForwardArgs& a, const int (&heads)[3], int64_t tokens, int dim, int dt, bool int4,
                          hipStream_t s);
hipError_t launch_qk_norm_back(const QkArgs& a, int dim, int dt, hipStream_t s);
hipError_t launch_lp(const LpArgs& a, int dt, hipStream_t s);
hipError_t launch_lp_grad(const LpGradArgs& a, int dt, hipStream_t s);

static thread_local int g_last_hip = 0;

static constexpr int kMaxDevices = 64;
static int g_cu[kMaxDevices];
static std::once_flag g_cu_once[kMaxDevices];

int device_cu_count(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return 256;
  std::call_once(g_cu_once[dev], [dev] {
    int cu = 0;
    if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cu < 1)
      cu = 256;
    g_cu[dev] = cu;
  });
  return g_cu[dev];
}

}  // namespace whtq

using namespace whtq;

static whtq_status hip_status(hipError_t e) {
  if (e == hipSuccess) return WHTQ_OK;
  g_last_hip = (int)e;
  return WHTQ_EHIP;
}

// A device must be present and current before anything is launched.
static whtq_status need_device() {
  static std::atomic<bool> found{false};  // devices do not go away; the count costs a microsecond a call
  if (found.load(std::memory_order_relaxed)) return WHTQ_OK;
  int n = 0;
  hipError_t e = hipGetDeviceCount(&n);
  if (e != hipSuccess) return hip_status(e);
  if (n < 1) return hip_status(hipErrorNoDevice);
  found.store(true, std::memory_order_relaxed);
  return WHTQ_OK;
}

static int ilog2_pow2(int64_t n) {
  if (n < 1 || (n & (n - 1))) return -1;
  int l = 0;
  while ((int64_t(1) << l) < n) ++l;
  return l;
}

static int dt_bytes(int dt) { return dt == WHTQ_F32 ? 4 : 2; }
static bool dt_valid(int dt) { return dt == WHTQ_F32 || dt == WHTQ_BF16 || dt == WHTQ_F16; }

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row-matrix alignment rule: 16-byte base and row stride unless a row is
// shorter than 16 bytes, then element alignment.
static bool rows_aligned(const void* p, int64_t n, int64_t ld, int esz) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (n * esz >= 16) return (a & 15u) == 0 && ((ld * esz) & 15) == 0;
  return (a % (uintptr_t)esz) == 0;
}

extern "C" {

int whtq_abi_version(void) { return WHTQ_ABI_VERSION; }

int whtq_last_hip_error(void) { return g_last_hip; }

whtq_status whtq_stream_probe(const void* src, int64_t in_bytes, void* dst, int64_t out_bytes, void* stream) {
  if (in_bytes < 0 || out_bytes < 0 || (in_bytes & 15) || (out_bytes & 15)) return WHTQ_EINVAL;
  if ((in_bytes > 0 && !src) || (out_bytes > 0 && !dst)) return WHTQ_EINVAL;
  if ((src && !aligned16(src)) || (dst && !aligned16(dst))) return WHTQ_EALIGN;
  if (in_bytes == 0 && out_bytes == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(whtq::launch_stream_probe(src, in_bytes, dst, out_bytes, (hipStream_t)stream));
}

const char* whtq_status_string(whtq_status s) {
  switch (s) {
    case WHTQ_OK: return "ok";
    case WHTQ_EINVAL: return "invalid argument";
    case WHTQ_EUNSUPPORTED: return "unsupported configuration";
    case WHTQ_EALIGN: return "misaligned pointer or row stride";
    case WHTQ_EHIP: return "HIP runtime error";
    case WHTQ_ESCRATCH: return "sizes exceed the fixed scratch capacity";
  }
  return "unknown status";
}

whtq_status wht_batched(const void* x, whtq_dtype x_dtype, void* y, whtq_dtype y_dtype, int64_t rows,
                        int64_t n, int64_t ldx, int64_t ldy, const uint32_t* sign_bits, int sign_mode,
                        int normalize, void* stream) {
  if (!dt_valid(x_dtype) || !dt_valid(y_dtype)) return WHTQ_EINVAL;
  if (rows < 0 || n < 1 || ldx < n || ldy < n) return WHTQ_EINVAL;
  if (sign_mode < WHTQ_SIGN_NONE || sign_mode > WHTQ_SIGN_AFTER) return WHTQ_EINVAL;
  if (sign_mode != WHTQ_SIGN_NONE && !sign_bits) return WHTQ_EINVAL;
  if (normalize != 0 && normalize != 1) return WHTQ_EINVAL;
  if (rows > 0 && (!x || !y)) return WHTQ_EINVAL;
  const int logn = ilog2_pow2(n);
  if (logn < 1 || logn > 13) return WHTQ_EUNSUPPORTED;
  const bool same = x_dtype == y_dtype;
  const bool widen = y_dtype == WHTQ_F32 && x_dtype != WHTQ_F32;
  if (!same && !widen) return WHTQ_EUNSUPPORTED;
  if (x == y && (!same || ldx != ldy)) return WHTQ_EINVAL;
  if (!rows_aligned(x, n, ldx, dt_bytes(x_dtype)) || !rows_aligned(y, n, ldy, dt_bytes(y_dtype)))
    return WHTQ_EALIGN;
  if (sign_bits && (reinterpret_cast<uintptr_t>(sign_bits) & 3u)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  const float scale = normalize ? (float)(1.0 / std::sqrt((double)n)) : 1.0f;
  return hip_status(launch_wht(logn, x_dtype, y_dtype, x, y, rows, ldx, ldy, sign_bits, sign_mode, scale,
                               (hipStream_t)stream));
}

static whtq_status check_quant_shape(int64_t rows, int64_t n, int bits, int group, int* logn, int* logg) {
  if (rows < 0 || n < 1) return WHTQ_EINVAL;
  if (bits < 2 || bits > 4) return WHTQ_EINVAL;
  if (group < 1 || n % group) return WHTQ_EINVAL;
  *logn = ilog2_pow2(n);
  if (*logn < 0) return WHTQ_EUNSUPPORTED;
  *logg = ilog2_pow2(group);
  if (*logg < 3) return WHTQ_EINVAL;  // group must be a power of two >= 8 (it divides n)
  if (*logn < 6 || *logn > 13 || *logg > 8) return WHTQ_EUNSUPPORTED;
  return WHTQ_OK;
}

whtq_status rht_quantize_rtn(const void* w, whtq_dtype w_dtype, int64_t rows, int64_t n, int64_t ldw,
                             const uint32_t* sign_bits, int bits, int group, uint8_t* codes,
                             uint16_t* scales, void* stream) {
  if (!dt_valid(w_dtype)) return WHTQ_EINVAL;
  int logn = 0, logg = 0;
  whtq_status st = check_quant_shape(rows, n, bits, group, &logn, &logg);
  if (st != WHTQ_OK) return st;
  if (ldw < n) return WHTQ_EINVAL;
  if (rows > 0 && (!w || !codes || !scales)) return WHTQ_EINVAL;
  if (!rows_aligned(w, n, ldw, dt_bytes(w_dtype)) || !aligned16(codes) || !aligned16(scales))
    return WHTQ_EALIGN;
  if (sign_bits && (reinterpret_cast<uintptr_t>(sign_bits) & 3u)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_rht_quant(logn, w_dtype, bits, logg, w, rows, ldw, sign_bits, codes, scales,
                                     (hipStream_t)stream));
}

whtq_status rht_dequantize_inverse(const uint8_t* codes, const uint16_t* scales, int64_t rows, int64_t n,
                                   const uint32_t* sign_bits, int bits, int group, void* out,
                                   whtq_dtype out_dtype, int64_t ldo, void* stream) {
  if (!dt_valid(out_dtype)) return WHTQ_EINVAL;
  int logn = 0, logg = 0;
  whtq_status st = check_quant_shape(rows, n, bits, group, &logn, &logg);
  if (st != WHTQ_OK) return st;
  if (ldo < n) return WHTQ_EINVAL;
  if (rows > 0 && (!codes || !scales || !out)) return WHTQ_EINVAL;
  if (!rows_aligned(out, n, ldo, dt_bytes(out_dtype)) || !aligned16(codes) || !aligned16(scales))
    return WHTQ_EALIGN;
  if (sign_bits && (reinterpret_cast<uintptr_t>(sign_bits) & 3u)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_rht_dequant(logn, out_dtype, bits, logg, codes, scales, rows, sign_bits, out, ldo,
                                       (hipStream_t)stream));
}

whtq_status rht_lowbit_gemv(const void* x, int64_t tokens, int64_t ldx, const uint8_t* codes,
                            const uint16_t* scales, int64_t rows, int64_t n, const uint32_t* sign_bits,
                            int bits, int group, void* y, int64_t ldy, void* stream) {
  int logn = 0, logg = 0;
  whtq_status st = check_quant_shape(rows, n, bits, group, &logn, &logg);
  if (st != WHTQ_OK) return st;
  if (tokens < 0 || ldx < n || ldy < rows) return WHTQ_EINVAL;
  if (tokens > 0 && rows > 0 && (!x || !codes || !scales || !y)) return WHTQ_EINVAL;
  if (bits == 3 || (logn != 12 && logn != 13) || (1 << logg) < 32 / bits) return WHTQ_EUNSUPPORTED;
  if (!rows_aligned(x, n, ldx, 2) || !aligned16(codes) || !aligned16(scales) ||
      (reinterpret_cast<uintptr_t>(y) & 1u))
    return WHTQ_EALIGN;
  if (sign_bits && (reinterpret_cast<uintptr_t>(sign_bits) & 3u)) return WHTQ_EALIGN;
  if (tokens == 0 || rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_rht_gemv(logn, bits, logg, x, tokens, ldx, codes, scales, rows, sign_bits, y, ldy,
                                    (hipStream_t)stream));
}

// the argument rules of qwha_adapter_forward (shared with the planned form)
static whtq_status qwha_fwd_check(const void* x, whtq_dtype x_dtype, int64_t tokens, int64_t d_in, int64_t ldx,
                                  const int32_t* row_ptr, const int32_t* col_idx, const void* vals,
                                  whtq_dtype val_dtype, int64_t d_out, int64_t nnz, void* y, whtq_dtype y_dtype,
                                  int64_t ldy) {
  if (!dt_valid(x_dtype) || !dt_valid(val_dtype) || !dt_valid(y_dtype)) return WHTQ_EINVAL;
  if (tokens < 0 || d_in < 1 || d_out < 1 || nnz < 0 || ldx < d_in || ldy < d_out) return WHTQ_EINVAL;
  if (nnz > d_in * d_out) return WHTQ_EINVAL;
  if (!row_ptr || (nnz > 0 && (!col_idx || !vals))) return WHTQ_EINVAL;
  if (tokens > 0 && (!x || !y)) return WHTQ_EINVAL;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13 || d_out > 4096) return WHTQ_EUNSUPPORTED;
  if (x_dtype != WHTQ_BF16 || y_dtype != WHTQ_BF16) return WHTQ_EUNSUPPORTED;
  if (val_dtype != WHTQ_BF16 && val_dtype != WHTQ_F32) return WHTQ_EUNSUPPORTED;
  if (!rows_aligned(x, d_in, ldx, 2) || !rows_aligned(y, d_out, ldy, 2)) return WHTQ_EALIGN;
  if ((reinterpret_cast<uintptr_t>(row_ptr) & 3u) || !aligned16(col_idx) || !aligned16(vals)) return WHTQ_EALIGN;
  return WHTQ_OK;
}

whtq_status qwha_adapter_forward(const void* x, whtq_dtype x_dtype, int64_t tokens, int64_t d_in,
                                 int64_t ldx, const int32_t* row_ptr, const int32_t* col_idx,
                                 const void* vals, whtq_dtype val_dtype, int64_t d_out, int64_t nnz,
                                 void* y, whtq_dtype y_dtype, int64_t ldy, void* stream) {
  return qwha_adapter_forward_planned(x, x_dtype, tokens, d_in, ldx, row_ptr, col_idx, vals, val_dtype, d_out, nnz,
                                      nullptr, 0, y, y_dtype, ldy, stream);
}

int64_t qwha_forward_plan_bytes(int64_t tokens, int64_t d_in, int64_t d_out, int64_t nnz) {
  if (tokens < 1 || d_out < 1 || d_out > 4096 || nnz < 0 || nnz > d_in * d_out) return -1;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13) return -1;
  if (d_in > 4096) return 0;  // the d_in = 8192 kernel prepares nothing per chunk
  if (need_device() != WHTQ_OK) return -1;
  return qwha_fwd_plan_bytes(tokens, d_out, nnz);
}

whtq_status qwha_forward_plan(int64_t tokens, int64_t d_in, const int32_t* row_ptr, int64_t d_out, int64_t nnz,
                              void* plan, int64_t plan_bytes, void* stream) {
  if (tokens < 1 || d_out < 1 || nnz < 0 || nnz > d_in * d_out || plan_bytes < 0) return WHTQ_EINVAL;
  if (!row_ptr || (reinterpret_cast<uintptr_t>(row_ptr) & 3u)) return row_ptr ? WHTQ_EALIGN : WHTQ_EINVAL;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13 || d_out > 4096) return WHTQ_EUNSUPPORTED;
  if (d_in > 4096) return WHTQ_OK;  // nothing to plan
  if (!plan) return WHTQ_EINVAL;
  if (!aligned16(plan)) return WHTQ_EALIGN;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  if (plan_bytes < qwha_fwd_plan_bytes(tokens, d_out, nnz)) return WHTQ_EINVAL;
  return hip_status(launch_qwha_fwd_plan(tokens, row_ptr, d_out, nnz, plan, plan_bytes, (hipStream_t)stream));
}

whtq_status qwha_adapter_forward_planned(const void* x, whtq_dtype x_dtype, int64_t tokens, int64_t d_in,
                                         int64_t ldx, const int32_t* row_ptr, const int32_t* col_idx,
                                         const void* vals, whtq_dtype val_dtype, int64_t d_out, int64_t nnz,
                                         const void* plan, int64_t plan_bytes, void* y, whtq_dtype y_dtype,
                                         int64_t ldy, void* stream) {
  whtq_status st = qwha_fwd_check(x, x_dtype, tokens, d_in, ldx, row_ptr, col_idx, vals, val_dtype, d_out, nnz, y,
                                  y_dtype, ldy);
  if (st != WHTQ_OK) return st;
  if (plan_bytes < 0 || (plan && plan_bytes < 256)) return WHTQ_EINVAL;
  if (plan && !aligned16(plan)) return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_qwha(x, tokens, d_in, ldx, row_ptr, col_idx, vals, val_dtype, d_out, nnz, y, ldy,
                                plan, plan ? plan_bytes : 0, (hipStream_t)stream));
}

whtq_status qwha_csr_transpose(const int32_t* row_ptr, const int32_t* col_idx, int64_t d_out, int64_t d_in,
                               int64_t nnz, int32_t* t_row_ptr, int32_t* t_col_idx, int32_t* t_perm) {
  if (d_out < 1 || d_in < 1 || nnz < 0 || d_out > INT32_MAX || d_in > INT32_MAX || nnz > INT32_MAX)
    return WHTQ_EINVAL;
  if (!row_ptr || !t_row_ptr || (nnz > 0 && (!col_idx || !t_col_idx || !t_perm))) return WHTQ_EINVAL;
  // the CSR is read here, so it is checked in full first
  if (row_ptr[0] != 0 || row_ptr[d_out] != nnz) return WHTQ_EINVAL;
  for (int64_t o = 0; o < d_out; ++o)
    if (row_ptr[o + 1] < row_ptr[o]) return WHTQ_EINVAL;
  for (int64_t j = 0; j < nnz; ++j)
    if (col_idx[j] < 0 || col_idx[j] >= d_in) return WHTQ_EINVAL;
  // counting sort by column, stable in entry order (rows ascending within a
  // column); t_row_ptr[k] serves as column k's cursor, then shifts back
  for (int64_t k = 0; k <= d_in; ++k) t_row_ptr[k] = 0;
  for (int64_t j = 0; j < nnz; ++j) ++t_row_ptr[col_idx[j] + 1];
  for (int64_t k = 0; k < d_in; ++k) t_row_ptr[k + 1] += t_row_ptr[k];
  for (int64_t o = 0; o < d_out; ++o)
    for (int32_t j = row_ptr[o]; j < row_ptr[o + 1]; ++j) {
      const int32_t pos = t_row_ptr[col_idx[j]]++;
      t_col_idx[pos] = (int32_t)o;
      t_perm[pos] = j;
    }
  for (int64_t k = d_in; k > 0; --k) t_row_ptr[k] = t_row_ptr[k - 1];
  t_row_ptr[0] = 0;
  return WHTQ_OK;
}

whtq_status qwha_permute_values(const void* vals, whtq_dtype val_dtype, const int32_t* perm, int64_t nnz,
                                void* out, void* stream) {
  if (!dt_valid(val_dtype) || nnz < 0) return WHTQ_EINVAL;
  if (nnz > 0 && (!vals || !perm || !out)) return WHTQ_EINVAL;
  if (nnz > 0 && vals == out) return WHTQ_EINVAL;
  if (val_dtype == WHTQ_F16) return WHTQ_EUNSUPPORTED;
  const uintptr_t esz = (uintptr_t)dt_bytes(val_dtype);
  if ((reinterpret_cast<uintptr_t>(vals) % esz) || (reinterpret_cast<uintptr_t>(out) % esz) ||
      (reinterpret_cast<uintptr_t>(perm) & 3u))
    return WHTQ_EALIGN;
  if (nnz == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_permute(vals, val_dtype, perm, nnz, out, (hipStream_t)stream));
}

whtq_status qwha_adapter_backward_input(const void* dy, whtq_dtype dy_dtype, int64_t tokens, int64_t d_out,
                                        int64_t lddy, const int32_t* t_row_ptr, const int32_t* t_col_idx,
                                        const void* t_vals, whtq_dtype val_dtype, int64_t d_in, int64_t nnz,
                                        void* dx, whtq_dtype dx_dtype, int64_t lddx, void* stream) {
  if (!dt_valid(dy_dtype) || !dt_valid(val_dtype) || !dt_valid(dx_dtype)) return WHTQ_EINVAL;
  if (tokens < 0 || d_in < 1 || d_out < 1 || nnz < 0 || lddy < d_out || lddx < d_in) return WHTQ_EINVAL;
  if (nnz > d_in * d_out) return WHTQ_EINVAL;
  if (!t_row_ptr || (nnz > 0 && (!t_col_idx || !t_vals))) return WHTQ_EINVAL;
  if (tokens > 0 && (!dy || !dx)) return WHTQ_EINVAL;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13 || d_out > 4096) return WHTQ_EUNSUPPORTED;
  if (dy_dtype != WHTQ_BF16 || dx_dtype != WHTQ_BF16) return WHTQ_EUNSUPPORTED;
  if (val_dtype != WHTQ_BF16 && val_dtype != WHTQ_F32) return WHTQ_EUNSUPPORTED;
  // dy: element alignment suffices (16-byte loads are used where its rows allow them)
  if ((reinterpret_cast<uintptr_t>(dy) & 1u) || !rows_aligned(dx, d_in, lddx, 2)) return WHTQ_EALIGN;
  if ((reinterpret_cast<uintptr_t>(t_row_ptr) & 3u) || !aligned16(t_col_idx) || !aligned16(t_vals))
    return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_qwha_bwd_input(dy, tokens, lddy, d_out, t_row_ptr, t_col_idx, t_vals, val_dtype, d_in,
                                          nnz, dx, lddx, (hipStream_t)stream));
}

int64_t qwha_grad_values_workspace_bytes(int64_t tokens, int64_t d_in, int64_t nnz) {
  if (tokens < 0 || nnz < 0 || ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13) return -1;
  if (tokens == 0 || nnz == 0) return 0;
  return qwha_dc_workspace_bytes(tokens, d_in, nnz);
}

whtq_status qwha_adapter_grad_values(const void* x, const void* dy, whtq_dtype dtype, int64_t tokens,
                                     int64_t d_in, int64_t d_out, int64_t ldx, int64_t lddy,
                                     const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz, float* dc,
                                     void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dt_valid(dtype)) return WHTQ_EINVAL;
  if (tokens < 0 || d_in < 1 || d_out < 1 || nnz < 0 || ldx < d_in || lddy < d_out) return WHTQ_EINVAL;
  if (nnz > d_in * d_out || nnz > INT32_MAX) return WHTQ_EINVAL;
  if (!row_ptr || (nnz > 0 && (!col_idx || !dc))) return WHTQ_EINVAL;
  if (tokens > 0 && nnz > 0 && (!x || !dy || !workspace)) return WHTQ_EINVAL;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13 || d_out > 4096) return WHTQ_EUNSUPPORTED;
  if (dtype != WHTQ_BF16) return WHTQ_EUNSUPPORTED;
  // dy is read with element loads: element alignment suffices
  if (!rows_aligned(x, d_in, ldx, 2) || (reinterpret_cast<uintptr_t>(dy) & 1u)) return WHTQ_EALIGN;
  if ((reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u) ||
      (reinterpret_cast<uintptr_t>(dc) & 3u) || !aligned16(workspace))
    return WHTQ_EALIGN;
  if (tokens > 0 && nnz > 0 && workspace_bytes < qwha_dc_workspace_bytes(tokens, d_in, nnz)) return WHTQ_EINVAL;
  if (nnz == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  if (tokens == 0)  // an empty sum: dc = 0 (a fill kernel, not a memset node)
    return hip_status(launch_fill_zero(dc, nnz, (hipStream_t)stream));
  return hip_status(launch_qwha_dc(x, ldx, dy, lddy, tokens, d_in, d_out, row_ptr, col_idx, nnz, dc, workspace,
                                   (hipStream_t)stream));
}

}  // extern "C"

// Scratch of the allocation-free value gradient: one array per GPU, resolved
// to a device address once per device with that device current (the array's
// name in host code is only a host-side handle, never a device address).
static __device__ __align__(256) uint8_t scratch[WHTQ_QWHA_DC_SCRATCH_BYTES];
static void* g_scratch_ptr[kMaxDevices];
static hipError_t g_scratch_err[kMaxDevices];
static std::once_flag g_scratch_once[kMaxDevices];

static whtq_status scratch_of_current_device(void** ptr) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e);
  if (dev < 0 || dev >= kMaxDevices) return WHTQ_EUNSUPPORTED;
  std::call_once(g_scratch_once[dev], [dev] {
    void* p = nullptr;
    g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    g_scratch_ptr[dev] = g_scratch_err[dev] == hipSuccess ? p : nullptr;
  });
  if (g_scratch_err[dev] != hipSuccess) return hip_status(g_scratch_err[dev]);
  *ptr = g_scratch_ptr[dev];
  return WHTQ_OK;
}

extern "C" {

whtq_status qwha_adapter_grad_values_noalloc(const void* x, const void* dy, whtq_dtype dtype, int64_t tokens,
                                             int64_t d_in, int64_t d_out, int64_t ldx, int64_t lddy,
                                             const int32_t* row_ptr, const int32_t* col_idx, int64_t nnz,
                                             float* dc, void* stream) {
  // the same checks as qwha_adapter_grad_values, then the capacity
  if (!dt_valid(dtype)) return WHTQ_EINVAL;
  if (tokens < 0 || d_in < 1 || d_out < 1 || nnz < 0 || ldx < d_in || lddy < d_out) return WHTQ_EINVAL;
  if (nnz > d_in * d_out || nnz > INT32_MAX) return WHTQ_EINVAL;
  if (!row_ptr || (nnz > 0 && (!col_idx || !dc))) return WHTQ_EINVAL;
  if (tokens > 0 && nnz > 0 && (!x || !dy)) return WHTQ_EINVAL;
  if (ilog2_pow2(d_in) < 6 || ilog2_pow2(d_in) > 13 || d_out > 4096) return WHTQ_EUNSUPPORTED;
  if (dtype != WHTQ_BF16) return WHTQ_EUNSUPPORTED;
  if (!rows_aligned(x, d_in, ldx, 2) || (reinterpret_cast<uintptr_t>(dy) & 1u)) return WHTQ_EALIGN;
  if ((reinterpret_cast<uintptr_t>(row_ptr) & 3u) || (reinterpret_cast<uintptr_t>(col_idx) & 3u) ||
      (reinterpret_cast<uintptr_t>(dc) & 3u))
    return WHTQ_EALIGN;
  if (tokens > 0 && nnz > 0 && qwha_dc_workspace_bytes(tokens, d_in, nnz) > WHTQ_QWHA_DC_SCRATCH_BYTES)
    return WHTQ_ESCRATCH;
  if (nnz == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  if (tokens == 0) return hip_status(launch_fill_zero(dc, nnz, (hipStream_t)stream));
  void* ws = nullptr;
  st = scratch_of_current_device(&ws);
  if (st != WHTQ_OK) return st;
  return hip_status(launch_qwha_dc(x, ldx, dy, lddy, tokens, d_in, d_out, row_ptr, col_idx, nnz, dc, ws,
                                   (hipStream_t)stream));
}

whtq_status harp_rotate(const void* x, void* y, whtq_dtype dtype, int64_t tokens, int64_t d, int64_t ldx,
                        int64_t ldy, const uint32_t* sign_bits, int precondition, const int32_t* radices,
                        int n_stages, const void* blocks, whtq_dtype blocks_dtype, void* stream) {
  if (!dt_valid(dtype) || !dt_valid(blocks_dtype)) return WHTQ_EINVAL;
  if (tokens < 0 || d < 1 || ldx < d || ldy < d) return WHTQ_EINVAL;
  if (!radices || n_stages < 1 || n_stages > 64 || !blocks) return WHTQ_EINVAL;
  if (precondition != 0 && precondition != 1) return WHTQ_EINVAL;
  int64_t prod = 1;
  for (int t = 0; t < n_stages; ++t) {
    if (radices[t] < 2) return WHTQ_EINVAL;
    prod *= radices[t];
    if (prod > d) return WHTQ_EINVAL;
  }
  if (prod != d) return WHTQ_EINVAL;
  if (tokens > 0 && (!x || !y)) return WHTQ_EINVAL;
  if (tokens > 0 && x == y) return WHTQ_EINVAL;
  // the preconditioning is the Sylvester RHT, which exists for powers of two only
  if (precondition && ilog2_pow2(d) < 0) return WHTQ_EINVAL;
  // fp32 rows take the fp32-tile kernel for every schedule (the radix-16 one
  // multiplies in fp16)
  const bool r16 = dtype == WHTQ_BF16 && d == 4096 && n_stages == 3 && radices[0] == 16 && radices[1] == 16 &&
                   radices[2] == 16;
  if (!r16) {
    if (d > 8192 || n_stages > 16) return WHTQ_EUNSUPPORTED;
    for (int t = 0; t < n_stages; ++t)
      if (radices[t] > 16) return WHTQ_EUNSUPPORTED;
  }
  if ((dtype != WHTQ_BF16 && dtype != WHTQ_F32) || blocks_dtype == WHTQ_BF16) return WHTQ_EUNSUPPORTED;
  const int esz = dt_bytes(dtype);
  if (!rows_aligned(x, d, ldx, esz) || !rows_aligned(y, d, ldy, esz) || !aligned16(blocks)) return WHTQ_EALIGN;
  if (sign_bits && (reinterpret_cast<uintptr_t>(sign_bits) & 3u)) return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  if (r16)
    return hip_status(launch_harp(x, y, dtype, tokens, ldx, ldy, sign_bits, precondition, blocks, blocks_dtype,
                                  (hipStream_t)stream));
  return hip_status(launch_harp_gen(x, y, dtype, tokens, (int)d, ldx, ldy, sign_bits, precondition, radices, n_stages,
                                    blocks, blocks_dtype, (hipStream_t)stream));
}

whtq_status harp_build_blocks(const void* params, whtq_dtype params_dtype, const float* scales, int64_t d,
                              const int32_t* radices, int n_stages, const float* mixers, void* blocks,
                              whtq_dtype blocks_dtype, void* stream) {
  if (params_dtype != WHTQ_F32 && params_dtype != WHTQ_I8) return WHTQ_EINVAL;
  if (blocks_dtype != WHTQ_F32 && blocks_dtype != WHTQ_F16) return WHTQ_EINVAL;
  if (!radices || n_stages < 1 || n_stages > 64 || d < 1 || !params || !blocks) return WHTQ_EINVAL;
  if (params_dtype == WHTQ_I8 && !scales) return WHTQ_EINVAL;
  int64_t prod = 1;
  bool pow2 = true;
  for (int t = 0; t < n_stages; ++t) {
    if (radices[t] < 2) return WHTQ_EINVAL;
    prod *= radices[t];
    if (prod > d) return WHTQ_EINVAL;
    pow2 = pow2 && (radices[t] & (radices[t] - 1)) == 0;
  }
  if (prod != d) return WHTQ_EINVAL;
  // the Sylvester mixer exists for power-of-two radices only
  if (!mixers && !pow2) return WHTQ_EINVAL;
  if (n_stages > 16 || d > (int64_t(1) << 24)) return WHTQ_EUNSUPPORTED;
  for (int t = 0; t < n_stages; ++t)
    if (radices[t] > 16) return WHTQ_EUNSUPPORTED;
  if ((params_dtype == WHTQ_F32 && (reinterpret_cast<uintptr_t>(params) & 3u)) ||
      (reinterpret_cast<uintptr_t>(blocks) % (uintptr_t)dt_bytes(blocks_dtype)) ||
      (reinterpret_cast<uintptr_t>(mixers) & 3u) || (reinterpret_cast<uintptr_t>(scales) & 3u))
    return WHTQ_EALIGN;
  whtq_status st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_harp_build(params, params_dtype, scales, d, radices, n_stages, mixers, blocks,
                                      blocks_dtype, (hipStream_t)stream));
}


// ---------------------------------------------------------------- QWHA initialisation

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// n of the initialisation calls after the error coefficients: a power of two in [256, 8192]
static whtq_status qi_n(int64_t n) {
  const int l = ilog2_pow2(n);
  if (l < 0) return WHTQ_EINVAL;
  if (l < 8 || l > 13) return WHTQ_EUNSUPPORTED;
  return WHTQ_OK;
}

whtq_status qwha_init_error_coeffs(const void* w, whtq_dtype w_dtype, int64_t rows, int64_t n, int64_t ldw,
                                   const uint8_t* codes, const uint16_t* scales, const uint32_t* sign_bits,
                                   int bits, int group, float* f, int64_t ldf, void* stream) {
  if (!dt_valid(w_dtype)) return WHTQ_EINVAL;
  int logn = 0, logg = 0;
  whtq_status st = check_quant_shape(rows, n, bits, group, &logn, &logg);
  if (st != WHTQ_OK) return st;
  if (ldw < n || ldf < n) return WHTQ_EINVAL;
  if (rows > 0 && (!w || !codes || !scales || !f)) return WHTQ_EINVAL;
  if (rows > 0 && static_cast<const void*>(f) == w) return WHTQ_EINVAL;
  if ((reinterpret_cast<uintptr_t>(w) % (uintptr_t)dt_bytes(w_dtype)) || !rows_aligned(f, n, ldf, 4) ||
      !aligned16(codes) || !aligned16(scales))
    return WHTQ_EALIGN;
  if (sign_bits && !aligned4(sign_bits)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = launch_rht_dequant(logn, WHTQ_F32, bits, logg, codes, scales, rows, sign_bits, f, ldf, s);
  if (e == hipSuccess) e = launch_qi_sub(w, w_dtype, ldw, f, ldf, rows, n, s);
  if (e == hipSuccess)
    e = launch_wht(logn, WHTQ_F32, WHTQ_F32, f, f, rows, ldf, ldf, nullptr, WHTQ_SIGN_NONE,
                   (float)(1.0 / std::sqrt((double)n)), s);
  return hip_status(e);
}

whtq_status qwha_init_gram(const void* x, whtq_dtype x_dtype, int64_t tokens, int64_t n, int64_t ldx, float* z,
                           float* g, int accumulate, void* stream) {
  if (!dt_valid(x_dtype)) return WHTQ_EINVAL;
  whtq_status st = qi_n(n);
  if (st != WHTQ_OK) return st;
  if (tokens < 0 || ldx < n || (accumulate != 0 && accumulate != 1)) return WHTQ_EINVAL;
  if (!g || (tokens > 0 && (!x || !z))) return WHTQ_EINVAL;
  if (tokens > 0 && z == g) return WHTQ_EINVAL;  // Z is read while G is written
  if (!rows_aligned(x, n, ldx, dt_bytes(x_dtype)) || !aligned16(z) || !aligned16(g)) return WHTQ_EALIGN;
  if (tokens == 0 && accumulate) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (tokens > 0)
    e = launch_wht(ilog2_pow2(n), x_dtype, WHTQ_F32, x, z, tokens, ldx, n, nullptr, WHTQ_SIGN_NONE,
                   (float)(1.0 / std::sqrt((double)n)), s);
  if (e == hipSuccess) e = launch_qi_gram(z, tokens, n, g, accumulate ? 1.f : 0.f, s);
  return hip_status(e);
}

whtq_status qwha_init_channel_errors(const float* f, int64_t rows, int64_t n, int64_t ldf, const float* g,
                                     float* p, float* err, void* stream) {
  whtq_status st = qi_n(n);
  if (st != WHTQ_OK) return st;
  if (rows < 0 || ldf < n) return WHTQ_EINVAL;
  if (rows > 0 && (!f || !g || !p || !err)) return WHTQ_EINVAL;
  if (rows > 0 && (p == f || p == g || static_cast<const void*>(err) == static_cast<const void*>(f) ||
                   static_cast<const void*>(err) == static_cast<const void*>(g) || err == p))
    return WHTQ_EINVAL;  // outputs must not overlay the inputs
  if (!rows_aligned(f, n, ldf, 4) || !aligned16(g) || !aligned16(p) || !aligned4(err)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = launch_qi_fg(f, ldf, rows, n, g, p, s);
  if (e == hipSuccess) e = launch_qi_qform(f, ldf, p, rows, n, err, s);
  return hip_status(e);
}

whtq_status qwha_init_allocate(const float* err, int64_t rows, int64_t n, int64_t total, int floor, int cap,
                               int32_t* row_ptr) {
  if (rows < 1 || n < 1 || !err || !row_ptr) return WHTQ_EINVAL;
  if (floor < 0 || cap < floor || cap > n) return WHTQ_EINVAL;
  if (cap > WHTQ_QWHA_INIT_MAX_SUPPORT) return WHTQ_EUNSUPPORTED;
  if (total < (int64_t)floor * rows || total > (int64_t)cap * rows || total > INT32_MAX) return WHTQ_EINVAL;
  bool any = false;
  for (int64_t o = 0; o < rows; ++o) {
    if (!std::isfinite(err[o]) || err[o] < 0.f) return WHTQ_EINVAL;
    any = any || err[o] > 0.f;
  }
  const double p = (double)total;
  std::vector<double> e64(err, err + rows);
  auto budget = [&](double lam) {  // four independent partial sums (vectorisable)
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    const double lo_v = (double)floor, hi_v = (double)cap;
    int64_t o = 0;
    for (; o + 4 <= rows; o += 4)
      for (int q = 0; q < 4; ++q) acc[q] += std::min(hi_v, std::max(lo_v, lam * e64[o + q]));
    for (; o < rows; ++o) acc[0] += std::min(hi_v, std::max(lo_v, lam * e64[o]));
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
  };
  std::vector<double> real(rows);
  if (!any) {
    std::fill(real.begin(), real.end(), p / (double)rows);
  } else {
    // water level: the sum of clip(lam e, floor, cap) is continuous and
    // non-decreasing in lam; the largest lam found with sum <= p leaves a
    // non-negative remainder for the rounding below
    double lo = 0.0, hi = 1.0;
    int doublings = 0;
    while (budget(hi) < p) {
      hi *= 2.0;
      if (++doublings > 2100) return WHTQ_EINVAL;  // channels without error sit at the floor
    }
    for (int it = 0; it < 200; ++it) {
      const double mid = 0.5 * (lo + hi);
      if (mid == lo || mid == hi) break;  // adjacent doubles: further steps change nothing
      if (budget(mid) < p) lo = mid;
      else hi = mid;
    }
    for (int64_t o = 0; o < rows; ++o)
      real[o] = std::min((double)cap, std::max((double)floor, lo * (double)err[o]));
  }
  std::vector<int64_t> base(rows);
  std::vector<int64_t> order;
  int64_t sum = 0;
  for (int64_t o = 0; o < rows; ++o) {
    base[o] = (int64_t)std::floor(real[o]);
    sum += base[o];
    if (base[o] < cap) order.push_back(o);
  }
  const int64_t rem = total - sum;
  if (rem < 0 || rem > (int64_t)order.size()) return WHTQ_EINVAL;
  // the rem channels of largest fractional part, ties to the lower channel index
  if (rem > 0 && rem < (int64_t)order.size())
    std::nth_element(order.begin(), order.begin() + rem, order.end(), [&](int64_t a, int64_t b) {
      const double fa = real[a] - (double)base[a], fb = real[b] - (double)base[b];
      return fa > fb || (fa == fb && a < b);
    });
  for (int64_t q = 0; q < rem; ++q) ++base[order[q]];
  row_ptr[0] = 0;
  for (int64_t o = 0; o < rows; ++o) row_ptr[o + 1] = row_ptr[o] + (int32_t)base[o];
  return WHTQ_OK;
}

whtq_status qwha_init_select(const float* f, int64_t rows, int64_t n, int64_t ldf, const int32_t* row_ptr,
                             int32_t* col_idx, void* stream) {
  whtq_status st = qi_n(n);
  if (st != WHTQ_OK) return st;
  if (rows < 0 || ldf < n) return WHTQ_EINVAL;
  if (rows > 0 && (!f || !row_ptr || !col_idx)) return WHTQ_EINVAL;
  if (rows > INT32_MAX) return WHTQ_EUNSUPPORTED;
  if (!rows_aligned(f, n, ldf, 4) || !aligned4(row_ptr) || !aligned4(col_idx)) return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_qi_select(f, ldf, rows, (int)n, row_ptr, col_idx, (hipStream_t)stream));
}

whtq_status qwha_init_refine(const float* g, int64_t n, const float* p, int64_t rows, const int32_t* row_ptr,
                             const int32_t* col_idx, float* vals, void* stream) {
  whtq_status st = qi_n(n);
  if (st != WHTQ_OK) return st;
  if (rows < 0) return WHTQ_EINVAL;
  if (rows > 0 && (!g || !p || !row_ptr || !col_idx || !vals)) return WHTQ_EINVAL;
  if (rows > INT32_MAX) return WHTQ_EUNSUPPORTED;
  if (!aligned4(g) || !aligned4(p) || !aligned4(row_ptr) || !aligned4(col_idx) || !aligned4(vals))
    return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_qi_refine(g, n, p, rows, row_ptr, col_idx, vals, (hipStream_t)stream));
}

}  // extern "C"

// ---------------------------------------------------------------- paged key/value cache

namespace {

constexpr int64_t kMost = int64_t(1) << 30;  // tokens, keys, pages: 32-bit positions in the kernels

bool kv_dtype(int dt) { return dt == WHTQ_BF16 || dt == WHTQ_F16; }

// the rules of a cache; fills the kernels' view of it
whtq_status kv_check(const whtq_kv_cache* c, KvCache* out) {
  if (!c) return WHTQ_EINVAL;
  if (c->format != WHTQ_KV_DENSE && c->format != WHTQ_KV_INT4) return WHTQ_EINVAL;
  const bool int4 = c->format == WHTQ_KV_INT4;
  if (!int4 && !kv_dtype(c->dtype)) return WHTQ_EINVAL;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->dim < 1 || c->page_size < 1) return WHTQ_EINVAL;
  if (!c->k || !c->v || (int4 && (!c->k_scales || !c->v_scales))) return WHTQ_EINVAL;
  const int64_t esz = int4 ? 1 : 2;
  for (int i = 0; i < 3; ++i)
    if (c->k_stride[i] < 0 || c->v_stride[i] < 0) return WHTQ_EINVAL;
  if (int4)
    for (int i = 0; i < 2; ++i)
      if (c->ks_stride[i] < 0 || c->vs_stride[i] < 0) return WHTQ_EINVAL;
  const int shift = ilog2_pow2(c->page_size);
  if (c->dim != 64 && c->dim != 128) return WHTQ_EUNSUPPORTED;
  if (shift < 4 || shift > 16 || c->num_pages > kMost || c->kv_heads > 65535) return WHTQ_EUNSUPPORTED;
  // offsets inside a page of one head are 32-bit
  if (std::max(c->k_stride[2], c->v_stride[2]) >= (int64_t(1) << 31) / c->page_size / esz) return WHTQ_EUNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return WHTQ_EALIGN;
  for (int i = 0; i < 3; ++i)
    if ((c->k_stride[i] * esz & 15) || (c->v_stride[i] * esz & 15)) return WHTQ_EALIGN;
  if (int4) {
    if ((reinterpret_cast<uintptr_t>(c->k_scales) & 7u) || (reinterpret_cast<uintptr_t>(c->v_scales) & 7u)) return WHTQ_EALIGN;
    for (int i = 0; i < 2; ++i)
      if ((c->ks_stride[i] & 3) || (c->vs_stride[i] & 3)) return WHTQ_EALIGN;
    if (reinterpret_cast<uintptr_t>(c->sign_bits) & 3u) return WHTQ_EALIGN;
  }
  *out = KvCache{};
  out->k = {(uint8_t*)c->k, c->k_scales, c->k_stride[0] * esz, c->k_stride[1] * esz, c->k_stride[2] * esz,
            c->ks_stride[0], c->ks_stride[1]};
  out->v = {(uint8_t*)c->v, c->v_scales, c->v_stride[0] * esz, c->v_stride[1] * esz, c->v_stride[2] * esz,
            c->vs_stride[0], c->vs_stride[1]};
  out->signs = int4 ? c->sign_bits : nullptr;
  out->num_pages = c->num_pages;
  out->page_shift = shift;
  out->kv_heads = (int)c->kv_heads;
  return WHTQ_OK;
}

// rows of 16-bit head vectors: [token][head] strides in elements
bool kv_rows_valid(const int64_t* st) { return st && st[0] >= 0 && st[1] >= 0; }
bool kv_rows_aligned(const void* p, const int64_t* st) { return aligned16(p) && !((st[0] * 2) & 15) && !((st[1] * 2) & 15); }

KvRows kv_rows_of(const void* p, const int64_t* st) {
  return p ? KvRows{(const uint8_t*)p, st[0] * 2, st[1] * 2} : KvRows{};
}

// the rules of rotary positions for rows of dim values, but for alignment
whtq_status kv_rope_check(const whtq_rope* r, int64_t dim, int64_t tokens) {
  if (!r) return WHTQ_OK;
  if (r->rot_dim < 16 || r->rot_dim > dim || r->rot_dim % 16) return WHTQ_EINVAL;
  if (r->interleaved != 0 && r->interleaved != 1) return WHTQ_EINVAL;
  if (r->max_position < 1 || r->ld < r->rot_dim / 2) return WHTQ_EINVAL;
  if (tokens > 0 && (!r->cos || !r->sin || !r->positions)) return WHTQ_EINVAL;
  return WHTQ_OK;
}
bool kv_rope_aligned(const whtq_rope* r) {
  return !r || (aligned16(r->cos) && aligned16(r->sin) && !(r->ld & 3) && aligned4(r->positions));
}
KvTurn kv_turn_of(const whtq_rope* r) {
  if (!r) return KvTurn{};
  return KvTurn{r->cos, r->sin, r->positions, r->ld, r->max_position, r->rot_dim, r->interleaved};
}
// the type of norm weights; their rules, but for alignment
int kv_norm_dtype(const whtq_qk_norm* n) { return n->dtype & ~(WHTQ_CLEAR_Q | WHTQ_CLEAR_K); }
whtq_status kv_norm_check(const whtq_qk_norm* n) {
  if (!dt_valid(kv_norm_dtype(n)) || !std::isfinite(n->eps) || n->eps < 0.f) return WHTQ_EINVAL;
  if (n->q_head < 0 || n->k_head < 0) return WHTQ_EINVAL;
  return WHTQ_OK;
}
bool kv_norm_aligned(const whtq_qk_norm* n) {
  const int64_t esz = dt_bytes(kv_norm_dtype(n));
  return aligned16(n->q) && aligned16(n->k) && !(n->q_head * esz & 15) && !(n->k_head * esz & 15);
}
KvNorm kv_norm_of(const whtq_qk_norm* n) {
  const int64_t esz = dt_bytes(kv_norm_dtype(n));
  return KvNorm{{(const uint8_t*)n->q, n->q_head * esz}, {(const uint8_t*)n->k, n->k_head * esz}, kv_norm_dtype(n), n->eps};
}

// how an attention call runs: which kernel, and over how many blocks the keys of a row are split
struct KvPlan {
  bool step;
  int nq, blocks, rows, waves, splits;
  int64_t grid, parts, bytes;  // parts: partial rows kept
};

KvPlan kv_plan(const whtq_kv_cache* c, int64_t q_tokens, int64_t heads, int64_t seqs, int64_t max_q, int64_t max_kv,
               int64_t window, int64_t sinks, int cus) {
  KvPlan p{};
  // sinks and window, and a tile's rounding of each: the keys of a step, whatever the length (without sinks the
  // step's blocks are planned for max_kv, as they were)
  if (sinks > 0) max_kv = std::min(max_kv, std::min(window, kMost) + std::min(sinks, kMost) + max_q + 128);
  const int64_t group = heads / c->kv_heads, kvh = c->kv_heads;
  const bool int4 = c->format == WHTQ_KV_INT4;
  p.splits = 1;
  // Figures here are of bf16 rows, 32 heads on 8 of 128 unless said: a call in a
  // captured graph of calls on caches in turn, all of one machine.  The step
  // kernel reads an INT4 row once for up to 32 rows (32 sequences of 1000 to
  // 1500 keys, 4 tokens each: 19 us against the chunk kernel's 55, 8 tokens: 54
  // against 59; under a window of 700 with 4 sinks 18 and 42, 41 and 43) and
  // shares ragged sequences evenly (64 of 17 to 8191 keys, 16-bit pages, 2 tokens
  // each: 110 us against 126, 4 tokens: 113 with either).  With 17 to 32 rows of
  // 16-bit pages it would hold 255 + 132 registers: 41 us against the chunk
  // kernel's 33 (128 sequences of 1000 to 1500 keys, 32 heads on one).
  p.step = max_q * group <= (int4 ? 32 : 16);
  if (p.step) {
    p.nq = max_q * group <= 16 ? 1 : 2;
    p.rows = (int)(max_q * group);
    // A block of 8 waves takes a whole sequence, which saves the joining
    // kernel, when every block has a CU at once and its sequence is short, the
    // shorter the fewer blocks there are.  One token, 16-bit pages (a unit is
    // 256 keys), whole against shared, us: 64 keys 5.5 and 7.3, 256 keys 8.6 and
    // 9.7; 32 sequences (256 blocks) of 1024 keys 28.8 and 32.8; 16 of 512 keys
    // 14.2 and 16.3; but 4 of 512 keys 11.1 and 10.5, 64 of 256 keys 22.4 and 19.7.
    const int64_t unit = kv_step_unit((int)c->dim, int4, true), shared = kv_step_unit((int)c->dim, int4, false);
    if (p.nq == 1 && seqs * kvh <= cus && max_kv <= std::max<int64_t>(1, 4 * seqs * kvh / cus) * unit) {
      p.grid = seqs * kvh;
      return p;
    }
    const int64_t want = 2 * (int64_t)cus;
    const int64_t most = seqs * ((std::max<int64_t>(max_kv, 1) + shared - 1) / shared + 1);
    p.blocks = (int)std::max<int64_t>(1, std::min((want + kvh - 1) / kvh, most));
    p.grid = p.blocks * kvh;
    p.parts = (p.blocks + seqs) * kvh * p.rows;
  } else {
    // INT4 tiles are unpacked once a block: blocks of 8 waves halve that work
    // where there are rows for them (64 heads on 8, 512 tokens over 20000 keys:
    // 370 us against 412 with 4 waves; 40 tokens: 65 against 61).  16-bit tiles
    // cost a copy, and blocks of 4 waves wait for fewer others.
    p.waves = int4 && max_q * group > 128 ? 8 : 4;
    const int64_t rows = 32 * p.waves;
    // Blocks at work at a time, as a CU holds them with 16-bit pages.  INT4 blocks
    // of 4 waves need more: 2 are held at 64 dims and, with fp16 rows, 1 at 128
    // dims.  Counting those instead helps as often as it hurts, because blocks
    // that sequences do not fill are not counted either (INT4, fp16 rows, 128
    // dims: 12 x 8 rows on 8 key heads over 33000 keys 69 -> 56 us, 100 rows on
    // 32 over 4000 51 -> 40, but 24 sequences of 16 x 4 rows on 8 over 4000 154
    // -> 189; 64 dims: the last 81 -> 70, 4 sequences of 100 rows on 32 63 -> 69).
    const int64_t slots = (p.waves == 8 ? 1 : c->dim == 64 ? 3 : 2) * (int64_t)cus;
    // (as if sequences filled their tiles: many short chunks split more, which
    // evens out ragged lengths: 64 sequences of 17 to 8191 keys, 16-bit pages, 2
    // tokens each, 124 us against 180 counting a tile for each; 128 of 1000 to
    // 1500: 159 and 127)
    const int64_t blocks = (q_tokens * group + rows - 1) / rows * kvh;
    const int64_t keys = window > 0 ? std::min(max_kv, std::min(window, kMost) + std::min(sinks, kMost) + rows / group + 64) : max_kv;
    // split the keys of a block's rows where that shortens the longest chain
    // of tiles a slot works off; the joining kernel costs about 8 tiles' time
    // (16-bit pages, 512 tokens over 33000 keys: 303 us against 661 unsplit and
    // 314 in 16; 64 over 8000: 32 against 172 and 33)
    const int64_t tiles = (keys + 63) / 64;
    int64_t best = (blocks + slots - 1) / slots * tiles, splits = 1;
    const bool joins = q_tokens * heads * (c->dim / 8) <= kLaunchThreads;  // the joining kernel's threads
    for (int64_t n = 2; joins && n <= 64 && 4 * n <= tiles; ++n) {
      const int64_t cost = (blocks * n + slots - 1) / slots * ((tiles + n - 1) / n) + 8;
      if (cost < best) best = cost, splits = n;
    }
    p.splits = (int)splits;
    p.grid = (q_tokens * group / rows + seqs) * kvh * splits;
    if (splits > 1) p.parts = splits * q_tokens * heads;
  }
  if (p.parts) p.bytes = (p.parts * (c->dim + 2) * 4 + (p.step ? seqs * 8 : 0) + 15) / 16 * 16;
  return p;
}

whtq_status kv_attn_sizes(const whtq_kv_cache* c, int64_t q_tokens, int64_t heads, int64_t seqs, int64_t max_q,
                          int64_t max_kv) {
  if (q_tokens < 0 || seqs < 0 || heads < 1 || max_q < 0 || max_kv < 0 || heads % c->kv_heads) return WHTQ_EINVAL;
  if (q_tokens > kMost || seqs > kMost || heads > 65535 || max_q > kMost || max_kv > kMost) return WHTQ_EUNSUPPORTED;
  if (q_tokens > 0 && seqs > 0 && max_q < 1) return WHTQ_EINVAL;  // no row would have a place
  if ((q_tokens + seqs) * (heads / c->kv_heads) > kMost) return WHTQ_EUNSUPPORTED;  // rows of a head: 32-bit
  return WHTQ_OK;
}

int kv_cus() {
  int dev = 0;
  (void)hipGetDevice(&dev);
  return device_cu_count(dev);
}

}  // namespace

extern "C" {

whtq_status kv_append(const whtq_kv_cache* cache, const void* k, const int64_t* k_stride, const void* v,
                      const int64_t* v_stride, whtq_dtype dtype, int64_t tokens, const int64_t* slots,
                      const whtq_rope* rope, const void* q, const int64_t* q_stride, int64_t heads, void* q_out,
                      const int64_t* q_out_stride, void* stream) {
  return kv_append_norm(cache, k, k_stride, v, v_stride, dtype, tokens, slots, nullptr, rope, q, q_stride, heads, q_out,
                        q_out_stride, stream);
}

whtq_status kv_append_norm(const whtq_kv_cache* cache, const void* k, const int64_t* k_stride, const void* v,
                           const int64_t* v_stride, whtq_dtype dtype, int64_t tokens, const int64_t* slots,
                           const whtq_qk_norm* norm, const whtq_rope* rope, const void* q, const int64_t* q_stride,
                           int64_t heads, void* q_out, const int64_t* q_out_stride, void* stream) {
  KvCache c;
  whtq_status st = kv_check(cache, &c);
  if (st != WHTQ_OK) return st;
  if (!kv_dtype(dtype) || tokens < 0) return WHTQ_EINVAL;
  if (cache->format == WHTQ_KV_DENSE && dtype != cache->dtype) return WHTQ_EINVAL;
  if (!kv_rows_valid(k_stride) || !kv_rows_valid(v_stride)) return WHTQ_EINVAL;
  if (tokens > 0 && (!k || !v || !slots)) return WHTQ_EINVAL;
  if (q && (heads < 1 || !q_out || !kv_rows_valid(q_stride) || !kv_rows_valid(q_out_stride))) return WHTQ_EINVAL;
  if (q && q == q_out && (q_stride[0] != q_out_stride[0] || q_stride[1] != q_out_stride[1])) return WHTQ_EINVAL;
  st = kv_rope_check(rope, cache->dim, tokens);
  if (st == WHTQ_OK && norm) st = kv_norm_check(norm);
  if (st != WHTQ_OK) return st;
  if (norm && norm->q && !q) return WHTQ_EINVAL;
  if (tokens > kMost || (q && heads > 65535)) return WHTQ_EUNSUPPORTED;
  if (!kv_rows_aligned(k, k_stride) || !kv_rows_aligned(v, v_stride)) return WHTQ_EALIGN;
  if (q && (!kv_rows_aligned(q, q_stride) || !kv_rows_aligned(q_out, q_out_stride))) return WHTQ_EALIGN;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return WHTQ_EALIGN;
  if (!kv_rope_aligned(rope) || (norm && !kv_norm_aligned(norm))) return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const bool int4 = cache->format == WHTQ_KV_INT4;
  const int64_t capacity = cache->num_pages * cache->page_size;
  const KvNorm n = norm ? kv_norm_of(norm) : KvNorm{};
  QkForwardArgs a{};
  a.f[0] = {kv_rows_of(k, k_stride), {}, c.k, n.k, rope != nullptr, {}, 0, 0};
  a.f[1] = {kv_rows_of(v, v_stride), {}, c.v, {}, false, {}, 0, 0};
  if (q) a.f[2] = {kv_rows_of(q, q_stride), kv_rows_of(q_out, q_out_stride), {}, n.q, rope != nullptr, {}, 0, 0, norm && (norm->dtype & WHTQ_CLEAR_Q)};
  a.c = c;
  a.slots = slots;
  a.capacity = capacity;
  a.turn = kv_turn_of(rope);
  a.dt = n.dt;
  a.eps = n.eps;
  return hip_status(launch_qk_norm(a, {c.kv_heads, c.kv_heads, q ? (int)heads : 0}, tokens, (int)cache->dim, dtype, int4,
                                   (hipStream_t)stream));
}

whtq_status kv_gather(const whtq_kv_cache* cache, int64_t tokens, const int64_t* slots, void* k_out,
                      const int64_t* k_stride, void* v_out, const int64_t* v_stride, whtq_dtype dtype,
                      void* stream) {
  KvCache c;
  whtq_status st = kv_check(cache, &c);
  if (st != WHTQ_OK) return st;
  if (!kv_dtype(dtype) || tokens < 0) return WHTQ_EINVAL;
  if (cache->format == WHTQ_KV_DENSE && dtype != cache->dtype) return WHTQ_EINVAL;
  if ((k_out && !kv_rows_valid(k_stride)) || (v_out && !kv_rows_valid(v_stride))) return WHTQ_EINVAL;
  if (tokens > 0 && ((!k_out && !v_out) || !slots)) return WHTQ_EINVAL;
  if (tokens > kMost) return WHTQ_EUNSUPPORTED;
  if ((k_out && !kv_rows_aligned(k_out, k_stride)) || (v_out && !kv_rows_aligned(v_out, v_stride))) return WHTQ_EALIGN;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  return hip_status(launch_kv_gather(c, (int)cache->dim, dtype, cache->format == WHTQ_KV_INT4, tokens, slots,
                                     cache->num_pages * cache->page_size, k_out, k_stride, v_out, v_stride,
                                     (hipStream_t)stream));
}

int64_t kv_attention_workspace_bytes(const whtq_kv_cache* cache, int64_t q_tokens, int64_t heads, int64_t seqs,
                                     int64_t max_q_len, int64_t max_kv_len, int64_t window) {
  return kv_attention_sinks_workspace_bytes(cache, q_tokens, heads, seqs, max_q_len, max_kv_len, window, 0);
}

int64_t kv_attention_sinks_workspace_bytes(const whtq_kv_cache* cache, int64_t q_tokens, int64_t heads, int64_t seqs,
                                           int64_t max_q_len, int64_t max_kv_len, int64_t window, int64_t sinks) {
  KvCache c;
  if (kv_check(cache, &c) != WHTQ_OK) return -1;
  if (kv_attn_sizes(cache, q_tokens, heads, seqs, max_q_len, max_kv_len) != WHTQ_OK) return -1;
  if (window < 0 || sinks < 0 || need_device() != WHTQ_OK) return -1;
  if (q_tokens == 0 || seqs == 0) return 0;
  return kv_plan(cache, q_tokens, heads, seqs, max_q_len, max_kv_len, window, window > 0 ? sinks : 0, kv_cus()).bytes;
}

whtq_status kv_attention(const whtq_kv_cache* cache, const void* q, const int64_t* q_stride, whtq_dtype dtype,
                         int64_t q_tokens, int64_t heads, int64_t seqs, const int32_t* q_start,
                         const int32_t* kv_len, const int32_t* block_table, int64_t table_stride,
                         int64_t table_width, int64_t max_q_len, int64_t max_kv_len, float scale, int causal,
                         int64_t window, void* out, const int64_t* out_stride, float* lse, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  return kv_attention_sinks(cache, q, q_stride, dtype, q_tokens, heads, seqs, q_start, kv_len, block_table, table_stride,
                            table_width, max_q_len, max_kv_len, scale, causal, window, 0, out, out_stride, lse, workspace,
                            workspace_bytes, stream);
}

whtq_status kv_attention_sinks(const whtq_kv_cache* cache, const void* q, const int64_t* q_stride, whtq_dtype dtype,
                               int64_t q_tokens, int64_t heads, int64_t seqs, const int32_t* q_start,
                               const int32_t* kv_len, const int32_t* block_table, int64_t table_stride,
                               int64_t table_width, int64_t max_q_len, int64_t max_kv_len, float scale, int causal,
                               int64_t window, int64_t sinks, void* out, const int64_t* out_stride, float* lse,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  KvAttnArgs a{};
  whtq_status st = kv_check(cache, &a.c);
  if (st != WHTQ_OK) return st;
  st = kv_attn_sizes(cache, q_tokens, heads, seqs, max_q_len, max_kv_len);
  if (st != WHTQ_OK) return st;
  if (!kv_dtype(dtype) || (cache->format == WHTQ_KV_DENSE && dtype != cache->dtype)) return WHTQ_EINVAL;
  if ((causal != 0 && causal != 1) || window < 0 || sinks < 0 || !std::isfinite(scale) || workspace_bytes < 0) return WHTQ_EINVAL;
  if (table_width < 0 || table_stride < table_width) return WHTQ_EINVAL;
  if (!kv_rows_valid(q_stride) || !kv_rows_valid(out_stride)) return WHTQ_EINVAL;
  const bool any = q_tokens > 0 && seqs > 0;
  if (any && (!q || !out || !q_start || !kv_len || (table_width > 0 && !block_table))) return WHTQ_EINVAL;
  if (any && q == out) return WHTQ_EINVAL;
  if (table_width > kMost) return WHTQ_EUNSUPPORTED;
  if (!kv_rows_aligned(q, q_stride) || !kv_rows_aligned(out, out_stride) || !aligned16(workspace)) return WHTQ_EALIGN;
  if (!aligned4(q_start) || !aligned4(kv_len) || !aligned4(block_table) || !aligned4(lse)) return WHTQ_EALIGN;
  if (!any) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  if (window == 0) sinks = 0;  // every key is seen
  const KvPlan p = kv_plan(cache, q_tokens, heads, seqs, max_q_len, max_kv_len, window, sinks, kv_cus());
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return WHTQ_EINVAL;
  if (p.grid > INT32_MAX) return WHTQ_EUNSUPPORTED;
  a.q = (const uint8_t*)q;
  a.out = (uint8_t*)out;
  a.q_tok = q_stride[0] * 2;
  a.q_head = q_stride[1] * 2;
  a.o_tok = out_stride[0] * 2;
  a.o_head = out_stride[1] * 2;
  a.lse = lse;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.table = block_table;
  a.table_stride = table_stride;
  a.table_width = (int)table_width;
  a.q_tokens = q_tokens;
  a.heads = (int)heads;
  a.group = (int)(heads / cache->kv_heads);
  a.seqs = (int)seqs;
  a.causal = causal;
  a.window = (int)std::min(window, kMost);
  a.sinks = (int)std::min(sinks, kMost);
  a.splits = p.splits;
  a.grid = (int)p.grid;
  a.scale = scale * 1.4426950408889634f;
  a.part_o = (float*)workspace;
  a.part_ml = a.part_o + p.parts * cache->dim;
  a.reach = (int*)(a.part_ml + 2 * p.parts);
  a.blocks = p.blocks;
  a.rows = p.rows;
  const bool int4 = cache->format == WHTQ_KV_INT4;
  const hipStream_t s = (hipStream_t)stream;
  const int dim = (int)cache->dim;
  hipError_t e = p.step ? launch_kv_step(a, dim, dtype, int4, p.nq, s) : launch_kv_chunk(a, dim, dtype, int4, p.waves, s);
  if (e == hipSuccess && !p.step && p.splits > 1) e = launch_kv_join(a, dim, dtype, int4, s);
  return hip_status(e);
}

}  // extern "C"

// ---------------------------------------------------------------- norms and positions of dense rows

namespace {

// one side of a call; rows: in and out (x, y) or, backward, x, dy and dx
whtq_status qk_side(const void* x, const int64_t* xs, const void* a, const int64_t* as, const void* b, const int64_t* bs,
                    bool back, int64_t heads, int64_t tokens, const void* w) {
  if (heads == 0) return x || a || b || w ? WHTQ_EINVAL : WHTQ_OK;
  if (!w || !kv_rows_valid(xs) || !kv_rows_valid(as) || (back && !kv_rows_valid(bs))) return WHTQ_EINVAL;
  if (tokens > 0 && (!x || !a || (back && !b))) return WHTQ_EINVAL;
  auto alias = [](const void* p, const int64_t* ps, const void* r, const int64_t* rs) {
    return p && p == r && (ps[0] != rs[0] || ps[1] != rs[1]);
  };
  if (back ? alias(x, xs, b, bs) || alias(a, as, b, bs) : alias(x, xs, a, as)) return WHTQ_EINVAL;
  return WHTQ_OK;
}
whtq_status qk_check(int64_t heads, int64_t kv_heads, int dtype, int64_t dim, int64_t tokens, const whtq_qk_norm* norm,
                     const whtq_rope* rope) {
  if (heads < 0 || kv_heads < 0 || heads + kv_heads < 1 || tokens < 0 || !norm || !kv_dtype(dtype) || dim < 1) return WHTQ_EINVAL;
  whtq_status st = kv_norm_check(norm);
  if (st == WHTQ_OK) st = kv_rope_check(rope, dim, tokens);
  if (st != WHTQ_OK) return st;
  if ((dim != 64 && dim != 128) || tokens > kMost || heads > 65535 || kv_heads > 65535) return WHTQ_EUNSUPPORTED;
  return WHTQ_OK;
}
int qk_classes(int64_t heads, int64_t stride) { return heads == 0 ? 0 : stride ? (int)heads : 1; }
bool qk_aligned(const void* p, const int64_t* st) { return !p || kv_rows_aligned(p, st); }

}  // namespace

extern "C" {

whtq_status qk_norm_rope(const void* q, const int64_t* q_stride, int64_t heads, const void* k, const int64_t* k_stride,
                         int64_t kv_heads, whtq_dtype dtype, int64_t dim, int64_t tokens, const whtq_qk_norm* norm,
                         const whtq_rope* rope, void* q_out, const int64_t* q_out_stride, void* k_out,
                         const int64_t* k_out_stride, void* stream) {
  whtq_status st = qk_check(heads, kv_heads, dtype, dim, tokens, norm, rope);
  if (st == WHTQ_OK) st = qk_side(q, q_stride, q_out, q_out_stride, nullptr, nullptr, false, heads, tokens, norm->q);
  if (st == WHTQ_OK) st = qk_side(k, k_stride, k_out, k_out_stride, nullptr, nullptr, false, kv_heads, tokens, norm->k);
  if (st != WHTQ_OK) return st;
  if (!qk_aligned(q, q_stride) || !qk_aligned(q_out, q_out_stride) || !qk_aligned(k, k_stride) ||
      !qk_aligned(k_out, k_out_stride) || !kv_norm_aligned(norm) || !kv_rope_aligned(rope))
    return WHTQ_EALIGN;
  if (tokens == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const KvNorm n = kv_norm_of(norm);
  QkForwardArgs a{};
  if (heads) a.f[0] = {kv_rows_of(q, q_stride), kv_rows_of(q_out, q_out_stride), {}, n.q, rope != nullptr, {}, 0, 0, (norm->dtype & WHTQ_CLEAR_Q) != 0};
  if (kv_heads) a.f[1] = {kv_rows_of(k, k_stride), kv_rows_of(k_out, k_out_stride), {}, n.k, rope != nullptr, {}, 0, 0, (norm->dtype & WHTQ_CLEAR_K) != 0};
  a.turn = kv_turn_of(rope);
  a.dt = n.dt;
  a.eps = n.eps;
  return hip_status(launch_qk_norm(a, {(int)heads, (int)kv_heads, 0}, tokens, (int)dim, dtype, false, (hipStream_t)stream));
}

int64_t qk_norm_rope_backward_workspace_bytes(int64_t heads, int64_t kv_heads, int64_t dim, int64_t tokens,
                                              const whtq_qk_norm* norm) {
  if (qk_check(heads, kv_heads, WHTQ_BF16, dim, tokens, norm, nullptr) != WHTQ_OK || need_device() != WHTQ_OK) return -1;
  QkArgs a{};
  a.tokens = tokens;
  a.q.heads = (int)heads;
  a.k.heads = (int)kv_heads;
  a.q.classes = qk_classes(heads, norm->q_head);
  a.k.classes = qk_classes(kv_heads, norm->k_head);
  return qk_norm_split(a, (int)dim, kv_cus()) * dim * 4;
}

whtq_status qk_norm_rope_backward(const void* dq_out, const int64_t* dq_out_stride, const void* q,
                                  const int64_t* q_stride, int64_t heads, const void* dk_out,
                                  const int64_t* dk_out_stride, const void* k, const int64_t* k_stride, int64_t kv_heads,
                                  whtq_dtype dtype, int64_t dim, int64_t tokens, const whtq_qk_norm* norm,
                                  const whtq_rope* rope, void* dq, const int64_t* dq_stride, void* dk,
                                  const int64_t* dk_stride, float* dq_norm, float* dk_norm, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  whtq_status st = qk_check(heads, kv_heads, dtype, dim, tokens, norm, rope);
  if (st == WHTQ_OK) st = qk_side(q, q_stride, dq_out, dq_out_stride, dq, dq_stride, true, heads, tokens, norm->q);
  if (st == WHTQ_OK) st = qk_side(k, k_stride, dk_out, dk_out_stride, dk, dk_stride, true, kv_heads, tokens, norm->k);
  if (st != WHTQ_OK) return st;
  if ((heads > 0) != (dq_norm != nullptr) || (kv_heads > 0) != (dk_norm != nullptr) || workspace_bytes < 0) return WHTQ_EINVAL;
  if (!qk_aligned(q, q_stride) || !qk_aligned(dq_out, dq_out_stride) || !qk_aligned(dq, dq_stride) ||
      !qk_aligned(k, k_stride) || !qk_aligned(dk_out, dk_out_stride) || !qk_aligned(dk, dk_stride) ||
      !kv_norm_aligned(norm) || !kv_rope_aligned(rope) || !aligned4(dq_norm) || !aligned4(dk_norm) || !aligned16(workspace))
    return WHTQ_EALIGN;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const KvNorm n = kv_norm_of(norm);
  QkArgs a{};
  a.q = {kv_rows_of(q, q_stride), kv_rows_of(dq_out, dq_out_stride), kv_rows_of(dq, dq_stride), n.q, dq_norm, (int)heads,
         qk_classes(heads, norm->q_head), 0, (norm->dtype & WHTQ_CLEAR_Q) != 0};
  a.k = {kv_rows_of(k, k_stride), kv_rows_of(dk_out, dk_out_stride), kv_rows_of(dk, dk_stride), n.k, dk_norm, (int)kv_heads,
         qk_classes(kv_heads, norm->k_head), 0, (norm->dtype & WHTQ_CLEAR_K) != 0};
  a.turn = kv_turn_of(rope);
  a.tokens = tokens;
  a.dt = n.dt;
  a.eps = n.eps;
  const int64_t bytes = qk_norm_split(a, (int)dim, kv_cus()) * dim * 4;
  if (bytes > 0 && (!workspace || workspace_bytes < bytes)) return WHTQ_EINVAL;
  a.part = bytes > 0 ? (float*)workspace : nullptr;
  return hip_status(launch_qk_norm_back(a, (int)dim, dtype, (hipStream_t)stream));
}

}  // extern "C"

// ---------------------------------------------------------------- log probabilities

namespace {

static_assert(LP_MOST_TOP == WHTQ_TOP_MOST, "room for the likeliest tokens of a row");

whtq_status lp_check(int dtype, int64_t rows, int64_t vocab, int64_t ld, float scale) {
  if (!dt_valid(dtype) || rows < 0 || vocab < 1 || ld < vocab) return WHTQ_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return WHTQ_EINVAL;
  if (rows > kMost || vocab > LP_MOST_VOCAB) return WHTQ_EUNSUPPORTED;
  return WHTQ_OK;
}
bool lp_aligned(const void* p, int dtype) { return !(reinterpret_cast<uintptr_t>(p) & (dt_bytes(dtype) - 1)); }
bool aligned8(const void* p) { return !(reinterpret_cast<uintptr_t>(p) & 7u); }

// How a call runs: blocks of a row, groups whose maxima are kept, and the bytes of both.
struct LpPlan {
  int splits, width, groups;
  int64_t parts, bytes;
};
LpPlan lp_plan(int64_t rows, int64_t vocab, int64_t top, int cus) {
  LpPlan p{};
  const int64_t chunks = (vocab + 7 + LP_CHUNK - 1) / LP_CHUNK;
  // A block for each row saves the second kernel and its launch, which is 2.5 us of a call.  It is taken where rows are
  // short (64 chunks), by what calls take one after another from Python.  bf16, 5 tokens, us a call so, one block
  // against the best of 2 to 16: 1 row of 8192 13.0 and 15.5, of 32000 13.0 and 15.4, of 32768 (65 chunks) 13.0 and
  // 15.3; 64 rows of 16384 13.1 and 15.4, of 32000 17.3 and 17.4; but 300 of 32000 18.8 and 17.3.  Between captured
  // calls the second kernel costs next to nothing, and from 16384 logits on several blocks are the faster: 1 row of 8192
  // 6.9 and 7.5, of 16384 8.4 and 7.5, of 32000 12.8 and 7.9; 64 rows of 32000 17.2 and 10.1, 300 18.7 and 15.2.  fp32
  // rows are within 1.5 us of these times, but for 300 over several blocks (16384: 13.5 against one block's 11.9; 32000:
  // 17.5 against 18.2).
  // It is taken too where there are enough rows (700 rows of 50257: 22.5 and 24.6, 1000 of 131072: 51.2 and 54.5; but
  // 600 of 131072: 41.5 and 37.3, 300: 33.3 and 25.9).  Otherwise as many blocks as the machine holds, each of 4 chunks
  // a wave or more (64 rows of 131072: 15.0 with 16 blocks a row, 15.1 with 32).
  p.splits = chunks <= 64 || 2 * rows >= 5 * (int64_t)cus
                 ? 1
                 : (int)std::max<int64_t>(1, std::min(8 * (int64_t)cus / std::max<int64_t>(rows, 1), chunks / 16));
  if (top) {
    // groups enough that the last one's maximum leaves few candidates, large enough that their maxima are few bytes: at
    // most 512 up to 262144 logits, but for a row of 4096, 32768 or 262144 that does not begin at 16 bytes (one more, and
    // they are picked from in pairs).  A row over several blocks has more than 64 chunks, each a group.
    p.width = p.splits > 1 || vocab > 32768 ? LP_CHUNK : vocab <= 4096 ? 8 : 64;
    p.groups = (int)((vocab + 7 + p.width - 1) / p.width);  // (7: a row may begin inside 16 bytes)
  }
  // a block that has all of its row keeps both to itself
  if (p.splits > 1) {
    p.parts = rows * p.splits * 3;
    p.bytes = (p.parts + rows * p.groups) * 4;
  }
  return p;
}

}  // namespace

extern "C" {

int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top) {
  if (lp_check(WHTQ_F32, rows, vocab, vocab, 1.f) != WHTQ_OK || top < 0 || top > std::min<int64_t>(vocab, LP_MOST_TOP)) return -1;
  if (need_device() != WHTQ_OK) return -1;
  return lp_plan(rows, vocab, top, kv_cus()).bytes;
}

whtq_status token_logprobs(const void* logits, whtq_dtype dtype, int64_t rows, int64_t vocab, int64_t ld, float scale,
                           const int64_t* targets, float* logprob, float* lse, float* row_ref, float* row_sum,
                           float* entropy, int64_t top, float* top_logprob, int64_t* top_id, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  whtq_status st = lp_check(dtype, rows, vocab, ld, scale);
  if (st != WHTQ_OK) return st;
  if (top < 0 || top > vocab || workspace_bytes < 0) return WHTQ_EINVAL;
  if (top > WHTQ_TOP_MOST) return WHTQ_EUNSUPPORTED;
  if (rows > 0 && (!logits || (targets != nullptr) != (logprob != nullptr) || (row_ref != nullptr) != (row_sum != nullptr) || (top > 0 && (!top_logprob || !top_id)))) return WHTQ_EINVAL;
  if (!lp_aligned(logits, dtype) || !aligned8(targets) || !aligned8(top_id) || !aligned4(logprob) || !aligned4(lse) ||
      !aligned4(row_ref) || !aligned4(row_sum) || !aligned4(entropy) || !aligned4(top_logprob) || !aligned16(workspace))
    return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  const LpPlan p = lp_plan(rows, vocab, top, kv_cus());
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return WHTQ_EINVAL;
  LpArgs a{};
  a.x = (const uint8_t*)logits;
  a.ld = ld * dt_bytes(dtype);
  a.rows = rows;
  a.vocab = (int)vocab;
  a.scale = scale;
  a.targets = targets;
  a.logprob = logprob;
  a.lse = lse;
  a.ref = row_ref;
  a.sum = row_sum;
  a.entropy = entropy;
  a.top = (int)top;
  a.top_logprob = top_logprob;
  a.top_id = top_id;
  a.splits = p.splits;
  a.width = p.width;
  a.groups = p.groups;
  a.part = (float*)workspace;
  a.best = (uint32_t*)(a.part + p.parts);
  return hip_status(launch_lp(a, dtype, (hipStream_t)stream));
}

whtq_status token_logprobs_backward(const void* logits, whtq_dtype dtype, int64_t rows, int64_t vocab, int64_t ld,
                                    float scale, const int64_t* targets, const float* row_ref, const float* row_sum,
                                    const float* entropy, const float* dlogprob, const float* dentropy, void* dlogits,
                                    int64_t ldd, void* stream) {
  whtq_status st = lp_check(dtype, rows, vocab, ld, scale);
  if (st != WHTQ_OK) return st;
  if (ldd < vocab || (logits && logits == dlogits && ld != ldd)) return WHTQ_EINVAL;
  if (rows > 0 && (!logits || !dlogits || !row_ref || !row_sum || (!dlogprob && !dentropy) || (dlogprob && !targets) || (dentropy && !entropy)))
    return WHTQ_EINVAL;
  if (!lp_aligned(logits, dtype) || !lp_aligned(dlogits, dtype) || !aligned8(targets) || !aligned4(row_ref) ||
      !aligned4(row_sum) || !aligned4(entropy) || !aligned4(dlogprob) || !aligned4(dentropy))
    return WHTQ_EALIGN;
  if (rows == 0) return WHTQ_OK;
  st = need_device();
  if (st != WHTQ_OK) return st;
  LpGradArgs a{};
  a.x = (const uint8_t*)logits;
  a.dx = (uint8_t*)dlogits;
  a.ld = ld * dt_bytes(dtype);
  a.ldd = ldd * dt_bytes(dtype);
  a.rows = rows;
  a.vocab = (int)vocab;
  a.scale = scale;
  a.targets = targets;
  a.ref = row_ref;
  a.sum = row_sum;
  a.entropy = entropy;
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  return hip_status(launch_lp_grad(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
