// rs_ops.cu -- the C ABI of the layer norm and of the products in 8 bits (include/rs.h):
// argument checks, the layout of the caller's scratch and the launch sequences.
#include <cstdint>

#include <cuda_runtime.h>

#include "rs.h"
#include "rs_ops.h"

namespace {

constexpr int kMaxDim = 1 << 27;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == RS_FP32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == RS_BF16 || dtype == RS_FP16 || dtype == RS_FP32; }
bool dim_ok(int n) { return n >= 1 && n < kMaxDim; }
uint64_t up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }
uint64_t scale_bytes(int64_t rows, int64_t K) {
  return static_cast<uint64_t>((rows + 127) / 128) * static_cast<uint64_t>((K + 511) / 512) * 512;
}

#define RS_TRY(expr)            \
  do {                          \
    const int _s = (expr);      \
    if (_s != RS_OK) return _s; \
  } while (0)
#define RS_CUDA(expr)             \
  do {                            \
    if ((expr) != cudaSuccess) {  \
      cudaGetLastError();         \
      return RS_ERR_CUDA;         \
    }                             \
  } while (0)

// A strided matrix of 16- or 32-bit elements: is every row a whole number of 16-byte vectors
// that starts on 16 bytes?
bool rows16(const void* p, int64_t ld, int width, int es) {
  return p == nullptr || (aligned(p, 16) && ld * es % 16 == 0 && static_cast<int64_t>(width) * es % 16 == 0);
}

// A quantised operand [rows, K].
int check_q(const void* q, int64_t ldq, const void* scales, int64_t K) {
  if (!q || !scales) return RS_ERR_NULL;
  if (ldq < K || ldq % 16 != 0) return RS_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(scales, 16)) return RS_ERR_ALIGN;
  return RS_OK;
}

int check_ws(const void* ws, uint64_t bytes, uint64_t need) {
  if (need == 0) return RS_OK;
  if (!ws) return RS_ERR_NULL;
  if (!aligned(ws, 256)) return RS_ERR_ALIGN;
  return bytes < need ? RS_ERR_NO_MEM : RS_OK;
}

int check_norm(const void* x, int64_t ldx, int M, int C, int dtype, const void* gamma,
               const void* beta, int param_dtype, float eps) {
  if (M < 0 || M >= kMaxDim || C < 1 || C > RS_MAX_LN_C || !float_type(dtype)) return RS_ERR_SHAPE;
  if (param_dtype != RS_FP32 && param_dtype != dtype) return RS_ERR_SHAPE;
  if (!(eps > 0.f) || ldx < C) return RS_ERR_SHAPE;
  if (M == 0) return RS_OK;
  if (!x) return RS_ERR_NULL;
  if (!aligned(x, elem_bytes(dtype)) || !aligned(gamma, elem_bytes(param_dtype)) ||
      !aligned(beta, elem_bytes(param_dtype)))
    return RS_ERR_ALIGN;
  return RS_OK;
}

rs::LnForward norm_args(const void* x, int64_t ldx, int M, int C, const void* gamma,
                        const void* beta, int param_dtype, float eps, float* stats) {
  rs::LnForward p{};
  p.x = x;
  p.ldx = ldx;
  p.M = M;
  p.C = C;
  p.gamma = gamma;
  p.beta = beta;
  p.p32 = param_dtype == RS_FP32;
  p.eps = eps;
  p.stats = reinterpret_cast<float2*>(stats);
  return p;
}

int gemm(rs::Fp8Gemm p, int out_dtype, cudaStream_t s, bool pdl, int debug_skip_kb = -1,
         unsigned long long timeout_ns = rs::kDefaultTimeoutNs) {
  int sms = 0;
  RS_TRY(rs::device_flag(&sms, &p.err));
  p.timeout_ns = timeout_ns;
  p.debug_skip_kb = debug_skip_kb;
  const int es = out_dtype == RS_E4M3 ? 1 : elem_bytes(out_dtype);
  p.direct = !(aligned(p.out, 16) && p.ldo * es % 16 == 0);
  p.rvec = p.resid != nullptr && aligned(p.resid, 16) && p.ldr * es % 16 == 0;
  p.kqo = (p.N + 511) / 512;
  return rs::launch_fp8_gemm(
      p, out_dtype == RS_BF16 ? rs::kOutBf16 : out_dtype == RS_FP32 ? rs::kOutFp32 : rs::kOutQ8, sms,
      s, pdl);
}

int check_gemm_dims(int M, int N, int K) {
  if (M < 0 || M >= kMaxDim || !dim_ok(N) || !dim_ok(K)) return RS_ERR_SHAPE;
  const int64_t tiles = (static_cast<int64_t>(M) / 128 + 1) * (static_cast<int64_t>(N) / 64 + 1);
  return tiles < (1 << 30) ? RS_OK : RS_ERR_SHAPE;
}

int check_epilogue(const void* bias, int gelu, const void* resid, int64_t ldr, int N, int es) {
  if (gelu != 0 && gelu != 1) return RS_ERR_SHAPE;
  if (!aligned(bias, 16)) return RS_ERR_ALIGN;
  if (resid != nullptr) {
    if (ldr < N) return RS_ERR_SHAPE;
    if (!aligned(resid, es)) return RS_ERR_ALIGN;
  }
  return RS_OK;
}

// Scratch of a quantised [rows, K] matrix: the rows, then the scale tiles.
struct QSpace {
  uint64_t ld, scales, bytes;
};
QSpace q_space(int64_t rows, int64_t K) {
  QSpace w;
  w.ld = up(K, 16);
  w.scales = up(static_cast<uint64_t>(rows) * w.ld, 256);
  w.bytes = up(w.scales + scale_bytes(rows, K), 256);
  return w;
}

}  // namespace

extern "C" {

int rs_ln_forward(const void* x, int64_t ldx, int M, int C, int dtype, const void* gamma,
                  const void* beta, int param_dtype, float eps, void* y, int64_t ldy,
                  float* stats, void* stream) {
  RS_TRY(check_norm(x, ldx, M, C, dtype, gamma, beta, param_dtype, eps));
  if (ldy < C) return RS_ERR_SHAPE;
  if (M == 0) return RS_OK;
  if (!y) return RS_ERR_NULL;
  const int es = elem_bytes(dtype);
  if (!aligned(y, es) || !aligned(stats, 8)) return RS_ERR_ALIGN;
  int sms = 0;
  RS_TRY(rs::device_sms(&sms));
  rs::LnForward p = norm_args(x, ldx, M, C, gamma, beta, param_dtype, eps, stats);
  p.y = y;
  p.ldy = ldy;
  const bool vec = rows16(x, ldx, C, es) && rows16(y, ldy, C, es) && aligned(gamma, 16) && aligned(beta, 16);
  RS_CUDA(rs::launch_ln_forward(p, dtype, vec, sms, static_cast<cudaStream_t>(stream)));
  return RS_OK;
}

int rs_ln_quantize(const void* x, int64_t ldx, int M, int C, int dtype, const void* gamma,
                   const void* beta, int param_dtype, float eps, void* q, int64_t ldq,
                   void* scales, float* stats, void* stream) {
  RS_TRY(check_norm(x, ldx, M, C, dtype, gamma, beta, param_dtype, eps));
  if (dtype == RS_FP32 || C % 8 != 0) return RS_ERR_SHAPE;
  if (M == 0) return RS_OK;
  RS_TRY(check_q(q, ldq, scales, C));
  if (!rows16(x, ldx, C, 2) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(stats, 8))
    return RS_ERR_ALIGN;
  int sms = 0;
  RS_TRY(rs::device_sms(&sms));
  rs::LnForward p = norm_args(x, ldx, M, C, gamma, beta, param_dtype, eps, stats);
  p.q = static_cast<uint8_t*>(q);
  p.ldq = ldq;
  p.scales = static_cast<uint8_t*>(scales);
  p.kq = (C + 511) / 512;
  RS_CUDA(rs::launch_ln_quantize(p, dtype, sms, static_cast<cudaStream_t>(stream)));
  return RS_OK;
}

uint64_t rs_ln_backward_ws_bytes(int M, int C) {
  if (M < 0 || M >= kMaxDim || C < 1 || C > RS_MAX_LN_C) return 0;
  if (rs::ln_backward_few(M, C)) return 0;
  int sms = 0;
  if (rs::device_sms(&sms) != RS_OK) return 0;
  const uint64_t blocks = M < sms ? (M > 0 ? M : 1) : sms;
  return up(blocks * 2 * static_cast<uint64_t>(C) * 4, 256);
}

int rs_ln_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* dres,
                   int64_t lddres, const float* stats, const void* gamma, int param_dtype, int M,
                   int C, int dtype, void* dx, int64_t lddx, float* dgamma, float* dbeta, void* ws,
                   uint64_t ws_bytes, void* stream) {
  RS_TRY(check_norm(x, ldx, M, C, dtype, gamma, nullptr, param_dtype, 1.f));
  if (lddy < C || (dres && lddres < C) || (dx && lddx < C)) return RS_ERR_SHAPE;
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return RS_ERR_ALIGN;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // sums over no rows
    if (dgamma) RS_CUDA(cudaMemsetAsync(dgamma, 0, static_cast<size_t>(C) * 4, s));
    if (dbeta) RS_CUDA(cudaMemsetAsync(dbeta, 0, static_cast<size_t>(C) * 4, s));
    return RS_OK;
  }
  if (!dy || !stats) return RS_ERR_NULL;
  const int es = elem_bytes(dtype);
  if (!aligned(dy, es) || !aligned(dres, es) || !aligned(dx, es) || !aligned(stats, 8))
    return RS_ERR_ALIGN;
  const bool sums = dgamma != nullptr || dbeta != nullptr;
  if (!sums && dx == nullptr) return RS_OK;
  int sms = 0;
  RS_TRY(rs::device_sms(&sms));
  if (sums) RS_TRY(check_ws(ws, ws_bytes, rs_ln_backward_ws_bytes(M, C)));
  rs::LnBackward p{};
  p.dy = dy;
  p.lddy = lddy;
  p.x = x;
  p.ldx = ldx;
  p.dres = dx ? dres : nullptr;
  p.lddres = lddres;
  p.stats = reinterpret_cast<const float2*>(stats);
  p.gamma = gamma;
  p.p32 = param_dtype == RS_FP32;
  p.M = M;
  p.C = C;
  p.dx = dx;
  p.lddx = lddx;
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  p.sums = sums;
  p.partials = static_cast<float*>(ws);
  const bool vec = rows16(dy, lddy, C, es) && rows16(x, ldx, C, es) &&
                   rows16(p.dres, lddres, C, es) && rows16(dx, lddx, C, es) && aligned(gamma, 16);
  RS_CUDA(rs::launch_ln_backward(p, dtype, vec, sms, s));
  return RS_OK;
}

uint64_t rs_fp8_scale_bytes(int rows, int K) {
  return rows < 0 || rows >= kMaxDim || !dim_ok(K) ? 0 : scale_bytes(rows, K);
}

uint64_t rs_fp8_quantize_ws_bytes(int rows, int K) {
  if (rows < 0 || rows >= kMaxDim || !dim_ok(K)) return 0;
  const uint64_t chunks = rows > 0 ? rs::quant_chunks(rows, K) : 1;
  return up(chunks * static_cast<uint64_t>(K) * 4, 256);
}

int rs_fp8_quantize(const void* x, int64_t ldx, int rows, int K, int dtype, void* q, int64_t ldq,
                    void* scales, void* qt, int64_t ldqt, void* scales_t, float* colsum, void* ws,
                    uint64_t ws_bytes, void* stream) {
  if (rows < 0 || rows >= kMaxDim || !dim_ok(K) || !float_type(dtype) || ldx < K) return RS_ERR_SHAPE;
  if (!aligned(colsum, 4)) return RS_ERR_ALIGN;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (colsum) RS_CUDA(cudaMemsetAsync(colsum, 0, static_cast<size_t>(K) * 4, s));
    return RS_OK;
  }
  if (colsum && !qt) return RS_ERR_NULL;
  if (!q && !qt) return RS_OK;
  if (!x) return RS_ERR_NULL;
  const int es = elem_bytes(dtype);
  if (!aligned(x, es)) return RS_ERR_ALIGN;
  if (q) RS_TRY(check_q(q, ldq, scales, K));
  if (qt) RS_TRY(check_q(qt, ldqt, scales_t, rows));
  if (colsum) RS_TRY(check_ws(ws, ws_bytes, rs_fp8_quantize_ws_bytes(rows, K)));
  rs::Quant p{};
  p.x = x;
  p.ldx = ldx;
  p.rows = rows;
  p.K = K;
  p.q = static_cast<uint8_t*>(q);
  p.ldq = ldq;
  p.scales = static_cast<uint8_t*>(scales);
  p.qt = static_cast<uint8_t*>(qt);
  p.ldqt = ldqt;
  p.scales_t = static_cast<uint8_t*>(scales_t);
  const bool direct = colsum && rs::quant_direct(rows);
  p.partials = direct ? colsum : colsum ? static_cast<float*>(ws) : nullptr;
  p.chunks = direct ? 1 : rs::quant_chunks(rows, K);
  const bool vec = aligned(x, 16) && ldx * es % 16 == 0 && K % 8 == 0;
  RS_CUDA(rs::launch_quantize(p, dtype, vec, s));
  if (colsum && !direct)
    RS_CUDA(rs::launch_col_reduce(p.partials, p.chunks, K, K, colsum, nullptr, s, true));
  return RS_OK;
}

static int fp8_gemm(const void* a, int64_t lda, const void* scales_a, const void* b, int64_t ldb,
                    const void* scales_b, int M, int N, int K, const void* bias, int gelu,
                    const void* resid, int64_t ldr, void* out, int64_t ldo, int out_dtype,
                    void* out_scales, cudaStream_t s, int debug_skip_kb,
                    unsigned long long timeout_ns) {
  RS_TRY(check_gemm_dims(M, N, K));
  if (out_dtype != RS_BF16 && out_dtype != RS_FP32 && out_dtype != RS_E4M3) return RS_ERR_SHAPE;
  const int es = out_dtype == RS_E4M3 ? 1 : elem_bytes(out_dtype);
  RS_TRY(check_epilogue(bias, gelu, resid, ldr, N, es));
  if (out_dtype == RS_E4M3 ? resid != nullptr : out_scales != nullptr) return RS_ERR_SHAPE;
  if (ldo < N) return RS_ERR_SHAPE;
  if (M == 0) return RS_OK;
  RS_TRY(check_q(a, lda, scales_a, K));
  RS_TRY(check_q(b, ldb, scales_b, K));
  if (out_dtype == RS_E4M3) {
    RS_TRY(check_q(out, ldo, out_scales, N));
  } else {
    if (!out) return RS_ERR_NULL;
    if (!aligned(out, es)) return RS_ERR_ALIGN;
  }
  rs::Fp8Gemm p{};
  p.a = a;
  p.lda = lda;
  p.sa = scales_a;
  p.b = b;
  p.ldb = ldb;
  p.sb = scales_b;
  p.M = M;
  p.N = N;
  p.K = K;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.gelu = gelu;
  p.resid = resid;
  p.ldr = ldr;
  p.out = out;
  p.ldo = ldo;
  p.out_scales = static_cast<uint8_t*>(out_scales);
  return gemm(p, out_dtype, s, false, debug_skip_kb, timeout_ns);
}

int rs_fp8_gemm(const void* a, int64_t lda, const void* scales_a, const void* b, int64_t ldb,
                const void* scales_b, int M, int N, int K, const void* bias, int gelu,
                const void* resid, int64_t ldr, void* out, int64_t ldo, int out_dtype,
                void* out_scales, void* stream) {
  return fp8_gemm(a, lda, scales_a, b, ldb, scales_b, M, N, K, bias, gelu, resid, ldr, out, ldo,
                  out_dtype, out_scales, static_cast<cudaStream_t>(stream), -1, rs::kDefaultTimeoutNs);
}

int rs_debug_fp8_skip_load(const void* a, int64_t lda, const void* scales_a, const void* b,
                           int64_t ldb, const void* scales_b, int M, int N, int K, void* out,
                           int64_t ldo, int out_dtype, void* out_scales, int skip_kblock,
                           int timeout_us, void* stream) {
  if (K < 1 || skip_kblock < 0 || skip_kblock >= (K - 1) / 128 + 1 || timeout_us < 1 ||
      timeout_us > 10000000)
    return RS_ERR_SHAPE;
  return fp8_gemm(a, lda, scales_a, b, ldb, scales_b, M, N, K, nullptr, 0, nullptr, 0, out, ldo,
                  out_dtype, out_scales, static_cast<cudaStream_t>(stream), skip_kblock,
                  static_cast<unsigned long long>(timeout_us) * 1000ull);
}

uint64_t rs_fp8_linear_ws_bytes(int M, int K) {
  if (M < 0 || M >= kMaxDim || !dim_ok(K) || rs::fp8_few_rows(M, 1 << 26, K)) return 0;
  return q_space(M, K).bytes;
}

static int fp8_linear(const void* x, int64_t ldx, int M, int K, int N, const void* wq, int64_t ldw,
                      const void* scales_w, const void* bias, int gelu, const void* resid,
                      int64_t ldr, void* out, int64_t ldo, void* ws, uint64_t ws_bytes,
                      cudaStream_t s, bool debug_skip, unsigned long long timeout_ns) {
  RS_TRY(check_gemm_dims(M, N, K));
  RS_TRY(check_epilogue(bias, gelu, resid, ldr, N, 2));
  if (ldx < K || ldo < N) return RS_ERR_SHAPE;
  if (M == 0) return RS_OK;
  if (!x || !out) return RS_ERR_NULL;
  if (!aligned(x, 2) || !aligned(out, 2)) return RS_ERR_ALIGN;
  RS_TRY(check_q(wq, ldw, scales_w, K));
  if (rs::fp8_few_rows(M, N, K)) {
    rs::Fp8Few f{};
    f.x = static_cast<const __nv_bfloat16*>(x);
    f.ldx = ldx;
    f.xvec = aligned(x, 16) && ldx % 8 == 0;
    f.M = M;
    f.N = N;
    f.K = K;
    f.w = wq;
    f.ldw = ldw;
    f.sw = scales_w;
    f.bias = static_cast<const __nv_bfloat16*>(bias);
    f.gelu = gelu;
    f.resid = static_cast<const __nv_bfloat16*>(resid);
    f.ldr = ldr;
    f.out = static_cast<__nv_bfloat16*>(out);
    f.ldo = ldo;
    f.timeout_ns = timeout_ns;
    f.debug_skip = debug_skip;
    int sms = 0;
    RS_TRY(rs::device_flag(&sms, &f.err));
    return rs::launch_fp8_few(f, sms, s);
  }
  RS_TRY(check_ws(ws, ws_bytes, rs_fp8_linear_ws_bytes(M, K)));
  const QSpace w = q_space(M, K);
  rs::Quant qp{};
  qp.x = x;
  qp.ldx = ldx;
  qp.rows = M;
  qp.K = K;
  qp.q = static_cast<uint8_t*>(ws);
  qp.ldq = static_cast<int64_t>(w.ld);
  qp.scales = qp.q + w.scales;
  qp.chunks = rs::quant_chunks(M, K);
  rs::Fp8Gemm p{};
  p.a = qp.q;
  p.lda = qp.ldq;
  p.sa = qp.scales;
  p.b = wq;
  p.ldb = ldw;
  p.sb = scales_w;
  p.M = M;
  p.N = N;
  p.K = K;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.gelu = gelu;
  p.resid = resid;
  p.ldr = ldr;
  p.out = out;
  p.ldo = ldo;
  RS_CUDA(rs::launch_quantize(qp, RS_BF16, aligned(x, 16) && ldx % 8 == 0 && K % 8 == 0, s));
  return gemm(p, RS_BF16, s, true);
}

int rs_fp8_linear(const void* x, int64_t ldx, int M, int K, int N, const void* wq, int64_t ldw,
                  const void* scales_w, const void* bias, int gelu, const void* resid, int64_t ldr,
                  void* out, int64_t ldo, void* ws, uint64_t ws_bytes, void* stream) {
  return fp8_linear(x, ldx, M, K, N, wq, ldw, scales_w, bias, gelu, resid, ldr, out, ldo, ws,
                    ws_bytes, static_cast<cudaStream_t>(stream), false, rs::kDefaultTimeoutNs);
}

int rs_debug_fp8_linear_skip_load(const void* x, int64_t ldx, int M, int K, int N, const void* wq,
                                  int64_t ldw, const void* scales_w, void* out, int64_t ldo,
                                  int timeout_us, void* stream) {
  if (M < 1 || !dim_ok(K) || !dim_ok(N) || !rs::fp8_few_rows(M, N, K) || timeout_us < 1 ||
      timeout_us > 10000000)
    return RS_ERR_SHAPE;
  return fp8_linear(x, ldx, M, K, N, wq, ldw, scales_w, nullptr, 0, nullptr, 0, out, ldo, nullptr, 0,
                    static_cast<cudaStream_t>(stream), true,
                    static_cast<unsigned long long>(timeout_us) * 1000ull);
}

uint64_t rs_fp8_linear_backward_ws_bytes(int M, int N) {
  if (M < 0 || M >= kMaxDim || !dim_ok(N)) return 0;
  const int m = M > 0 ? M : 1;
  return q_space(m, N).bytes + q_space(N, m).bytes + rs_fp8_quantize_ws_bytes(m, N);
}

int rs_fp8_linear_backward(const void* dy, int64_t lddy, int M, int N, int K, const void* xt,
                           int64_t ldxt, const void* scales_xt, const void* wt, int64_t ldwt,
                           const void* scales_wt, void* dx, int64_t lddx, void* dw, int64_t lddw,
                           int dw_dtype, float* db, void* ws, uint64_t ws_bytes, void* stream) {
  RS_TRY(check_gemm_dims(M, N, K));
  RS_TRY(check_gemm_dims(M, K, N));
  RS_TRY(check_gemm_dims(N, K, M > 0 ? M : 1));
  if (dw_dtype != RS_BF16 && dw_dtype != RS_FP32) return RS_ERR_SHAPE;
  const int wes = elem_bytes(dw_dtype);
  if (lddy < N || (dx && lddx < K) || (dw && lddw < K)) return RS_ERR_SHAPE;
  if (!aligned(dx, 2) || !aligned(dw, wes) || !aligned(db, 4)) return RS_ERR_ALIGN;
  if (!dx && !dw && !db) return RS_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dw) RS_CUDA(cudaMemset2DAsync(dw, lddw * wes, 0, static_cast<size_t>(K) * wes, N, s));
    if (db) RS_CUDA(cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 4, s));
    return RS_OK;
  }
  if (!dy) return RS_ERR_NULL;
  if (!aligned(dy, 2)) return RS_ERR_ALIGN;
  if (dx) RS_TRY(check_q(wt, ldwt, scales_wt, N));
  if (dw) RS_TRY(check_q(xt, ldxt, scales_xt, M));
  RS_TRY(check_ws(ws, ws_bytes, rs_fp8_linear_backward_ws_bytes(M, N)));
  const QSpace w = q_space(M, N), wtr = q_space(N, M);
  uint8_t* base = static_cast<uint8_t*>(ws);
  rs::Quant qp{};
  qp.x = dy;
  qp.ldx = lddy;
  qp.rows = M;
  qp.K = N;
  if (dx) {
    qp.q = base;
    qp.ldq = static_cast<int64_t>(w.ld);
    qp.scales = base + w.scales;
  }
  if (dw || db) {
    qp.qt = base + w.bytes;
    qp.ldqt = static_cast<int64_t>(wtr.ld);
    qp.scales_t = qp.qt + wtr.scales;
  }
  const bool direct = db && rs::quant_direct(M);
  if (db) qp.partials = direct ? db : reinterpret_cast<float*>(base + w.bytes + wtr.bytes);
  qp.chunks = direct ? 1 : rs::quant_chunks(M, N);
  RS_CUDA(rs::launch_quantize(qp, RS_BF16, aligned(dy, 16) && lddy % 8 == 0 && N % 8 == 0, s));
  if (dx) {
    rs::Fp8Gemm p{};
    p.a = qp.q;
    p.lda = qp.ldq;
    p.sa = qp.scales;
    p.b = wt;
    p.ldb = ldwt;
    p.sb = scales_wt;
    p.M = M;
    p.N = K;
    p.K = N;
    p.out = dx;
    p.ldo = lddx;
    RS_TRY(gemm(p, RS_BF16, s, true));
  }
  if (dw) {
    rs::Fp8Gemm p{};
    p.a = qp.qt;
    p.lda = qp.ldqt;
    p.sa = qp.scales_t;
    p.b = xt;
    p.ldb = ldxt;
    p.sb = scales_xt;
    p.M = N;
    p.N = K;
    p.K = M;
    p.out = dw;
    p.ldo = lddw;
    RS_TRY(gemm(p, dw_dtype, s, true));
  }
  if (db && !direct)
    RS_CUDA(rs::launch_col_reduce(qp.partials, qp.chunks, N, N, db, nullptr, s, true));
  return RS_OK;
}

uint64_t rs_mlp_forward_fp8_ws_bytes(int M, int C, int H) {
  if (M < 0 || M >= kMaxDim || C < 64 || C > RS_MAX_C || C % 64 != 0 || H < 64 || H > RS_MAX_H ||
      H % 64 != 0)
    return 0;
  const int m = M > 0 ? M : 1;
  return q_space(m, C).bytes + q_space(m, H).bytes;
}

int rs_mlp_forward_fp8(const void* x, int M, int C, int H, const void* w1q, int64_t ldw1,
                       const void* scales_w1, const void* b1, const void* w2q, int64_t ldw2,
                       const void* scales_w2, const void* b2, const void* gamma, const void* beta,
                       void* y, void* ws, uint64_t ws_bytes, void* stream) {
  const uint64_t need = rs_mlp_forward_fp8_ws_bytes(M, C, H);
  if (need == 0) return RS_ERR_SHAPE;
  RS_TRY(check_gemm_dims(M, H, C));
  if (M == 0) return RS_OK;
  if (!x || !y || !b1 || !b2 || !gamma || !beta) return RS_ERR_NULL;
  RS_TRY(check_q(w1q, ldw1, scales_w1, C));
  RS_TRY(check_q(w2q, ldw2, scales_w2, H));
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(b1, 16) || !aligned(b2, 16) ||
      !aligned(gamma, 16) || !aligned(beta, 16))
    return RS_ERR_ALIGN;
  RS_TRY(check_ws(ws, ws_bytes, need));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const QSpace wu = q_space(M, C), wa = q_space(M, H);
  uint8_t* u = static_cast<uint8_t*>(ws);
  uint8_t* a = u + wu.bytes;
  int sms = 0;
  RS_TRY(rs::device_sms(&sms));
  rs::LnForward n = norm_args(x, C, M, C, gamma, beta, RS_BF16, rs::kLnEps, nullptr);
  n.q = u;
  n.ldq = static_cast<int64_t>(wu.ld);
  n.scales = u + wu.scales;
  n.kq = (C + 511) / 512;
  RS_CUDA(rs::launch_ln_quantize(n, RS_BF16, sms, s));
  rs::Fp8Gemm p{};
  p.a = u;
  p.lda = n.ldq;
  p.sa = n.scales;
  p.b = w1q;
  p.ldb = ldw1;
  p.sb = scales_w1;
  p.M = M;
  p.N = H;
  p.K = C;
  p.bias = static_cast<const __nv_bfloat16*>(b1);
  p.gelu = 1;
  p.out = a;
  p.ldo = static_cast<int64_t>(wa.ld);
  p.out_scales = a + wa.scales;
  RS_TRY(gemm(p, RS_E4M3, s, true));
  rs::Fp8Gemm f{};
  f.a = a;
  f.lda = p.ldo;
  f.sa = p.out_scales;
  f.b = w2q;
  f.ldb = ldw2;
  f.sb = scales_w2;
  f.M = M;
  f.N = C;
  f.K = H;
  f.bias = static_cast<const __nv_bfloat16*>(b2);
  f.resid = x;
  f.ldr = C;
  f.out = y;
  f.ldo = C;
  return gemm(f, RS_BF16, s, true);
}

}  // extern "C"
