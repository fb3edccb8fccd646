// C ABI of the 8-bit projections: argument checks and launches.
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace {

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of K bf16, `stride` apart (a single row has no stride), that a kernel reads or writes in 16-byte vectors.
int check_rows(const void* p, int64_t stride, int rows, int K) {
  if (!p || (rows > 1 && stride < K)) return MOE_ERR_INVALID;
  return aligned(p, 16) && (rows == 1 || stride % 8 == 0) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// Codes of K values a row, and their scales in `high` rows a row of scales.
int check_block8(const void* codes, int64_t ld, const void* scales, int64_t lds, int rows, int high, int K) {
  const bool one = rows == 1, one_s = rows <= high;
  if (!codes || !scales || (!one && ld < K) || (!one_s && lds < (static_cast<int64_t>(K) + 127) / 128)) return MOE_ERR_INVALID;
  return aligned(codes, 16) && (one || ld % 16 == 0) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int check_sizes(int64_t rows, int K) {
  if (rows < 0 || K <= 0) return MOE_ERR_INVALID;
  return K % 16 || K > INT_MAX - 1024 ? MOE_ERR_UNSUPPORTED : MOE_OK;   // (K is counted in blocks of 128)
}

}  // namespace

extern "C" {

int moe_rms_norm8(const void* x, int64_t x_stride, const void* residual, int64_t r_stride, const void* weight, float eps,
                  int T, int H, void* h, int64_t h_stride, void* y, int64_t y_stride, void* codes, int64_t ld,
                  void* scales, int64_t lds, cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_sizes(T, H);
  if (rc == MOE_ERR_INVALID || !(eps >= 0.f && isfinite(eps))) return MOE_ERR_INVALID;
  if (rc || H > 65536) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!residual != !h || (!y && !codes) || !codes != !scales) return MOE_ERR_INVALID;
  if ((rc = check_rows(x, x_stride, T, H)) || (residual && ((rc = check_rows(residual, r_stride, T, H)) || (rc = check_rows(h, h_stride, T, H)))) ||
      (y && (rc = check_rows(y, y_stride, T, H))) || (codes && (rc = check_block8(codes, ld, scales, lds, T, 1, H))))
    return rc;
  if (!aligned(weight, 16)) return MOE_ERR_UNSUPPORTED;
  const moe::Norm8 a{x, x_stride, residual, r_stride, weight, eps, H, h, h_stride, y, y_stride, static_cast<uint8_t*>(codes), ld,
                     static_cast<uint8_t*>(scales), lds};
  int n = 0;
  rc = moe::rms_norm8_launch(a, T, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

int moe_quantize8(const void* x, int64_t x_stride, int T, int K, int act, void* codes, int64_t ld, void* scales, int64_t lds,
                  cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_sizes(T, K);
  if (rc || (act != 0 && act != 1)) return rc ? rc : MOE_ERR_INVALID;
  if (K > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((rc = check_rows(x, x_stride, T, act ? 2 * K : K)) || (rc = check_block8(codes, ld, scales, lds, T, 1, K))) return rc;
  if (static_cast<int64_t>(T) * ((K + 127) / 128) > INT_MAX) return MOE_ERR_UNSUPPORTED;   // (blocks are counted in 32 bits)
  int n = 0;
  rc = moe::quantize8_launch({x, x_stride, K, static_cast<uint8_t*>(codes), ld, static_cast<uint8_t*>(scales), lds}, T, act, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

int moe_quantize8_weight(const void* w, int64_t w_stride, int N, int K, void* codes, int64_t ld, void* scales, int64_t lds,
                         cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_sizes(N, K);
  if (rc) return rc;
  if (N > 65535 * 128) return MOE_ERR_UNSUPPORTED;   // (a grid's y)
  if (N == 0) return MOE_OK;
  if ((rc = check_rows(w, w_stride, N, K)) || (rc = check_block8(codes, ld, scales, lds, N, 128, K))) return rc;
  int n = 0;
  rc = moe::quantize8_weight_launch({w, w_stride, K, static_cast<uint8_t*>(codes), ld, static_cast<uint8_t*>(scales), lds}, N, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

int moe_linear8(const void* a, int64_t lda, const void* a_scales, int64_t las, const void* w, int64_t ldw, const void* w_scales,
                int64_t lws, int T, int N, int K, void* out, int64_t out_stride, cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_sizes(T, K);
  if (rc == MOE_ERR_INVALID || N <= 0) return MOE_ERR_INVALID;
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!out || (T > 1 && out_stride < N)) return MOE_ERR_INVALID;
  if ((rc = check_block8(a, lda, a_scales, las, T, 1, K)) || (rc = check_block8(w, ldw, w_scales, lws, N, 128, K))) return rc;
  if (!aligned(out, 2)) return MOE_ERR_UNSUPPORTED;
  // (tiles end past T and N, and still fit an int)
  if (T > INT_MAX - 1024 || N > INT_MAX - 1024) return MOE_ERR_UNSUPPORTED;
  if (!moe::device_local(a) || !moe::device_local(w) || !moe::device_local(out)) return MOE_ERR_UNSUPPORTED;
  int* status = nullptr;
  int sms = 0, n = 0;
  if ((rc = moe::current_device_info(&status, &sms))) return rc;
  rc = moe::linear8_launch({static_cast<const uint8_t*>(a), lda, static_cast<const uint8_t*>(a_scales), las,
                            static_cast<const uint8_t*>(w), ldw, static_cast<const uint8_t*>(w_scales), lws, T, N, K,
                            static_cast<__nv_bfloat16*>(out), out_stride}, status, sms, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

}  // extern "C"
