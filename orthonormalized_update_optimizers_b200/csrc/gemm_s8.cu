// int8_matmul: D = diag(a_scale) (A B^T) diag(b_scale), A (M x K) and B
// (N x K) 8-bit integers, the products summed exactly in 32 bits.
#include "tokens.cuh"

namespace ouo {
namespace {

// CUDA cores: 64 x 64 tile per block, 32 bytes of K per step, 4 x 4 outputs
// per thread, four products per dp4a.  Takes any row pitch and alignment.
__global__ void __launch_bounds__(256)
s8_simt_kernel(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, const float* as,
               const float* bs, void* D, int64_t ldd, int bf16, int64_t M, int64_t N, int64_t K,
               int64_t tiles_n) {
  __shared__ int sa[64][9], sb[64][9];
  const int64_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    for (int e = threadIdx.x; e < 512; e += 256) {
      const int r = e >> 3, w = e & 7;
      int va = 0, vb = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t k = k0 + 4 * w + b;
        if (k < K && m0 + r < M) va |= (int)(uint8_t)A[(m0 + r) * lda + k] << (8 * b);
        if (k < K && n0 + r < N) vb |= (int)(uint8_t)B[(n0 + r) * ldb + k] << (8 * b);
      }
      sa[r][w] = va;
      sb[r][w] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      int x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = sa[ty * 4 + i][w];
        y[i] = sb[tx + 16 * i][w];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx + 16 * j;
      if (n < N) st1(D, m * ldd + n, (float)acc[i][j] * as[m] * bs[n], bf16);
    }
  }
}

}  // namespace
}  // namespace ouo

extern "C" int int8_matmul(const ouo_mat* A, const float* const* a_scale, const ouo_mat* B,
                           const float* const* b_scale, const ouo_mat* D, int d_dtype, int nmat,
                           int* dev_status, void* stream) {
  using namespace ouo;
  clear_error();
  if (nmat < 0 || nmat > OUO_MAX_BATCH)
    return set_error(OUO_ERR_INVALID_ARG, "nmat %d out of range", nmat);
  if (nmat == 0) return OUO_OK;
  if (!A || !B || !D || !a_scale || !b_scale)
    return set_error(OUO_ERR_INVALID_ARG, "NULL batch array");
  OUO_TRY(validate_dtype(d_dtype, "D"));
  if ((uintptr_t)dev_status % 4 != 0)
    return set_error(OUO_ERR_INVALID_ARG, "dev_status: not 4-byte aligned");
  for (int i = 0; i < nmat; ++i) {
    OUO_TRY(validate_tokens(A[i], 1, "A", i));
    OUO_TRY(validate_tokens(B[i], 1, "B", i));
    OUO_TRY(validate_tokens(D[i], elem_size(d_dtype), "D", i));
    if (A[i].cols != B[i].cols)
      return set_error(OUO_ERR_INVALID_ARG, "A[%d] has %lld columns, B[%d] has %lld", i,
                       (long long)A[i].cols, i, (long long)B[i].cols);
    if (A[i].cols > OUO_INT8_MAX_DEPTH)
      return set_error(OUO_ERR_UNSUPPORTED,
                       "A[%d]: depth %lld above %d (the sums would leave 32 bits)", i,
                       (long long)A[i].cols, OUO_INT8_MAX_DEPTH);
    OUO_TRY(validate_shape(D[i], A[i].rows, B[i].rows, "D", i));
    OUO_TRY(validate_vec(a_scale[i], A[i].rows, 4, "a_scale"));
    OUO_TRY(validate_vec(b_scale[i], B[i].rows, 4, "b_scale"));
  }
  OUO_TRY(require_sm100());
  cudaStream_t s = (cudaStream_t)stream;
  for (int i = 0; i < nmat; ++i) {
    if (D[i].rows == 0 || D[i].cols == 0) continue;
    const int64_t tn = ceil_div(D[i].cols, 64), tiles = ceil_div(D[i].rows, 64) * tn;
    if (tiles > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "D[%d]: too many tiles", i);
    s8_simt_kernel<<<(unsigned)tiles, 256, 0, s>>>(
        (const int8_t*)A[i].ptr, A[i].ld, (const int8_t*)B[i].ptr, B[i].ld, a_scale[i], b_scale[i],
        D[i].ptr, D[i].ld, d_dtype == OUO_BF16, D[i].rows, D[i].cols, A[i].cols, tn);
    OUO_CHECK_LAUNCH();
  }
  return OUO_OK;
}
