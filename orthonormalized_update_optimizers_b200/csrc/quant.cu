// quantize_int8: matrices to 8-bit integers with one scale per row, or
// transposed with one scale per column.
//
//   scale_i = max_j |x_ij| / 127,  q_ij = rint(x_ij / scale_i)
//
// HBM-bound: each element is read once and leaves as one byte.
#include "tokens.cuh"

namespace ouo {
namespace {

constexpr int kQThreads = 256;

struct QuantArgs {
  int nmat, bf16;
  int64_t row_start[kChunk + 1];
  int64_t cols[kChunk];
  const void* X[kChunk];
  int64_t ldx[kChunk];
  int8_t* Q[kChunk];
  int64_t ldq[kChunk];
  float* scale[kChunk];
};

// One block per row: largest magnitude, then the rounding (the second read
// comes from the caches).
__global__ void __launch_bounds__(kQThreads) quant_rows_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t red[32];
  const int64_t total = a.row_start[a.nmat];
  for (int64_t row = blockIdx.x; row < total; row += gridDim.x) {
    int lo = 0, hi = a.nmat - 1;
    while (lo < hi) {
      int mid = (lo + hi + 1) >> 1;
      if (a.row_start[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int64_t r = row - a.row_start[lo], n = a.cols[lo];
    const char* x = reinterpret_cast<const char*>(a.X[lo]) + r * a.ldx[lo] * (a.bf16 ? 2 : 4);
    uint32_t m = 0;
    for (int64_t j = threadIdx.x; j < n; j += kQThreads) m = max(m, mag(ld1(x, j, a.bf16)));
    m = block_max(m, red);
    const Quant q = quant_of(m);
    if (threadIdx.x == 0) a.scale[lo][r] = q.scale;
    int8_t* o = a.Q[lo] + r * a.ldq[lo];
    for (int64_t j = threadIdx.x; j < n; j += kQThreads) o[j] = (int8_t)quant1(ld1(x, j, a.bf16), q);
  }
}

// Transposed: one block per 32 columns of one matrix.
__global__ void __launch_bounds__(256)
quant_cols_kernel(const void* X, int bf16, int64_t rows, int64_t cols, int64_t ldx, int8_t* Q,
                  int64_t ldq, float* scale) {
  __shared__ uint32_t amax[8][33];
  __shared__ int8_t tile[32][36];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  uint32_t m = 0;
  if (c < cols)
    for (int64_t r = w; r < rows; r += 8) m = max(m, mag(ld1(X, r * ldx + c, bf16)));
  amax[w][lane] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = max(m, amax[i][lane]);
  const Quant q = quant_of(m);
  if (w == 0 && c < cols) scale[c] = q.scale;
  for (int64_t r0 = 0; r0 < rows; r0 += 32) {
    for (int i = w; i < 32; i += 8)
      tile[lane][i] = c < cols && r0 + i < rows
          ? (int8_t)quant1(ld1(X, (r0 + i) * ldx + c, bf16), q) : (int8_t)0;
    __syncthreads();
    for (int i = w; i < 32; i += 8) {
      const int64_t oc = (int64_t)blockIdx.x * 32 + i;
      if (oc < cols && r0 + lane < rows) Q[oc * ldq + r0 + lane] = tile[i][lane];
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace ouo

extern "C" int quantize_int8(const ouo_mat* X, int x_dtype, const ouo_mat* Q, float* const* scale,
                             int nmat, int transpose, void* stream) {
  using namespace ouo;
  clear_error();
  if (nmat < 0 || nmat > OUO_MAX_BATCH)
    return set_error(OUO_ERR_INVALID_ARG, "nmat %d out of range", nmat);
  if (nmat == 0) return OUO_OK;
  if (!X || !Q || !scale) return set_error(OUO_ERR_INVALID_ARG, "NULL batch array");
  if (transpose != 0 && transpose != 1)
    return set_error(OUO_ERR_INVALID_ARG, "transpose must be 0 or 1");
  OUO_TRY(validate_dtype(x_dtype, "X"));
  for (int i = 0; i < nmat; ++i) {
    OUO_TRY(validate_tokens(X[i], elem_size(x_dtype), "X", i));
    OUO_TRY(validate_tokens(Q[i], 1, "Q", i));
    OUO_TRY(validate_shape(Q[i], transpose ? X[i].cols : X[i].rows,
                           transpose ? X[i].rows : X[i].cols, "Q", i));
    OUO_TRY(validate_vec(scale[i], Q[i].rows, 4, "scale"));
  }
  OUO_TRY(require_sm100());
  cudaStream_t s = (cudaStream_t)stream;
  const int bf16 = x_dtype == OUO_BF16;
  if (transpose) {
    for (int i = 0; i < nmat; ++i) {
      if (X[i].cols == 0) continue;
      quant_cols_kernel<<<(unsigned)ceil_div(X[i].cols, 32), 256, 0, s>>>(
          X[i].ptr, bf16, X[i].rows, X[i].cols, X[i].ld, (int8_t*)Q[i].ptr, Q[i].ld, scale[i]);
      OUO_CHECK_LAUNCH();
    }
    return OUO_OK;
  }
  for (int c0 = 0; c0 < nmat; c0 += kChunk) {
    const int cn = nmat - c0 < kChunk ? nmat - c0 : kChunk;
    QuantArgs a;
    a.nmat = cn;
    a.bf16 = bf16;
    int64_t acc = 0;
    for (int i = 0; i < cn; ++i) {
      const ouo_mat& x = X[c0 + i];
      a.row_start[i] = acc;
      a.cols[i] = x.cols;
      a.X[i] = x.ptr;
      a.ldx[i] = x.ld;
      a.Q[i] = (int8_t*)Q[c0 + i].ptr;
      a.ldq[i] = Q[c0 + i].ld;
      a.scale[i] = scale[c0 + i];
      acc += x.rows;
    }
    a.row_start[cn] = acc;
    if (acc == 0) continue;
    const int64_t cap = (int64_t)num_sms() * 8;
    quant_rows_kernel<<<(unsigned)(acc < cap ? acc : cap), kQThreads, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
  }
  return OUO_OK;
}
