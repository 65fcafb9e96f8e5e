// rms_norm and rms_norm_backward: the root-mean-square norm in front of a
// product, with the residual's addition and an 8-bit output.
//
//   h = x + residual (rounded to H's type),  r = 1 / sqrt(mean(h^2) + eps),
//   y = h r w;   8-bit output: q = rint(y / scale), scale = max |y| / 127
//   dx = dh + r (w dy - h r^2 mean(w dy h)),  dw = sum over rows of dy h r
//
// HBM-bound: every matrix is read or written once.
#include "tokens.cuh"

namespace ouo {
namespace {

constexpr int kNThreads = 256;

struct NormArgs {
  const void* X; int64_t ldx; int x_bf16;
  const void* R; int64_t ldr;
  void* H; int64_t ldh; int h_bf16;
  const void* W; int w_bf16;
  void* Y; int64_t ldy; int y_bf16;
  int8_t* Q; int64_t ldq; float* scale;
  float* rstd;
  int64_t rows, cols;
  float eps;
};

__device__ __forceinline__ const char* row_of(const void* p, int64_t r, int64_t ld, int bf16) {
  return reinterpret_cast<const char*>(p) + r * ld * (bf16 ? 2 : 4);
}

__global__ void __launch_bounds__(kNThreads) rms_kernel(const __grid_constant__ NormArgs a) {
  __shared__ uint32_t red[32];
  const int64_t n = a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* x = row_of(a.X, row, a.ldx, a.x_bf16);
    const char* rs = a.R ? row_of(a.R, row, a.ldr, a.h_bf16) : nullptr;
    char* h = a.H ? const_cast<char*>(row_of(a.H, row, a.ldh, a.h_bf16)) : nullptr;
    auto value = [&](int64_t j) {  // h, once written
      return h ? ld1(h, j, a.h_bf16) : ld1(x, j, a.x_bf16);
    };
    float acc = 0.f;
    for (int64_t j = threadIdx.x; j < n; j += kNThreads) {
      float v = ld1(x, j, a.x_bf16);
      if (rs) v += ld1(rs, j, a.h_bf16);
      if (h) {
        st1(h, j, v, a.h_bf16);
        v = round_to(v, a.h_bf16);
      }
      acc = fmaf(v, v, acc);
    }
    acc = block_sum(acc, reinterpret_cast<float*>(red));
    const float rstd = __frsqrt_rn(acc / (float)n + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    uint32_t m = 0;
    for (int64_t j = threadIdx.x; j < n; j += kNThreads) {
      const float y = value(j) * rstd * ld1(a.W, j, a.w_bf16);
      m = max(m, mag(y));
      if (a.Y) st1(const_cast<char*>(row_of(a.Y, row, a.ldy, a.y_bf16)), j, y, a.y_bf16);
    }
    if (!a.Q) continue;
    const Quant q = quant_of(block_max(m, red));
    if (threadIdx.x == 0) a.scale[row] = q.scale;
    for (int64_t j = threadIdx.x; j < n; j += kNThreads)
      a.Q[row * a.ldq + j] = (int8_t)quant1(value(j) * rstd * ld1(a.W, j, a.w_bf16), q);
  }
}

struct NormBwdArgs {
  const void* dY; int64_t lddy; int dy_bf16;
  const void* H; int64_t ldh; int h_bf16;
  const void* W; int w_bf16;
  const float* rstd;
  const void* dH; int64_t lddh;
  void* dX; int64_t lddx; int dx_bf16;
  float* part;
  int64_t rows, cols;
};

// Block b takes rows b, b + grid, ...; its share of dw goes to row b of the
// partial sums (each thread keeps its own columns, so nothing races).
__global__ void __launch_bounds__(kNThreads) rms_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  __shared__ uint32_t red[32];
  const int64_t n = a.cols;
  float* part = a.part ? a.part + blockIdx.x * n : nullptr;
  if (part)
    for (int64_t j = threadIdx.x; j < n; j += kNThreads) part[j] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* dy = row_of(a.dY, row, a.lddy, a.dy_bf16);
    const char* h = row_of(a.H, row, a.ldh, a.h_bf16);
    const char* dh = a.dH ? row_of(a.dH, row, a.lddh, a.dx_bf16) : nullptr;
    char* dx = const_cast<char*>(row_of(a.dX, row, a.lddx, a.dx_bf16));
    const float r = a.rstd[row];
    float acc = 0.f;
    for (int64_t j = threadIdx.x; j < n; j += kNThreads) {
      const float g = ld1(dy, j, a.dy_bf16), xh = ld1(h, j, a.h_bf16) * r;
      acc = fmaf(g * ld1(a.W, j, a.w_bf16), xh, acc);
      if (part) part[j] = fmaf(g, xh, part[j]);
    }
    const float c = block_sum(acc, reinterpret_cast<float*>(red)) / (float)n;
    for (int64_t j = threadIdx.x; j < n; j += kNThreads) {
      const float g = ld1(dy, j, a.dy_bf16) * ld1(a.W, j, a.w_bf16);
      float v = r * (g - ld1(h, j, a.h_bf16) * r * c);
      if (dh) v += ld1(dh, j, a.dx_bf16);
      st1(dx, j, v, a.dx_bf16);
    }
  }
}

// dw = sum of the partial rows, in a fixed order.
__global__ void __launch_bounds__(256)
rms_dw_kernel(const float* part, int nparts, int64_t cols, float* dw) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= cols) return;
  float v = 0.f;
  for (int p = 0; p < nparts; ++p) v += part[p * cols + j];
  dw[j] = v;
}

// Rows of partial sums of dw: a function of the shape alone, so that the
// workspace query needs no device.
constexpr int64_t kMaxParts = 296;
int64_t bwd_parts(int64_t rows) { return rows < kMaxParts ? rows : kMaxParts; }

}  // namespace
}  // namespace ouo

extern "C" {

int rms_norm(const ouo_mat* X, int x_dtype, const ouo_mat* residual, const ouo_mat* H, int h_dtype,
             const void* weight, int w_dtype, float eps, const ouo_mat* Y, int y_dtype,
             const ouo_mat* Q, float* scale, float* rstd, void* stream) {
  using namespace ouo;
  clear_error();
  if (!X) return set_error(OUO_ERR_INVALID_ARG, "X: NULL matrix");
  OUO_TRY(validate_dtype(x_dtype, "X"));
  OUO_TRY(validate_dtype(w_dtype, "weight"));
  OUO_TRY(validate_tokens(*X, elem_size(x_dtype), "X", 0));
  const int64_t T = X->rows, n = X->cols;
  if (T > 0 && n == 0) return set_error(OUO_ERR_INVALID_ARG, "X: rows without columns");
  if (!Y && !Q) return set_error(OUO_ERR_INVALID_ARG, "Y or Q is required");
  if (residual && !H) return set_error(OUO_ERR_INVALID_ARG, "residual needs H");
  if (!(eps >= 0.f)) return set_error(OUO_ERR_INVALID_ARG, "eps must be >= 0");
  if (residual || H) {
    OUO_TRY(validate_dtype(h_dtype, "H"));
    OUO_TRY(validate_tokens(*H, elem_size(h_dtype), "H", 0));
    OUO_TRY(validate_shape(*H, T, n, "H", 0));
  }
  if (residual) {
    OUO_TRY(validate_tokens(*residual, elem_size(h_dtype), "residual", 0));
    OUO_TRY(validate_shape(*residual, T, n, "residual", 0));
  }
  if (Y) {
    OUO_TRY(validate_dtype(y_dtype, "Y"));
    OUO_TRY(validate_tokens(*Y, elem_size(y_dtype), "Y", 0));
    OUO_TRY(validate_shape(*Y, T, n, "Y", 0));
  }
  if (Q) {
    OUO_TRY(validate_tokens(*Q, 1, "Q", 0));
    OUO_TRY(validate_shape(*Q, T, n, "Q", 0));
    OUO_TRY(validate_vec(scale, T, 4, "scale"));
  }
  OUO_TRY(validate_vec(weight, n, elem_size(w_dtype), "weight"));
  OUO_TRY(validate_vec(rstd, 0, 4, "rstd"));
  if (T == 0) return OUO_OK;
  OUO_TRY(require_sm100());
  NormArgs a{};
  a.X = X->ptr; a.ldx = X->ld; a.x_bf16 = x_dtype == OUO_BF16;
  if (residual) { a.R = residual->ptr; a.ldr = residual->ld; }
  if (H) { a.H = H->ptr; a.ldh = H->ld; a.h_bf16 = h_dtype == OUO_BF16; }
  a.W = weight; a.w_bf16 = w_dtype == OUO_BF16;
  if (Y) { a.Y = Y->ptr; a.ldy = Y->ld; a.y_bf16 = y_dtype == OUO_BF16; }
  if (Q) { a.Q = (int8_t*)Q->ptr; a.ldq = Q->ld; a.scale = scale; }
  a.rstd = rstd;
  a.rows = T; a.cols = n; a.eps = eps;
  const int64_t cap = (int64_t)num_sms() * 8;
  rms_kernel<<<(unsigned)(T < cap ? T : cap), kNThreads, 0, (cudaStream_t)stream>>>(a);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

size_t rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return (size_t)(ouo::bwd_parts(rows) * cols) * sizeof(float);
}

int rms_norm_backward(const ouo_mat* dY, int dy_dtype, const ouo_mat* H, int h_dtype,
                      const void* weight, int w_dtype, const float* rstd, const ouo_mat* dH,
                      const ouo_mat* dX, int dx_dtype, float* dweight, void* ws, size_t ws_bytes,
                      void* stream) {
  using namespace ouo;
  clear_error();
  if (!dY || !H || !dX) return set_error(OUO_ERR_INVALID_ARG, "dY, H and dX are required");
  OUO_TRY(validate_dtype(dy_dtype, "dY"));
  OUO_TRY(validate_dtype(h_dtype, "H"));
  OUO_TRY(validate_dtype(w_dtype, "weight"));
  OUO_TRY(validate_dtype(dx_dtype, "dX"));
  OUO_TRY(validate_tokens(*dY, elem_size(dy_dtype), "dY", 0));
  const int64_t T = dY->rows, n = dY->cols;
  if (T > 0 && n == 0) return set_error(OUO_ERR_INVALID_ARG, "dY: rows without columns");
  OUO_TRY(validate_tokens(*H, elem_size(h_dtype), "H", 0));
  OUO_TRY(validate_shape(*H, T, n, "H", 0));
  OUO_TRY(validate_tokens(*dX, elem_size(dx_dtype), "dX", 0));
  OUO_TRY(validate_shape(*dX, T, n, "dX", 0));
  if (dH) {
    OUO_TRY(validate_tokens(*dH, elem_size(dx_dtype), "dH", 0));
    OUO_TRY(validate_shape(*dH, T, n, "dH", 0));
  }
  OUO_TRY(validate_vec(weight, n, elem_size(w_dtype), "weight"));
  OUO_TRY(validate_vec(rstd, T, 4, "rstd"));
  OUO_TRY(validate_vec(dweight, 0, 4, "dweight"));
  const size_t need = dweight ? rms_norm_backward_workspace_bytes(T, n) : 0;
  if (need > 0 && (!ws || ws_bytes < need || (uintptr_t)ws % 16 != 0))
    return set_error(OUO_ERR_WORKSPACE, "workspace: %zu bytes needed (16-byte aligned), %zu given",
                     need, ws ? ws_bytes : (size_t)0);
  OUO_TRY(require_sm100());
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t parts = bwd_parts(T);
  if (T > 0) {
    NormBwdArgs a{};
    a.dY = dY->ptr; a.lddy = dY->ld; a.dy_bf16 = dy_dtype == OUO_BF16;
    a.H = H->ptr; a.ldh = H->ld; a.h_bf16 = h_dtype == OUO_BF16;
    a.W = weight; a.w_bf16 = w_dtype == OUO_BF16;
    a.rstd = rstd;
    if (dH) { a.dH = dH->ptr; a.lddh = dH->ld; }
    a.dX = dX->ptr; a.lddx = dX->ld; a.dx_bf16 = dx_dtype == OUO_BF16;
    a.part = dweight ? (float*)ws : nullptr;
    a.rows = T; a.cols = n;
    rms_bwd_kernel<<<(unsigned)parts, kNThreads, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
  }
  if (dweight && n > 0) {
    rms_dw_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, s>>>((const float*)ws, (int)parts, n,
                                                             dweight);
    OUO_CHECK_LAUNCH();
  }
  return OUO_OK;
}

}  // extern "C"
