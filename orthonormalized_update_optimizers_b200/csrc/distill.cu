// distill_loss and distill_loss_backward: the loss of a student's logits
// against a teacher's top logits, and its gradient.
//
//   p = softmax(t / tau) over a row's teacher entries, q = softmax(s / tau)
//   over the vocabulary:  L = tau^2 sum_k p_k (log p_k - log q_{i_k})
//   dS_v = dL tau (q_v - sum_{k: i_k = v} p_k)
//
// HBM-bound: the loss reads the logits once (running maximum and sum), the
// gradient reads and writes them once.
#include "tokens.cuh"

namespace ouo {
namespace {

constexpr int kDThreads = 512;
constexpr float kLowest = -3.402823466e38f;  // finite: -inf - m stays -inf
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct DistillArgs {
  const void* S; int64_t lds; int s_bf16;
  const void* T; int64_t ldt; int t_bf16;
  const int32_t* I; int64_t ldi;
  int64_t rows, V;
  int K;
  float tau, inv_tau;
  float* loss;
  float* lse;
  const float* dloss;
  void* dS; int64_t ldds; int ds_bf16;
};

struct Teacher {
  float p[OUO_DISTILL_MAX_ENTRIES];
  int idx[OUO_DISTILL_MAX_ENTRIES];
};

__device__ __forceinline__ float block_fmax(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : kLowest;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  return v;
}

// The row's teacher entries in shared memory: idx = -1 for one that does not
// count (index outside the vocabulary, logit -inf), p its probability.
// Returns the log of the normalizer, and through `any` whether one counts.
__device__ __forceinline__ float teacher_probs(const DistillArgs& a, int64_t row, Teacher& t,
                                               float* red, bool* any) {
  float m = kLowest;
  int some = 0;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    int i = a.I[row * a.ldi + k];
    const float v = ld1(a.T, row * a.ldt + k, a.t_bf16) * a.inv_tau;
    if (i < 0 || i >= a.V || v == -INFINITY) i = -1;
    t.idx[k] = i;
    t.p[k] = v;
    if (i >= 0) {
      m = fmaxf(m, v);
      some = 1;
    }
  }
  *any = __syncthreads_or(some) != 0;
  m = block_fmax(m, red);
  float z = 0.f;
  for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
    t.p[k] -= m;
    if (t.idx[k] >= 0) z += expf(t.p[k]);
  }
  z = block_sum(z, red);
  const float lz = logf(z);
  for (int k = threadIdx.x; k < a.K; k += blockDim.x)
    t.p[k] = t.idx[k] >= 0 ? t.p[k] - lz : -INFINITY;  // log p
  __syncthreads();
  return lz;
}

__global__ void __launch_bounds__(kDThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ Teacher t;
  __shared__ float red[32];
  __shared__ double redd[32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    bool any;
    teacher_probs(a, row, t, red, &any);
    if (!any) {
      if (threadIdx.x == 0) {
        a.loss[row] = 0.f;
        a.lse[row] = 0.f;
      }
      __syncthreads();
      continue;
    }
    // running maximum and sum of the thread's share
    float m = kLowest, z = 0.f;
    for (int64_t j = threadIdx.x; j < a.V; j += kDThreads) {
      const float v = ld1(a.S, row * a.lds + j, a.s_bf16) * a.inv_tau;
      const float mn = fmaxf(m, v);
      z = z * ex2((m - mn) * kLog2e) + ex2((v - mn) * kLog2e);
      m = mn;
    }
    const float M = block_fmax(m, red);
    z = block_sum(z * ex2((m - M) * kLog2e), red);
    const double lse = (double)M + log((double)z);
    double acc = 0.0;
    for (int k = threadIdx.x; k < a.K; k += kDThreads) {
      if (t.idx[k] < 0) continue;
      const float lp = t.p[k], p = expf(lp);
      if (p == 0.f) continue;  // also where the student's logit is -inf
      acc += (double)p * ((double)lp - ((double)(ld1(a.S, row * a.lds + t.idx[k], a.s_bf16) *
                                                 a.inv_tau) - lse));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if ((threadIdx.x & 31) == 0) redd[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kDThreads / 32; ++w) acc += redd[w];
      a.loss[row] = (float)((double)a.tau * (double)a.tau * acc);
      a.lse[row] = (float)lse;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kDThreads)
distill_bwd_kernel(const __grid_constant__ DistillArgs a) {
  __shared__ Teacher t;
  __shared__ float sq[OUO_DISTILL_MAX_ENTRIES];
  __shared__ float red[32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float g = a.dloss[row] * a.tau, lse = a.lse[row];
    bool any = false;
    if (g != 0.f) teacher_probs(a, row, t, red, &any);
    if (!any) {
      for (int64_t j = threadIdx.x; j < a.V; j += kDThreads)
        st1(a.dS, row * a.ldds + j, 0.f, a.ds_bf16);
      __syncthreads();
      continue;
    }
    auto prob = [&](int64_t j) {
      return ex2((ld1(a.S, row * a.lds + j, a.s_bf16) * a.inv_tau - lse) * kLog2e);
    };
    // dS may be S itself: the entries' own probabilities are read first
    for (int k = threadIdx.x; k < a.K; k += kDThreads)
      if (t.idx[k] >= 0) {
        sq[k] = prob(t.idx[k]);
        t.p[k] = expf(t.p[k]);
      }
    __syncthreads();
    for (int64_t j = threadIdx.x; j < a.V; j += kDThreads)
      st1(a.dS, row * a.ldds + j, g * prob(j), a.ds_bf16);
    __syncthreads();
    // the first entry of each index takes every entry of that index
    for (int k = threadIdx.x; k < a.K; k += kDThreads) {
      const int i = t.idx[k];
      if (i < 0) continue;
      float p = 0.f;
      bool first = true;
      for (int l = 0; l < a.K; ++l)
        if (t.idx[l] == i) {
          if (l < k) { first = false; break; }
          p += t.p[l];
        }
      if (first) st1(a.dS, row * a.ldds + i, g * (sq[k] - p), a.ds_bf16);
    }
    __syncthreads();
  }
}

int check_distill(const ouo_mat* S, int s_dtype, const ouo_mat* teacher, int t_dtype,
                  const ouo_mat* idx, float temperature) {
  if (!S || !teacher || !idx)
    return set_error(OUO_ERR_INVALID_ARG, "S, teacher and idx are required");
  OUO_TRY(validate_dtype(s_dtype, "S"));
  OUO_TRY(validate_dtype(t_dtype, "teacher"));
  OUO_TRY(validate_tokens(*S, elem_size(s_dtype), "S", 0));
  OUO_TRY(validate_tokens(*teacher, elem_size(t_dtype), "teacher", 0));
  OUO_TRY(validate_tokens(*idx, 4, "idx", 0));
  const int64_t T = S->rows;
  if (T > 0 && S->cols == 0) return set_error(OUO_ERR_INVALID_ARG, "S: rows without columns");
  if (T > 0 && teacher->cols == 0)
    return set_error(OUO_ERR_INVALID_ARG, "teacher: rows without entries");
  OUO_TRY(validate_shape(*teacher, T, teacher->cols, "teacher", 0));
  OUO_TRY(validate_shape(*idx, T, teacher->cols, "idx", 0));
  if (teacher->cols > OUO_DISTILL_MAX_ENTRIES)
    return set_error(OUO_ERR_UNSUPPORTED, "teacher: %lld entries a row, at most %d",
                     (long long)teacher->cols, OUO_DISTILL_MAX_ENTRIES);
  if (!(temperature >= 1e-3f && temperature <= 1e3f))
    return set_error(OUO_ERR_INVALID_ARG, "temperature must be in [1e-3, 1e3]");
  return OUO_OK;
}

DistillArgs distill_args(const ouo_mat* S, int s_dtype, const ouo_mat* teacher, int t_dtype,
                         const ouo_mat* idx, float temperature) {
  DistillArgs a{};
  a.S = S->ptr; a.lds = S->ld; a.s_bf16 = s_dtype == OUO_BF16;
  a.T = teacher->ptr; a.ldt = teacher->ld; a.t_bf16 = t_dtype == OUO_BF16;
  a.I = (const int32_t*)idx->ptr; a.ldi = idx->ld;
  a.rows = S->rows; a.V = S->cols; a.K = (int)teacher->cols;
  a.tau = temperature;
  a.inv_tau = 1.f / temperature;
  return a;
}

}  // namespace
}  // namespace ouo

extern "C" {

int distill_loss(const ouo_mat* S, int s_dtype, const ouo_mat* teacher, int t_dtype,
                 const ouo_mat* idx, float temperature, float* loss, float* lse, void* stream) {
  using namespace ouo;
  clear_error();
  OUO_TRY(check_distill(S, s_dtype, teacher, t_dtype, idx, temperature));
  OUO_TRY(validate_vec(loss, S->rows, 4, "loss"));
  OUO_TRY(validate_vec(lse, S->rows, 4, "lse"));
  if (S->rows == 0) return OUO_OK;
  OUO_TRY(require_sm100());
  DistillArgs a = distill_args(S, s_dtype, teacher, t_dtype, idx, temperature);
  a.loss = loss;
  a.lse = lse;
  const int64_t cap = (int64_t)num_sms() * 4;
  distill_kernel<<<(unsigned)(a.rows < cap ? a.rows : cap), kDThreads, 0, (cudaStream_t)stream>>>(a);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

int distill_loss_backward(const ouo_mat* S, int s_dtype, const ouo_mat* teacher, int t_dtype,
                          const ouo_mat* idx, float temperature, const float* lse,
                          const float* dloss, const ouo_mat* dS, int ds_dtype, void* stream) {
  using namespace ouo;
  clear_error();
  OUO_TRY(check_distill(S, s_dtype, teacher, t_dtype, idx, temperature));
  if (!dS) return set_error(OUO_ERR_INVALID_ARG, "dS is required");
  OUO_TRY(validate_dtype(ds_dtype, "dS"));
  OUO_TRY(validate_tokens(*dS, elem_size(ds_dtype), "dS", 0));
  OUO_TRY(validate_shape(*dS, S->rows, S->cols, "dS", 0));
  if (dS->ptr == S->ptr && (ds_dtype != s_dtype || dS->ld != S->ld) && S->rows > 0)
    return set_error(OUO_ERR_INVALID_ARG, "dS in place of S needs S's type and row pitch");
  OUO_TRY(validate_vec(lse, S->rows, 4, "lse"));
  OUO_TRY(validate_vec(dloss, S->rows, 4, "dloss"));
  if (S->rows == 0) return OUO_OK;
  OUO_TRY(require_sm100());
  DistillArgs a = distill_args(S, s_dtype, teacher, t_dtype, idx, temperature);
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dS = dS->ptr; a.ldds = dS->ld; a.ds_bf16 = ds_dtype == OUO_BF16;
  const int64_t cap = (int64_t)num_sms() * 4;
  distill_bwd_kernel<<<(unsigned)(a.rows < cap ? a.rows : cap), kDThreads, 0, (cudaStream_t)stream>>>(a);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

}  // extern "C"
