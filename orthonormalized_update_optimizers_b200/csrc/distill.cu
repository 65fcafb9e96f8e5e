// distill_loss and distill_loss_backward: the loss of a student's logits
// against a teacher's top logits, and its gradient.
//
//   p = softmax(t / tau) over a row's teacher entries, q = softmax(s / tau)
//   over the vocabulary:  L = tau^2 sum_k p_k (log p_k - log q_{i_k})
//   dS_v = dL tau (q_v - sum_{k: i_k = v} p_k)
//
// HBM-bound: the loss reads the logits once (running maximum and sum), the
// gradient reads and writes them once.
#include <cstring>

#include "tokens.cuh"
#include "umma.cuh"

namespace ouo {
namespace {

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

// R: as wide as the student's sum.  (In float64 at every temperature, the loss
// of 4096 x 131072 takes 177 us instead of 172.)
template <class R>
struct Teacher {
  R p[OUO_DISTILL_MAX_ENTRIES];      // probability
  float v[OUO_DISTILL_MAX_ENTRIES];  // logit
  alignas(16) int idx[OUO_DISTILL_MAX_ENTRIES];
};

template <int TH>
__device__ __forceinline__ float block_fmax(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TH / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

template <int TH, class R>
__device__ __forceinline__ R block_fsum(R v, R* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TH / 32; ++i) v += red[i];
  return v;
}

// The row's teacher entries in shared memory: idx = -1 for one that does not
// count (index outside the vocabulary, logit -inf); the largest logit and the
// sum of the exponentials.  False if none counts.  The largest logit is
// subtracted before the division by tau: what is divided is small where it
// matters, and finite.
template <int TH, class R>
__device__ __forceinline__ bool teacher_probs(const DistillArgs& a, int64_t row, Teacher<R>& t,
                                              float* redm, R* redz, float* largest, R* norm) {
  float m = kLowest;
  int some = 0;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    int i = a.I[row * a.ldi + k];
    const float v = ld1(a.T, row * a.ldt + k, a.t_bf16);
    if (i < 0 || i >= a.V || v == -INFINITY) i = -1;
    t.idx[k] = i;
    t.v[k] = v;
    if (i >= 0) {
      m = fmaxf(m, v);
      some = 1;
    }
  }
  if (threadIdx.x < 4) {  // whole groups of four for the search for equals
    const int k = a.K + threadIdx.x;
    if (k < OUO_DISTILL_MAX_ENTRIES) t.idx[k] = -1;
  }
  if (__syncthreads_or(some) == 0) return false;
  *largest = m = block_fmax<TH>(m, redm);
  R z = 0;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    t.p[k] = t.idx[k] >= 0 ? exp(((R)t.v[k] - (R)m) * (R)a.inv_tau) : (R)0;
    z += t.p[k];
  }
  *norm = z = block_fsum<TH>(z, redz);
  const R iz = 1 / z;
  for (int k = threadIdx.x; k < a.K; k += TH) t.p[k] *= iz;  // the thread's own entries
  return true;
}

// A run of logits [j0, j1) of a row in 16-byte pieces: [j0, ja) and [jb, j1)
// are taken one by one, [ja, jb) in chunks of 8 from 16-byte boundaries.
struct Run {
  int64_t ja, jb;
};
__device__ __forceinline__ Run split_run(const char* row, int es, int64_t j0, int64_t j1) {
  const uint32_t off = (uint32_t)((uintptr_t)(row + j0 * es) & 15);
  int64_t ja = j0 + (off ? (16 - off) / es : 0);
  if (ja > j1) ja = j1;
  return Run{ja, ja + (j1 - ja) / 8 * 8};
}

// Running maximum (of the raw logits) and sum of exponentials of what a
// thread has seen; c = log2(e) / tau turns logits into exponents of two.
struct Soft {
  using Z = float;
  float m = kLowest, z = 0.f, inv, c;
  __host__ __device__ explicit Soft(float inv_tau) : inv(inv_tau), c(inv_tau * kLog2e) {}
  __device__ __forceinline__ void raise(float mn) {
    if (mn > m) {
      z *= ex2((m - mn) * c);
      m = mn;
    }
  }
  __device__ __forceinline__ void add1(float v) {
    raise(v);
    z += ex2((v - m) * c);
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float mn = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mn = fmaxf(mn, v[i]);
    raise(mn);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      s0 += ex2((v[i] - m) * c);
      s1 += ex2((v[i + 1] - m) * c);
    }
    z += s0 + s1;
  }
  __device__ __forceinline__ float sum() const { return z; }
  // exp((x - y) / tau)
  __device__ __forceinline__ float ratio(float x, float y) const { return ex2((x - y) * c); }
};

// The same for high temperatures: an error of 1e-7 in the sum is tau^2 times
// that in the loss, while the loss itself does not grow with tau.  There all
// exponentials are near 1, and what is summed (in float64) is their distance
// from it, e^d - 1 with d = (x - m) / tau, each off by a few 2^-24 |d| only: the
// loss is off by some tau 2^-22 times the logits' mean distance from their
// maximum.  m follows the maximum only where d would pass 1.
struct FineSoft {
  using Z = double;
  float m = kLowest, inv;
  int n = 0;
  double e = 0.0;
  __host__ __device__ explicit FineSoft(float inv_tau) : inv(inv_tau) {}
  __device__ __forceinline__ void raise(float mn) {
    if ((mn - m) * inv > 1.f || n == 0) {
      if (n) e += (e + n) * expm1(((double)m - (double)mn) * inv);
      m = fmaxf(mn, kLowest);
    }
  }
  // Taylor's series to d^10, whose rest is below 2^-24 of the value at |d| = 1
  __device__ __forceinline__ float dist(float v) const {
    const float d = (v - m) * inv;
    float r = 1.f / 3628800;
    r = fmaf(r, d, 1.f / 362880);
    r = fmaf(r, d, 1.f / 40320);
    r = fmaf(r, d, 1.f / 5040);
    r = fmaf(r, d, 1.f / 720);
    r = fmaf(r, d, 1.f / 120);
    r = fmaf(r, d, 1.f / 24);
    r = fmaf(r, d, 1.f / 6);
    r = fmaf(r, d, 0.5f);
    r = fmaf(d * d, r, d);
    return d < -1.f ? ex2(d * kLog2e) - 1.f : r;  // (a NaN stays one)
  }
  __device__ __forceinline__ void add1(float v) {
    raise(v);
    e += (double)dist(v);
    ++n;
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float mn = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mn = fmaxf(mn, v[i]);
    raise(mn);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      s0 += dist(v[i]);
      s1 += dist(v[i + 1]);
    }
    e += (double)(s0 + s1);
    n += N;
  }
  __device__ __forceinline__ double sum() const { return (double)n + e; }
  __device__ __forceinline__ double ratio(float x, float y) const {
    return exp(((double)x - (double)y) * inv);
  }
};

__device__ __forceinline__ float ld_cluster(uint32_t addr, float) { return ptx::ld_cluster_float(addr); }
__device__ __forceinline__ double ld_cluster(uint32_t addr, double) {
  return __hiloint2double(ptx::ld_cluster_int(addr + 4), ptx::ld_cluster_int(addr));
}

// Bound by HBM: 4096 x 131072 bf16 in 171-175 us, 6.2 TB/s (191 without the prefetch).
// One row per cluster: its CTAs divide the vocabulary and join their maxima
// and sums through distributed shared memory (one CTA: no join).
template <int BF, int TH, class SOFT>
__global__ void __launch_bounds__(TH, 1024 / TH)
distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kU = BF ? 4 : 2;  // chunks of 8 in flight per thread
  using Z = typename SOFT::Z;
  __shared__ Teacher<Z> t;
  __shared__ float red[2][TH / 32];
  __shared__ double redd[TH / 32];
  __shared__ Z redz[2][TH / 32];
  __shared__ float joinm;
  __shared__ Z joinz;
  uint32_t nct;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nct));
  const uint32_t rank = nct > 1 ? ptx::cluster_ctarank() : 0u;
  const int64_t row = blockIdx.x / nct;
  const char* s = reinterpret_cast<const char*>(a.S) + row * a.lds * (BF ? 2 : 4);
  const int64_t per = (a.V + nct - 1) / nct;
  const int64_t j0 = rank * per < a.V ? rank * per : a.V;
  const int64_t j1 = j0 + per < a.V ? j0 + per : a.V;
  const Run r = split_run(s, BF ? 2 : 4, j0, j1);
  SOFT f(a.inv_tau);
  int64_t j = r.ja + 8 * threadIdx.x;
  // kU chunks at a time, the next ones on their way while these are summed (the
  // first ones while the teacher's entries are)
  constexpr int kN = kU * (BF ? 1 : 2);
  constexpr int64_t kStep = (int64_t)8 * TH * kU;
  auto fetch = [&](uint4 (&raw)[kN], int64_t at) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint4* p = reinterpret_cast<const uint4*>(s + (at + 8 * TH * u) * (BF ? 2 : 4));
#pragma unroll
      for (int h = 0; h < kN / kU; ++h) raw[u * (kN / kU) + h] = __ldcs(p + h);
    }
  };
  auto whole = [&](int64_t at) { return at + 8 * TH * (kU - 1) < r.jb; };
  uint4 cur[kN];
  if (whole(j)) fetch(cur, j);
  float tm;
  Z tz;
  const bool any = teacher_probs<TH>(a, row, t, red[0], redz[0], &tm, &tz);  // as in the whole cluster
  if (!any) {
    if (threadIdx.x == 0 && rank == 0) {
      a.loss[row] = 0.f;
      a.lse[row] = 0.f;
    }
    return;
  }
  // the logit of the thread's first entry, needed last
  float at_entry = 0.f;
  if (threadIdx.x < a.K && t.idx[threadIdx.x] >= 0) at_entry = ld1(s, t.idx[threadIdx.x], BF);
  if (j0 + threadIdx.x < r.ja) f.add1(ld1(s, j0 + threadIdx.x, BF));
  while (whole(j)) {
    uint4 next[kN];
    if (whole(j + kStep)) fetch(next, j + kStep);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float v[8];
      if (BF) {
        unpack8(cur[u], v);
      } else {
        const uint4 x = cur[u * (kN / kU)], y = cur[u * (kN / kU) + kN / kU - 1];
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
        v[4] = __uint_as_float(y.x); v[5] = __uint_as_float(y.y);
        v[6] = __uint_as_float(y.z); v[7] = __uint_as_float(y.w);
      }
      f.add(v);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) cur[i] = next[i];
    j += kStep;
  }
  for (; j < r.jb; j += 8 * TH) {
    float v[8];
    ld8(s, j, BF, v);
    f.add(v);
  }
  if (r.jb + threadIdx.x < j1) f.add1(ld1(s, r.jb + threadIdx.x, BF));

  float M = block_fmax<TH>(f.m, red[1]);
  Z sum = block_fsum<TH>(f.sum() * f.ratio(f.m, M), redz[1]);
  if (nct > 1) {
    if (threadIdx.x == 0) {
      joinm = M;
      joinz = sum;
    }
    __syncwarp();
    ptx::cluster_sync();
    float m[8], mm = kLowest;
    Z z[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      m[p] = kLowest;
      z[p] = 0;
      if (p < (int)nct) {
        m[p] = ptx::ld_cluster_float(ptx::mapa(ptx::smem_u32(&joinm), p));
        z[p] = ld_cluster(ptx::mapa(ptx::smem_u32(&joinz), p), z[p]);
      }
      mm = fmaxf(mm, m[p]);
    }
    sum = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (p < (int)nct) sum += z[p] * f.ratio(m[p], mm);
    M = mm;
    __syncwarp();
    ptx::cluster_sync();  // everyone has read everyone's
    if (rank != 0) return;
  }
  // The few terms of the loss in float64: log p - log q cancels where the
  // student is near the teacher.  With both maxima and normalizers set apart,
  //   sum_k p_k (log p_k - log q_k) = sum_k p_k (t_k - tm - (s_k - M)) / tau + log(sum / tz)
  double acc = 0.0;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    const int i = t.idx[k];
    const double p = t.p[k];
    // below fp32's range p is 0, also where the student's logit is -inf
    if (i < 0 || (float)p == 0.f) continue;
    const float x = k == threadIdx.x ? at_entry : ld1(s, i, BF);
    acc += p * (((double)t.v[k] - (double)tm) - ((double)x - (double)M));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) redd[threadIdx.x >> 5] = acc;
  __syncthreads();
  const double inv = (double)a.inv_tau;
  if (threadIdx.x == 0) {
    for (int w = 1; w < TH / 32; ++w) acc += redd[w];
    const double kl = acc * inv + log((double)sum / (double)tz);
    a.loss[row] = (float)((double)a.tau * (double)a.tau * kl);
  }
  if (threadIdx.x == 32) a.lse[row] = (float)((double)M * inv + log((double)sum));
}

// Every CTA writes one segment of one row.  Bound by HBM: 4096 x 131072 bf16 in
// 361 us, 5.9 TB/s.
template <int BF, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH)
distill_bwd_kernel(const __grid_constant__ DistillArgs a, int64_t seg, int segs) {
  constexpr int kU = BF ? 4 : 2;
  __shared__ Teacher<float> t;
  __shared__ float sq[OUO_DISTILL_MAX_ENTRIES];
  __shared__ float red[2][TH / 32];
  const int64_t row = blockIdx.x / segs;
  const int64_t j0 = (blockIdx.x - row * segs) * seg;
  const int64_t j1 = j0 + seg < a.V ? j0 + seg : a.V;
  const float g = a.dloss[row] * a.tau, lse = a.lse[row];
  const char* s = reinterpret_cast<const char*>(a.S) + row * a.lds * (BF ? 2 : 4);
  char* d = reinterpret_cast<char*>(a.dS) + row * a.ldds * (a.ds_bf16 ? 2 : 4);
  float tm, tz;
  const bool any = g != 0.f && teacher_probs<TH>(a, row, t, red[0], red[1], &tm, &tz);
  // chunks that are 16-byte pieces of both matrices
  Run r = split_run(s, BF ? 2 : 4, j0, j1);
  if (((uintptr_t)d + r.ja * (a.ds_bf16 ? 2 : 4)) & 15) r.ja = r.jb = j0;
  // x / tau is not rounded before lse, of its size, is taken from it
  auto prob = [&](float x) { return ex2(fmaf(x, a.inv_tau, -lse) * kLog2e); };
  if (any) {
    // dS may be S itself: the entries' own probabilities are read first
    for (int k = threadIdx.x; k < a.K; k += TH) {
      const int i = t.idx[k];
      if (i >= j0 && i < j1) sq[k] = prob(ld1(s, i, BF));
    }
    __syncthreads();
    auto one = [&](int64_t j) { st1(d, j, g * prob(ld1(s, j, BF)), a.ds_bf16); };
    for (int64_t j = j0 + threadIdx.x; j < r.ja; j += TH) one(j);
    for (int64_t j = r.ja + 8 * threadIdx.x; j < r.jb; j += 8 * TH * kU) {
      uint4 raw[kU * (BF ? 1 : 2)];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t e = j + 8 * TH * u;
        if (e >= r.jb) break;
        const uint4* p = reinterpret_cast<const uint4*>(s + e * (BF ? 2 : 4));
        if (BF) {
          raw[u] = __ldcs(p);
        } else {
          raw[2 * u] = __ldcs(p);
          raw[2 * u + 1] = __ldcs(p + 1);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t e = j + 8 * TH * u;
        if (e >= r.jb) break;
        float v[8];
        if (BF) {
          unpack8(raw[u], v);
        } else {
          const uint4 x = raw[2 * u], y = raw[2 * u + 1];
          v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
          v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
          v[4] = __uint_as_float(y.x); v[5] = __uint_as_float(y.y);
          v[6] = __uint_as_float(y.z); v[7] = __uint_as_float(y.w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = g * prob(v[i]);
        st8(d, e, a.ds_bf16, v);
      }
    }
    for (int64_t j = r.jb + threadIdx.x; j < j1; j += TH) one(j);
    __syncthreads();
    // the first entry of each index takes every entry of that index
    const int4* i4 = reinterpret_cast<const int4*>(t.idx);
    for (int k = threadIdx.x; k < a.K; k += TH) {
      const int i = t.idx[k];
      if (i < j0 || i >= j1) continue;
      float p = 0.f;
      bool first = true;
      for (int l = 0; 4 * l < a.K; ++l) {
        const int4 x = i4[l];
        if (x.x != i && x.y != i && x.z != i && x.w != i) continue;
        const int e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (e[b] == i) {
            if (4 * l + b < k) first = false;
            p += t.p[4 * l + b];
          }
        if (!first) break;
      }
      if (first) st1(d, i, g * (sq[k] - p), a.ds_bf16);
    }
  } else {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t j = j0 + threadIdx.x; j < r.ja; j += TH) st1(d, j, 0.f, a.ds_bf16);
    for (int64_t j = r.ja + 8 * threadIdx.x; j < r.jb; j += 8 * TH) st8(d, j, a.ds_bf16, zero);
    for (int64_t j = r.jb + threadIdx.x; j < j1; j += TH) st1(d, j, 0.f, a.ds_bf16);
  }
}

// 128 threads a CTA rather than 256: for short runs of logits, where a row's
// barriers count (4096 x 8192 bf16: loss 31.7 -> 22.3 us, gradient 43.8 -> 32.1),
// and where the larger CTAs would fill the GPU between once and one and a half
// times (700 x 131072: 39.9 -> 36.6, 80.3 -> 68.7).  Else 256 keep more of a row
// on its way (gradient of 4096 x 131072: 359 us against 380).
bool small_blocks(int64_t logits, int64_t ctas) {
  return logits <= 16384 || (ctas > 4 * num_sms() && ctas < 6 * num_sms());
}

// Above it the loss sums with FineSoft.  A loss of 0.045 over 1000 logits, the
// teacher having all of them: 6e-5 of it off at tau = 4 with Soft, at tau = 8 /
// 100 / 1000 1e-6 / 2e-5 / 2e-4 with FineSoft (with Soft 2e-4 and more).  4096 x
// 131072 bf16: 171 us with Soft, 350-365 with FineSoft, bound by instructions.
constexpr float kFineTau = 4.f;

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
  OUO_TRY(validate_apart({operand(loss, S->rows, 4, "loss"), operand(lse, S->rows, 4, "lse")},
                         {operand(*S, (int64_t)elem_size(s_dtype), "S"),
                          operand(*teacher, (int64_t)elem_size(t_dtype), "teacher"),
                          operand(*idx, 4, "idx")}));
  DistillArgs a = distill_args(S, s_dtype, teacher, t_dtype, idx, temperature);
  a.loss = loss;
  a.lse = lse;
  // Few rows: a cluster per row, as long as all CTAs are resident together; a
  // CTA keeps at least 4096 logits.
  unsigned cluster = 1;
  while (cluster < 8 && a.rows * 2 * cluster <= 4 * num_sms() && a.V / (2 * cluster) >= 4096) cluster *= 2;
  if (a.rows * cluster > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "S: too many rows");
  const bool small = small_blocks(ceil_div(a.V, (int64_t)cluster), a.rows * cluster);
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(a.rows * cluster), 1, 1);
  cfg.blockDim = dim3(small ? 128 : 256, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto choose = [&](auto soft) {
    using S = decltype(soft);
    return a.s_bf16 ? (small ? distill_kernel<1, 128, S> : distill_kernel<1, 256, S>)
                    : (small ? distill_kernel<0, 128, S> : distill_kernel<0, 256, S>);
  };
  auto kern = temperature > kFineTau ? choose(FineSoft(1.f)) : choose(Soft(1.f));
  OUO_CHECK_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
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
  OUO_TRY(validate_in_place(*dS, ds_dtype, *S, s_dtype, "dS and S"));
  OUO_TRY(validate_vec(lse, S->rows, 4, "lse"));
  OUO_TRY(validate_vec(dloss, S->rows, 4, "dloss"));
  if (S->rows == 0) return OUO_OK;
  OUO_TRY(require_sm100());
  OUO_TRY(validate_apart({operand(*dS, (int64_t)elem_size(ds_dtype), "dS", S->ptr)},
                         {operand(*S, (int64_t)elem_size(s_dtype), "S"),
                          operand(*teacher, (int64_t)elem_size(t_dtype), "teacher"),
                          operand(*idx, 4, "idx"), operand(lse, S->rows, 4, "lse"),
                          operand(dloss, S->rows, 4, "dloss")}));
  DistillArgs a = distill_args(S, s_dtype, teacher, t_dtype, idx, temperature);
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dS = dS->ptr; a.ldds = dS->ld; a.ds_bf16 = ds_dtype == OUO_BF16;
  // Few rows are cut into segments, as many as are resident together, of 2048
  // logits at least.
  int64_t segs = (int64_t)4 * num_sms() / a.rows;
  if (segs > a.V / 2048) segs = a.V / 2048;
  if (segs < 1) segs = 1;
  const int64_t seg = ceil_div(ceil_div(a.V, segs), (int64_t)8) * 8;
  segs = ceil_div(a.V, seg);
  if (a.rows * segs > 0x7fffffff) return set_error(OUO_ERR_UNSUPPORTED, "S: too many rows");
  const unsigned grid = (unsigned)(a.rows * segs);
  cudaStream_t s = (cudaStream_t)stream;
  const bool small = small_blocks(seg, a.rows * segs);
  auto kern = a.s_bf16 ? (small ? distill_bwd_kernel<1, 128> : distill_bwd_kernel<1, 256>)
                       : (small ? distill_bwd_kernel<0, 128> : distill_bwd_kernel<0, 256>);
  kern<<<grid, small ? 128 : 256, 0, s>>>(a, seg, (int)segs);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

}  // extern "C"
