// rms_norm and rms_norm_backward: the root-mean-square norm in front of a
// product, with the residual's addition and an 8-bit output.
//
//   h = x + residual (rounded to H's type),  r = 1 / sqrt(mean(h^2) + eps),
//   y = h r w;   8-bit output: q = rint(y / scale), scale = max |y| / 127
//   dx = dh + r (w dy - h r^2 mean(w dy h)),  dw = sum over rows of dy h r
//
// HBM-bound: every matrix is read or written once.
#include "tokens.cuh"
#include "umma.cuh"

namespace ouo {
namespace {

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
  int vx, vr, vh, vw, vy, vq;  // 16-byte (vq: 8-byte) accesses allowed
};

__device__ __forceinline__ const char* row_of(const void* p, int64_t r, int64_t ld, int bf16) {
  return reinterpret_cast<const char*>(p) + r * ld * (bf16 ? 2 : 4);
}

// A team per row, h in registers (as the values that H's type holds): x and
// the residual are read once, and nothing is read back.  Bound by HBM: 16384 x
// 4096 bf16 with residual and 8-bit output in 71 us, 73 under a long load that
// lowers the clock (6.6, 6.4 TB/s); with types asked for at run time it was 92
// us, bound by instructions.
template <int TPR, int NV, int MODE>
__global__ void __launch_bounds__(kTeamThreads<TPR>) rms_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kWarps = kTeamThreads<TPR> / 32, kTeams = kTeamThreads<TPR> / TPR;
  __shared__ float reds[kWarps];
  __shared__ uint32_t redm[kWarps];
  const int64_t row = (int64_t)blockIdx.x * kTeams + (kTeams > 1 ? threadIdx.x / TPR : 0);
  if (kTeams > 1 && row >= a.rows) return;
  const int t = threadIdx.x % TPR, n = (int)a.cols;
  constexpr int XM = MODE == 5 ? 1 : MODE, HM = MODE == 5 ? 2 : MODE;  // x and y, residual and h
  const int xb = MODE ? XM == 1 || XM == 3 : a.x_bf16, yb = MODE ? xb : a.y_bf16;
  const int hb = MODE ? HM == 1 || HM == 3 : a.h_bf16;
  RowRaw<TPR, NV, XM> xr;
  RowRaw<TPR, NV, HM> rr;
  float v[NV][8];
  xr.load(row_of(a.X, row, a.ldx, xb), t, n, xb, a.vx);
  if (a.R) {
    rr.load(row_of(a.R, row, a.ldr, hb), t, n, hb, a.vr);
    xr.get(v);
    float u[NV][8];
    rr.get(u);
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += u[c][i];
  } else {
    xr.get(v);
  }
  if (a.H) {
    char* h = const_cast<char*>(row_of(a.H, row, a.ldh, hb));
    if (HM == 1) {
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const uint4 u = pack8(v[c]);
        if (8 * (t + c * TPR) < n) reinterpret_cast<uint4*>(h)[t + c * TPR] = u;
        unpack8(u, v[c]);
      }
    } else {
      store_row<TPR, NV, HM>(h, t, n, hb, a.vh, v);
      if (HM == 0 || HM == 3) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = round_to(v[c][i], hb);
      }
    }
  }
  float acc = 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(v[c][i], v[c][i], acc);
  // a weight of x's type is on its way while the squares are summed
  RowRaw<TPR, NV, XM> wr;
  const bool same = MODE == 0 || a.w_bf16 == xb;
  if (same) wr.load(a.W, t, n, a.w_bf16, a.vw);
  const float rstd = __frsqrt_rn(team_sum<TPR>(acc, reds) / (float)n + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  float m = 0.f;
  {
    float w[NV][8];
    if (same) {
      wr.get(w);
    } else {
      RowRaw<TPR, NV, kOtherType<XM>> other;
      other.load(a.W, t, n, a.w_bf16, a.vw);
      other.get(w);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = v[c][i] * rstd * w[c][i];
        m = max_mag(m, v[c][i]);
      }
  }
  if (a.Y)
    store_row<TPR, NV, XM>(const_cast<char*>(row_of(a.Y, row, a.ldy, yb)), t, n, yb, a.vy, v);
  if (!a.Q) return;
  const Quant q = quant_of<0>(team_max<TPR>(__float_as_uint(m), redm));
  if (t == 0) a.scale[row] = q.scale;
  store_q<TPR, NV, XM>(a.Q + row * a.ldq, t, n, a.vq, v, q);
}

// Rows too long for registers: one block per row; h is read back (from H, or
// from X when there is none) for each of the later passes.  2048 x 20000 bf16,
// residual, 8 bits: 84 us, 3.4 TB/s of what it has to move.
__global__ void __launch_bounds__(512) rms_long_kernel(const __grid_constant__ NormArgs a) {
  __shared__ uint32_t red[32];
  const int n = (int)a.cols;
  const int64_t row = blockIdx.x;
  const char* x = row_of(a.X, row, a.ldx, a.x_bf16);
  const char* rs = a.R ? row_of(a.R, row, a.ldr, a.h_bf16) : nullptr;
  char* h = a.H ? const_cast<char*>(row_of(a.H, row, a.ldh, a.h_bf16)) : nullptr;
  float acc = 0.f;
  for (int j = 8 * threadIdx.x; j < n; j += 8 * 512) {
    float v[8], u[8];
    row_ld8(x, j, n, a.x_bf16, a.vx, v);
    if (rs) {
      row_ld8(rs, j, n, a.h_bf16, a.vr, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    if (h) row_st8(h, j, n, a.h_bf16, a.vh, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (h) v[i] = round_to(v[i], a.h_bf16);
      acc = fmaf(v[i], v[i], acc);
    }
  }
  const float rstd = __frsqrt_rn(block_sum(acc, reinterpret_cast<float*>(red)) / (float)n + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  auto value = [&](int j, float v[8]) {
    float w[8];
    if (h) row_ld8(h, j, n, a.h_bf16, a.vh, v);
    else row_ld8(x, j, n, a.x_bf16, a.vx, v);
    row_ld8(a.W, j, n, a.w_bf16, a.vw, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * w[i];
  };
  float m = 0.f;
  for (int j = 8 * threadIdx.x; j < n; j += 8 * 512) {
    float v[8];
    value(j, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_mag(m, v[i]);
    if (a.Y)
      row_st8(const_cast<char*>(row_of(a.Y, row, a.ldy, a.y_bf16)), j, n, a.y_bf16, a.vy, v);
  }
  if (!a.Q) return;
  const Quant q = quant_of<0>(block_max(__float_as_uint(m), red));
  if (threadIdx.x == 0) a.scale[row] = q.scale;
  for (int j = 8 * threadIdx.x; j < n; j += 8 * 512) {
    float v[8];
    value(j, v);
    row_stq(a.Q + row * a.ldq, j, n, a.vq, quant8(v, q));
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
  int vdy, vh, vw, vdh, vdx, vpart;  // 16-byte accesses allowed
};

// The mode of each matrix (see RowRaw), and the 16-byte pieces of its chunks.
template <int MODE>
struct BwdModes {
  static constexpr int kDy = MODE == 5 ? 1 : MODE, kH = MODE == 5 ? 2 : MODE,
                       kDx = MODE == 5 ? 2 : MODE;
  static constexpr bool kRing = MODE == 1 || MODE == 2 || MODE == 5;
  static constexpr int kU0 = kDy == 2 ? 2 : 1, kU1 = kH == 2 ? 2 : 1, kU2 = kDx == 2 ? 2 : 1;
  static constexpr int kUnits = kU0 + kU1 + kU2;
};

// Blocks of the gradient that an SM holds at once, by the chunks of 8 columns
// that a block takes: what the grid counts on, so the registers are bounded to it
// (8000 x 4095 bf16: 153 us with a register too many, 90 with two blocks).
constexpr int bwd_blocks(int chunks) {
  return chunks <= 128 ? 7 : chunks <= 256 ? 4 : chunks <= 512 ? 2 : 1;
}

// A block of TPR threads takes rows b, b + grid, ...; every thread keeps the
// same columns of all of them, so that its share of dw stays in registers and
// leaves once, to row b of the partial sums.  In modes 1, 2 and 5 DEPTH rows of dY,
// H and dH are on their way to shared memory (cp.async, to slots that only the
// copying warp reads, so without block barriers), since the reduction of a row
// would otherwise leave the memory idle (16384 x 4096 bf16: 180 us without, 88 us
// with it and with 16 elements a thread; HBM-bound at 6.1 TB/s).
template <int TPR, int NV, int MODE, int DEPTH>
__global__ void __launch_bounds__(TPR, bwd_blocks(TPR * NV))
rms_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  __shared__ float red[2][TPR / 32];
  using M = BwdModes<MODE>;
  extern __shared__ __align__(16) uint4 ring[];  // [DEPTH][NV][dY, H, dH][TPR pieces a unit]
  const int t = threadIdx.x, n = (int)a.cols;
  const int dyb = MODE ? M::kDy == 1 || M::kDy == 3 : a.dy_bf16;
  const int hb = MODE ? M::kH == 1 || M::kH == 3 : a.h_bf16;
  const int dxb = MODE ? M::kDx == 1 || M::kDx == 3 : a.dx_bf16;
  float w[NV][8], dw[NV][8];
  if (MODE == 3 || MODE == 4) {
    if (a.w_bf16) {
      RowRaw<TPR, NV, 3> wr;
      wr.load(a.W, t, n, 1, 0);
      wr.get(w);
    } else {
      RowRaw<TPR, NV, 4> wr;
      wr.load(a.W, t, n, 0, 0);
      wr.get(w);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c) row_ld8(a.W, 8 * (t + c * TPR), n, a.w_bf16, a.vw, w[c]);
  }
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  const char* src[3] = {row_of(a.dY, blockIdx.x, a.lddy, dyb), row_of(a.H, blockIdx.x, a.ldh, hb),
                        a.dH ? row_of(a.dH, blockIdx.x, a.lddh, dxb) : nullptr};
  const int64_t step[3] = {a.lddy * (dyb ? 2 : 4) * gridDim.x, a.ldh * (hb ? 2 : 4) * gridDim.x,
                           a.lddh * (dxb ? 2 : 4) * gridDim.x};
  // slots of stage, chunk and matrix, in 16-byte pieces of the team
  auto slot = [&](int stage, int c, int before) {
    return ring + ((stage * NV + c) * M::kUnits + before) * TPR;
  };
  auto issue = [&](int64_t row, int stage) {
    if (row < a.rows) {
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        if (m == 2 && !a.dH) break;
        const int units = m == 0 ? M::kU0 : m == 1 ? M::kU1 : M::kU2;
        const int before = m == 0 ? 0 : m == 1 ? M::kU0 : M::kU0 + M::kU1;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
#pragma unroll
          for (int u = 0; u < units; ++u) {
            // a warp's copies of one instruction are 512 bytes in a row, so
            // with fp32 a lane's pieces are copied by other lanes of its warp
            const int piece = (t & ~31) * units + u * 32 + (t & 31);
            if ((units == 2 ? 4 : 8) * (c * TPR * units + piece) < n)
              ptx::copy16(slot(stage, c, before) + piece, src[m] + (c * TPR * units + piece) * 16);
          }
        }
        src[m] += step[m];
      }
    }
    ptx::copy16_commit();
  };
  auto fetch = [&](auto& r, int stage, int before, auto units) {
    constexpr int kU = decltype(units)::value;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const bool in = 8 * (t + c * TPR) < n;
      const uint4* q = slot(stage, c, before) + t * kU;
      r.a[c] = in ? q[0] : make_uint4(0, 0, 0, 0);
      if constexpr (kU == 2) r.b[c] = in ? q[1] : make_uint4(0, 0, 0, 0);
    }
  };
  int64_t ahead = blockIdx.x;
  if constexpr (M::kRing) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s, ahead += gridDim.x) issue(ahead, s);
  }
  float r_next = blockIdx.x < a.rows ? a.rstd[blockIdx.x] : 0.f;
  const float inv_n = 1.f / (float)n;
  char* dx = const_cast<char*>(row_of(a.dX, blockIdx.x, a.lddx, dxb));
  const int64_t dx_step = a.lddx * (dxb ? 2 : 4) * gridDim.x;
  int flip = 0, stage = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1, dx += dx_step) {
    const float r = r_next;
    if (row + gridDim.x < a.rows) r_next = a.rstd[row + gridDim.x];
    float g[NV][8], h[NV][8];
    RowRaw<TPR, NV, M::kDx> dr;
    {
      RowRaw<TPR, NV, M::kDy> gr;
      RowRaw<TPR, NV, M::kH> hr;
      if constexpr (M::kRing) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        if (MODE != 1) __syncwarp();
        fetch(gr, stage, 0, C<M::kU0>{});
        fetch(hr, stage, M::kU0, C<M::kU1>{});
        if (a.dH) fetch(dr, stage, M::kU0 + M::kU1, C<M::kU2>{});
      } else {
        gr.load(row_of(a.dY, row, a.lddy, dyb), t, n, dyb, a.vdy);
        hr.load(row_of(a.H, row, a.ldh, hb), t, n, hb, a.vh);
        if (a.dH) dr.load(row_of(a.dH, row, a.lddh, dxb), t, n, dxb, a.vdh);
      }
      gr.get(g);
      hr.get(h);
    }
    float acc = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[c][i] *= r;
        dw[c][i] = fmaf(g[c][i], h[c][i], dw[c][i]);
        g[c][i] *= w[c][i];
        acc = fmaf(g[c][i], h[c][i], acc);
      }
    // r (g - h m) + dh, with r m once per row
    const float rm = team_sum<TPR>(acc, red[flip]) * inv_n * r;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) g[c][i] = fmaf(g[c][i], r, -(h[c][i] * rm));
    if (a.dH) {
      dr.get(h);
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] += h[c][i];
    }
    if constexpr (M::kRing) {  // this stage's values are in registers
      if (MODE != 1) __syncwarp();
      issue(ahead, stage);
      ahead += gridDim.x;
      if (++stage == DEPTH) stage = 0;
    }
    store_row<TPR, NV, M::kDx>(dx, t, n, dxb, a.vdx, g);
  }
  if (M::kRing) ptx::copy16_wait_all();
  if (a.part) {
    float* part = a.part + blockIdx.x * a.cols;
    if (MODE == 3 || MODE == 4) {
      store_row<TPR, NV, 4>(part, t, n, 0, 0, dw);
    } else {
#pragma unroll
      for (int c = 0; c < NV; ++c)
        row_st8(part, 8 * (t + c * TPR), n, 0, a.vpart, dw[c]);
    }
  }
}

// Rows too long for registers: dw's shares stay in the partial sums, where
// each thread adds to its own columns.  Bound by the latency of its single-
// element accesses: 4096 x 16384 bf16 in 1.08 ms, 0.5 TB/s.
__global__ void __launch_bounds__(512) rms_bwd_long_kernel(const __grid_constant__ NormBwdArgs a) {
  __shared__ uint32_t red[32];
  const int n = (int)a.cols;
  float* part = a.part ? a.part + blockIdx.x * a.cols : nullptr;
  if (part)
    for (int j = threadIdx.x; j < n; j += 512) part[j] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* dy = row_of(a.dY, row, a.lddy, a.dy_bf16);
    const char* h = row_of(a.H, row, a.ldh, a.h_bf16);
    const char* dh = a.dH ? row_of(a.dH, row, a.lddh, a.dx_bf16) : nullptr;
    char* dx = const_cast<char*>(row_of(a.dX, row, a.lddx, a.dx_bf16));
    const float r = a.rstd[row];
    float acc = 0.f;
    for (int j = threadIdx.x; j < n; j += 512) {
      const float g = ld1(dy, j, a.dy_bf16), xh = ld1(h, j, a.h_bf16) * r;
      acc = fmaf(g * ld1(a.W, j, a.w_bf16), xh, acc);
      if (part) part[j] = fmaf(g, xh, part[j]);
    }
    const float c = block_sum(acc, reinterpret_cast<float*>(red)) / (float)n;
    for (int j = threadIdx.x; j < n; j += 512) {
      const float g = ld1(dy, j, a.dy_bf16) * ld1(a.W, j, a.w_bf16);
      float v = r * (g - ld1(h, j, a.h_bf16) * r * c);
      if (dh) v += ld1(dh, j, a.dx_bf16);
      st1(dx, j, v, a.dx_bf16);
    }
  }
}

// dw = sum of the partial rows, in a fixed order: 16 threads a column, each
// every 16th row, then their sums.
__global__ void __launch_bounds__(512)
rms_dw_kernel(const float* part, int nparts, int64_t cols, float* dw) {
  __shared__ float sum[16][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (j < cols)
    for (int p = w; p < nparts; p += 16) v += part[p * cols + j];
  sum[w][lane] = v;
  __syncthreads();
  if (w == 0 && j < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) v += sum[i][lane];
    dw[j] = v;
  }
}

template <int TPR, int NV, int MODE, int DEPTH>
int launch_bwd_as(const NormBwdArgs& a, unsigned grid, cudaStream_t s) {
  using M = BwdModes<MODE>;
  constexpr size_t kSmem = M::kRing ? (size_t)DEPTH * M::kUnits * NV * TPR * 16 : 0;
  if (kSmem > 40 * 1024) {  // with the static part, past the default limit
    static Once once;
    OUO_TRY(once.smem(rms_bwd_kernel<TPR, NV, MODE, DEPTH>, kSmem));
  }
  rms_bwd_kernel<TPR, NV, MODE, DEPTH><<<grid, TPR, kSmem, s>>>(a);
  OUO_CHECK_LAUNCH();
  return OUO_OK;
}

// All matrices in 16-byte accesses; and not all.
template <int TPR, int NV>
int launch_bwd_vec(const NormBwdArgs& a, unsigned grid, cudaStream_t s) {
  const int bf = a.dy_bf16 + a.h_bf16 + a.dx_bf16;
  if (bf == 1 && a.dy_bf16) return launch_bwd_as<TPR, NV, 5, 2>(a, grid, s);
  if (bf == 3) return launch_bwd_as<TPR, NV, 1, 4>(a, grid, s);
  if (bf == 0) return launch_bwd_as<TPR, NV, 2, 2>(a, grid, s);
  return launch_bwd_as<TPR, NV, 0, 1>(a, grid, s);
}

template <int TPR, int NV>
int launch_bwd_elem(const NormBwdArgs& a, unsigned grid, cudaStream_t s) {
  const int bf = a.dy_bf16 + a.h_bf16 + a.dx_bf16;
  if (bf == 3) return launch_bwd_as<TPR, NV, 3, 1>(a, grid, s);
  if (bf == 0) return launch_bwd_as<TPR, NV, 4, 1>(a, grid, s);
  return launch_bwd_as<TPR, NV, 0, 1>(a, grid, s);
}

// Blocks of the gradient, and rows of partial sums of dw: what 148 SMs hold
// at once; one for a few tokens, whose sums are dw then, without a second
// launch.  A function of the shape alone, so that the workspace query needs no
// device.
int64_t bwd_parts(int64_t rows, int64_t cols) {
  if (rows > 0 && rows <= 8 && rows * cols <= 16384) return 1;
  const int64_t most = 148 * bwd_blocks((int)(cols < 8192 ? ceil_div(cols, (int64_t)8) : 1024));
  return rows < most ? rows : most;
}

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
    OUO_TRY(validate_in_place(*H, h_dtype, *X, x_dtype, "H and X"));
  }
  if (residual) {
    OUO_TRY(validate_tokens(*residual, elem_size(h_dtype), "residual", 0));
    OUO_TRY(validate_shape(*residual, T, n, "residual", 0));
    OUO_TRY(validate_in_place(*H, h_dtype, *residual, h_dtype, "H and residual"));
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
  if (Y && !Q) OUO_TRY(validate_in_place(*Y, y_dtype, *X, x_dtype, "Y and X"));
  if (T == 0) return OUO_OK;
  OUO_TRY(require_sm100());
  {
    const ouo_mat none{};
    const int64_t hs = residual || H ? (int64_t)elem_size(h_dtype) : 1;
    OUO_TRY(validate_apart(
        {operand(H ? *H : none, hs, "H", X->ptr, residual ? residual->ptr : nullptr),
         operand(Y ? *Y : none, Y ? (int64_t)elem_size(y_dtype) : 1, "Y", Q ? nullptr : X->ptr),
         operand(Q ? *Q : none, 1, "Q"), operand(Q ? scale : nullptr, T, 4, "scale"),
         operand(rstd, T, 4, "rstd")},
        {operand(*X, (int64_t)elem_size(x_dtype), "X"),
         operand(residual ? *residual : none, hs, "residual"),
         operand(weight, n, (int64_t)elem_size(w_dtype), "weight")}));
  }
  NormArgs a{};
  a.X = X->ptr; a.ldx = X->ld; a.x_bf16 = x_dtype == OUO_BF16;
  if (residual) { a.R = residual->ptr; a.ldr = residual->ld; }
  if (H) { a.H = H->ptr; a.ldh = H->ld; a.h_bf16 = h_dtype == OUO_BF16; }
  a.W = weight; a.w_bf16 = w_dtype == OUO_BF16;
  if (Y) { a.Y = Y->ptr; a.ldy = Y->ld; a.y_bf16 = y_dtype == OUO_BF16; }
  if (Q) { a.Q = (int8_t*)Q->ptr; a.ldq = Q->ld; a.scale = scale; }
  a.rstd = rstd;
  a.rows = T; a.cols = n; a.eps = eps;
  a.vx = rows16(*X, elem_size(x_dtype));
  a.vr = residual ? rows16(*residual, elem_size(h_dtype)) : 0;
  a.vh = H ? rows16(*H, elem_size(h_dtype)) : 0;
  a.vw = (uintptr_t)weight % 16 == 0;
  a.vy = Y ? rows16(*Y, elem_size(y_dtype)) : 0;
  a.vq = Q ? (uintptr_t)a.Q % 8 == 0 && (T <= 1 || a.ldq % 8 == 0) : 0;
  cudaStream_t s = (cudaStream_t)stream;
  const bool vec = a.vx && a.vw && (!a.R || a.vr) && (!a.H || a.vh) && (!a.Y || a.vy) && n % 8 == 0;
  auto all = [&](int dt, int hdt) {
    return x_dtype == dt && (!H || h_dtype == hdt) && (!Y || y_dtype == dt);
  };
  const int mode = all(OUO_BF16, OUO_BF16) ? (vec ? 1 : 3)
                   : all(OUO_F32, OUO_F32) ? (vec ? 2 : 4)
                   : all(OUO_BF16, OUO_F32) && vec ? 5 : 0;
  const Team t = team_for(T, n, mode);
  if (t.tpr == 0) {
    rms_long_kernel<<<(unsigned)T, 512, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
    return OUO_OK;
  }
  return with_team(t, mode, [&](auto tpr, auto nv, auto md) -> int {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int MODE = decltype(md)::value;
    constexpr int kTeams = kTeamThreads<TPR> / TPR;
    rms_kernel<TPR, NV, MODE><<<(unsigned)ceil_div(T, (int64_t)kTeams), kTeamThreads<TPR>, 0, s>>>(a);
    OUO_CHECK_LAUNCH();
    return OUO_OK;
  });
}

size_t rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  const int64_t parts = ouo::bwd_parts(rows, cols);
  return parts > 1 ? (size_t)(parts * cols) * sizeof(float) : 0;
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
  OUO_TRY(validate_in_place(*dX, dx_dtype, *dY, dy_dtype, "dX and dY"));
  if (dH) OUO_TRY(validate_in_place(*dX, dx_dtype, *dH, dx_dtype, "dX and dH"));
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
  {
    const ouo_mat none{};
    const int64_t xs = (int64_t)elem_size(dx_dtype);
    OUO_TRY(validate_apart(
        {operand(*dX, xs, "dX", dY->ptr, dH ? dH->ptr : nullptr), operand(dweight, n, 4, "dweight")},
        {operand(*dY, (int64_t)elem_size(dy_dtype), "dY"),
         operand(*H, (int64_t)elem_size(h_dtype), "H"), operand(dH ? *dH : none, xs, "dH"),
         operand(weight, n, (int64_t)elem_size(w_dtype), "weight"), operand(rstd, T, 4, "rstd")}));
  }
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t parts = bwd_parts(T, n);
  if (T > 0) {
    NormBwdArgs a{};
    a.dY = dY->ptr; a.lddy = dY->ld; a.dy_bf16 = dy_dtype == OUO_BF16;
    a.H = H->ptr; a.ldh = H->ld; a.h_bf16 = h_dtype == OUO_BF16;
    a.W = weight; a.w_bf16 = w_dtype == OUO_BF16;
    a.rstd = rstd;
    if (dH) { a.dH = dH->ptr; a.lddh = dH->ld; }
    a.dX = dX->ptr; a.lddx = dX->ld; a.dx_bf16 = dx_dtype == OUO_BF16;
    a.part = !dweight ? nullptr : parts == 1 ? dweight : (float*)ws;
    a.vpart = (uintptr_t)a.part % 16 == 0 && n % 4 == 0;
    a.rows = T; a.cols = n;
    a.vdy = rows16(*dY, elem_size(dy_dtype));
    a.vh = rows16(*H, elem_size(h_dtype));
    a.vw = (uintptr_t)weight % 16 == 0;
    a.vdh = dH ? rows16(*dH, elem_size(dx_dtype)) : 0;
    a.vdx = rows16(*dX, elem_size(dx_dtype));
    const unsigned grid = (unsigned)parts;
    const bool vec = a.vdy && a.vh && a.vdx && (a.vdh || !dH) && n % 8 == 0;
    if (n <= 128 * 8)
      OUO_TRY((vec ? launch_bwd_vec<128, 1> : launch_bwd_elem<128, 1>)(a, grid, s));
    else if (n <= 512 * 8 && !vec) OUO_TRY((launch_bwd_elem<512, 1>(a, grid, s)));
    else if (n <= 128 * 16) OUO_TRY((launch_bwd_vec<128, 2>(a, grid, s)));
    else if (n <= 256 * 16) OUO_TRY((launch_bwd_vec<256, 2>(a, grid, s)));
    else if (n <= 512 * 16)
      OUO_TRY((vec ? launch_bwd_vec<512, 2> : launch_bwd_elem<512, 2>)(a, grid, s));
    else {
      rms_bwd_long_kernel<<<grid, 512, 0, s>>>(a);
      OUO_CHECK_LAUNCH();
    }
  }
  if (dweight && n > 0 && parts != 1) {
    rms_dw_kernel<<<(unsigned)ceil_div(n, 32), 512, 0, s>>>((const float*)ws, (int)parts, n,
                                                             dweight);
    OUO_CHECK_LAUNCH();
  }
  return OUO_OK;
}

}  // extern "C"
