// norm.cu -- layer norm of rows, forward and backward.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r,
//   y = xh w + b;
//   with g = dy w:  dx = r (g - mean(g) - xh mean(g xh)),
//                   dw = sum_rows dy xh,  db = sum_rows dy.
//
// Both passes are bound by memory: every element is read once and written
// once.  A group of threads holds a whole row in registers, so the variance
// is taken from the centred values (no cancellation) without reading the row
// again.  The backward's blocks are persistent: a thread keeps its columns
// through all its rows, adds dw and db in registers, and a second kernel joins
// the blocks' sums in block order in fp64 (no float atomic).
//
// Measured on B200 (L2 flushed): 1.5M rows of 128, fp32 to bf16, forward 187 us
// (6.2 TB/s), backward 308 us (6.2 TB/s); 16384 rows of 4096 bf16, forward 60 us
// (4.5 TB/s; instructions issue in 40 % of the cycles: 16 warps an SM with no row
// fetched ahead leave latency), backward 91 us (4.4 TB/s; issue 63 %, two sums a
// column kept in registers leave 16 warps an SM).
#include <algorithm>
#include <atomic>

#include "tc.cuh"

namespace recis {

namespace {

constexpr int kMaxRowThreads = 512;   // a block of the kernels that hold a row
constexpr int kWideThreads = 1024;    // a block of the kernels that read a row again

struct NormParams {
  const void* x;
  const void* w;
  const void* b;
  const void* gy;
  void* y;          // forward: y; backward: grad_x (or NULL)
  float* mean;      // forward: written (or NULL); backward: read
  float* rstd;
  float* partial;   // backward: [blocks][2][D] (or NULL)
  int64_t M, x_stride, gy_stride, y_stride;
  int D, units, tpr;  // tpr: threads a row
  int w_type;
  float eps;
};

__device__ __forceinline__ float param_at(const void* p, int type, int i) {
  if (type == RECIS_F32) return __ldg(static_cast<const float*>(p) + i);
  if (type == RECIS_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

template <int VEC>
__device__ __forceinline__ void param_vec(const void* p, int type, int c, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    if (type == RECIS_F32) {
      RawVec<float, 8> r;
      r.load(static_cast<const float*>(p) + c);
      r.unpack(f);
    } else if (type == RECIS_BF16) {
      RawVec<__nv_bfloat16, 8> r;
      r.load(static_cast<const __nv_bfloat16*>(p) + c);
      r.unpack(f);
    } else {
      RawVec<__half, 8> r;
      r.load(static_cast<const __half*>(p) + c);
      r.unpack(f);
    }
  }
}

// VEC parameters from column c on (`none` where the array is NULL)
template <int VEC>
__device__ __forceinline__ void load_params(const void* p, int type, int c, float none, float (&f)[VEC]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = none;
    return;
  }
  if (VEC == 8 && ((uintptr_t)p & 15) == 0) {
    param_vec(p, type, c, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = param_at(p, type, c + j);
}

// Sum of v over the tpr threads of the caller's row; every thread gets it.
// tpr <= 32: shuffles within the warp; more: tpr is a multiple of 32, and every
// thread of the block calls (`s` alternates between calls, so one barrier a
// call suffices).
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float (*s)[32]) {
  const int top = tpr < 32 ? tpr : 32;
  for (int off = top >> 1; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[k][w] = v[k];
    __syncthreads();
    const int nw = tpr >> 5, w0 = w / nw * nw;  // the row's warps
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = s[k][w0] + s[k][w0 + 1];
      for (int q = 2; q < nw; q += 2) {
        const float2 f = *reinterpret_cast<const float2*>(&s[k][w0 + q]);
        t += f.x + f.y;
      }
      v[k] = t;
    }
  }
}

// 1 / sqrt(x): the approximation and one Newton step (relative error below 2^-22)
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return isinf(r) || r == 0.f ? r : r * fmaf(-0.5f * x * r, r, 1.5f);  // 0 and infinity as they are
}

// Arithmetic on a thread's VEC columns, two at an instruction where there are 8.
template <int VEC>
__device__ __forceinline__ float vec_sum(const float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const float2 a = add2(add2(make_float2(f[0], f[1]), make_float2(f[2], f[3])),
                          add2(make_float2(f[4], f[5]), make_float2(f[6], f[7])));
    return a.x + a.y;
  } else {
    return f[0];
  }
}
// f -= mu; the sum of its squares
template <int VEC>
__device__ __forceinline__ float vec_center(float (&f)[VEC], float mu) {
  if constexpr (VEC == 8) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 d = add2(make_float2(f[j], f[j + 1]), make_float2(-mu, -mu));
      s = fma2(d, d, s);
      f[j] = d.x;
      f[j + 1] = d.y;
    }
    return s.x + s.y;
  } else {
    f[0] -= mu;
    return f[0] * f[0];
  }
}
// f r w + b
template <int VEC>
__device__ __forceinline__ void vec_affine(float (&f)[VEC], float r, const float (&w)[VEC], const float (&b)[VEC]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 d = fma2(mul2(make_float2(f[j], f[j + 1]), make_float2(r, r)), make_float2(w[j], w[j + 1]),
                            make_float2(b[j], b[j + 1]));
      f[j] = d.x;
      f[j + 1] = d.y;
    }
  } else {
    f[0] = fmaf(f[0] * r, w[0], b[0]);
  }
}
// Weight and bias of a thread's columns: in registers through all rows where a
// thread has few columns, else in shared memory as fp32 (the block's copy), so
// that the registers go to more rows an SM.
template <int VEC, int UPT, int N>
struct Params {
  static constexpr bool kKeep = UPT * VEC <= 8;
  float f[kKeep ? N : 1][kKeep ? UPT : 1][VEC];
  const float* s;
  // the block's threads all call; `s`: [N][D] floats
  __device__ __forceinline__ void init(const NormParams& p, float* s, int lane) {
    this->s = s;
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < UPT; ++k) {
        const int c = lane + k * p.tpr;
        if (c < p.units) {
          load_params(p.w, p.w_type, c * VEC, 1.0f, f[0][k]);
          if constexpr (N == 2) load_params(p.b, p.w_type, c * VEC, 0.0f, f[1][k]);
        }
      }
    } else {
      // a vector's halves lie in two planes: 16 bytes from lane to lane, no bank conflicts
      for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
        const int at = VEC == 8 ? (c >> 2 & 1) * (p.D >> 1) + (c >> 3) * 4 + (c & 3) : c;
        s[at] = p.w ? param_at(p.w, p.w_type, c) : 1.0f;
        if (N == 2) s[p.D + at] = p.b ? param_at(p.b, p.w_type, c) : 0.0f;
      }
      __syncthreads();
    }
  }
  __device__ __forceinline__ void get(int n, int k, int c, int D, float (&out)[VEC]) const {
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) out[j] = f[n][k][j];
    } else {
      if constexpr (VEC == 8) {
        RawVec<float, 8> r;
        r.a = *reinterpret_cast<const float4*>(s + n * D + c * 4);
        r.b = *reinterpret_cast<const float4*>(s + n * D + (D >> 1) + c * 4);
        r.unpack(out);
      } else {
        out[0] = s[n * D + c];
      }
    }
  }
};

// UPT vectors of VEC columns a thread: columns (lane + k * tpr) * VEC.  The
// blocks are persistent, and a row's loads are issued before the row before it
// is worked on.  EXACT: the threads' columns are the row's.
template <typename TX, typename TY, int VEC, int UPT, bool EXACT>
__global__ void __launch_bounds__(kMaxRowThreads, UPT * VEC <= 16 ? 2 : 1) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float s_red[2][1][32];
  extern __shared__ __align__(16) float s_dyn[];
  const int rows = blockDim.x / p.tpr;  // rows a block takes at once
  const int row = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  Params<VEC, UPT, 2> par;
  par.init(p, s_dyn, lane);
  const float inv = 1.0f / (float)p.D;
  const int64_t step = (int64_t)gridDim.x * rows;
  auto mine = [&](int k) { return EXACT || lane + k * p.tpr < p.units; };
  RawVec<TX, VEC> raw[UPT];
  auto fetch = [&](int64_t i) {
    const TX* x = static_cast<const TX*>(p.x) + (i < p.M ? i : p.M - 1) * p.x_stride + lane * VEC;
#pragma unroll
    for (int k = 0; k < UPT; ++k)
      if (mine(k)) raw[k].load(x + k * p.tpr * VEC);
  };
  int64_t i = (int64_t)blockIdx.x * rows + row;
  fetch(i);
  // every thread of the block goes through the same number of steps (a warp may
  // hold several rows, and all its lanes take part in the sums); a row past the
  // last is the last one again, and is not stored
  for (int64_t i0 = (int64_t)blockIdx.x * rows; i0 < p.M; i0 += step, i += step) {
    float v[UPT][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      if (!mine(k)) break;
      raw[k].unpack(v[k]);
      s[0] += vec_sum(v[k]);
    }
    fetch(i + step);
    row_sum<1>(s, p.tpr, s_red[0]);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      if (!mine(k)) break;
      s[0] += vec_center(v[k], mu);
    }
    row_sum<1>(s, p.tpr, s_red[1]);
    const float r = inv_sqrt(fmaf(s[0], inv, p.eps));
    if (i >= p.M) continue;
    if (lane == 0) {
      if (p.mean) p.mean[i] = mu;
      if (p.rstd) p.rstd[i] = r;
    }
    TY* y = static_cast<TY*>(p.y) + i * p.y_stride + lane * VEC;
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      if (!mine(k)) break;
      float w[VEC], b[VEC];
      par.get(0, k, lane + k * p.tpr, p.D, w);
      par.get(1, k, lane + k * p.tpr, p.D, b);
      vec_affine(v[k], r, w, b);
      store_vec(y + k * p.tpr * VEC, v[k]);
    }
  }
}

// Rows of several vectors a lane, a warp a row: the row stays in registers as it
// lies in memory (UPT x 8 values a lane) and is unpacked anew for the mean, the
// squares and the output, so a row needs no barrier, and ten shuffles in all.
template <typename TX, typename TY, int UPT>
__global__ void __launch_bounds__(256, 2) norm_row_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) float s_dyn[];
  const int lane = threadIdx.x & 31;
  Params<8, UPT, 2> par;
  par.init(p, s_dyn, lane);
  const float inv = 1.0f / (float)p.D;
  auto mine = [&](int k) { return lane + k * 32 < p.units; };
  auto warp_sum = [](float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < p.M; i += (int64_t)gridDim.x * 8) {
    const TX* x = static_cast<const TX*>(p.x) + i * p.x_stride + lane * 8;
    TY* y = static_cast<TY*>(p.y) + i * p.y_stride + lane * 8;
    RawVec<TX, 8> raw[UPT];
#pragma unroll
    for (int k = 0; k < UPT; ++k)
      if (mine(k)) raw[k].load(x + k * 256);
    float s = 0.f, v[8];
#pragma unroll
    for (int k = 0; k < UPT; ++k)
      if (mine(k)) {
        raw[k].unpack(v);
        s += vec_sum(v);
      }
    const float mu = warp_sum(s) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < UPT; ++k)
      if (mine(k)) {
        raw[k].unpack(v);
        s += vec_center(v, mu);
      }
    const float r = inv_sqrt(fmaf(warp_sum(s), inv, p.eps));
    if (lane == 0) {
      if (p.mean) p.mean[i] = mu;
      if (p.rstd) p.rstd[i] = r;
    }
#pragma unroll
    for (int k = 0; k < UPT; ++k)
      if (mine(k)) {
        float w[8], b[8];
        par.get(0, k, lane + k * 32, p.D, w);
        par.get(1, k, lane + k * 32, p.D, b);
        raw[k].unpack(v);
        vec_center(v, mu);
        vec_affine(v, r, w, b);
        store_vec(y + k * 256, v);
      }
  }
}

// Rows wider than the registers of a block hold: three reads of the row.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float s_red[2][1][32];
  const TX* x = static_cast<const TX*>(p.x) + (int64_t)blockIdx.x * p.x_stride;
  TY* y = static_cast<TY*>(p.y) + (int64_t)blockIdx.x * p.y_stride;
  float s[1] = {0.f};
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) s[0] += to_f32(x[c]);
  row_sum<1>(s, kWideThreads, s_red[0]);
  const float mu = s[0] / (float)p.D;
  s[0] = 0.f;
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float d = to_f32(x[c]) - mu;
    s[0] = fmaf(d, d, s[0]);
  }
  row_sum<1>(s, kWideThreads, s_red[1]);
  const float r = 1.0f / sqrtf(s[0] / (float)p.D + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mu;
    if (p.rstd) p.rstd[blockIdx.x] = r;
  }
  for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
    const float w = p.w ? param_at(p.w, p.w_type, c) : 1.0f, b = p.b ? param_at(p.b, p.w_type, c) : 0.0f;
    y[c] = from_f32<TY>(fmaf((to_f32(x[c]) - mu) * r, w, b));
  }
}

template <typename TX, typename TY, int VEC, int UPT, bool EXACT>
__global__ void __launch_bounds__(kMaxRowThreads) norm_back_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float s_red[2][2][32];
  // the weight (Params), and later [2][tpr * UPT * VEC] sums of the block's rows
  extern __shared__ __align__(16) float s_part[];
  const int rows = blockDim.x / p.tpr, row = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  Params<VEC, UPT, 1> par;
  par.init(p, s_part, lane);
  float dw[UPT][VEC], db[UPT][VEC];
#pragma unroll
  for (int k = 0; k < UPT; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[k][j] = db[k][j] = 0.f;
  auto mine = [&](int k) { return EXACT || lane + k * p.tpr < p.units; };
  const float inv = 1.0f / (float)p.D;
  const int64_t step = (int64_t)gridDim.x * rows;
  int flip = 0;
  RawVec<TX, VEC> rx[UPT];
  RawVec<TY, VEC> rg[UPT];
  float mu_next = 0.f, r_next = 0.f;
  auto fetch = [&](int64_t i) {
    if (i >= p.M) return;
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      const int c = lane + k * p.tpr;
      if (mine(k)) {
        rx[k].load(static_cast<const TX*>(p.x) + i * p.x_stride + (int64_t)c * VEC);
        rg[k].load(static_cast<const TY*>(p.gy) + i * p.gy_stride + (int64_t)c * VEC);
      }
    }
    mu_next = __ldg(p.mean + i);
    r_next = __ldg(p.rstd + i);
  };
  fetch((int64_t)blockIdx.x * rows + row);
  // every thread of the block goes through the same number of steps
  for (int64_t i0 = (int64_t)blockIdx.x * rows; i0 < p.M; i0 += step, flip ^= 1) {
    const int64_t i = i0 + row;
    const bool live = i < p.M;
    const float mu = live ? mu_next : 0.f, r = live ? r_next : 0.f;
    float xh[UPT][VEC], g[UPT][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      const int c = lane + k * p.tpr;
#pragma unroll
      for (int j = 0; j < VEC; ++j) xh[k][j] = g[k][j] = 0.f;
      if (live && mine(k)) {
        rx[k].unpack(xh[k]);
        rg[k].unpack(g[k]);
        float w[VEC];
        par.get(0, k, c, p.D, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[k][j] = (xh[k][j] - mu) * r;
          db[k][j] += g[k][j];
          dw[k][j] = fmaf(g[k][j], xh[k][j], dw[k][j]);
          g[k][j] *= w[j];
          s[0] += g[k][j];
          s[1] = fmaf(g[k][j], xh[k][j], s[1]);
        }
      }
    }
    fetch(i + step);
    if (!p.y) continue;
    row_sum<2>(s, p.tpr, s_red[flip]);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    if (live) {
      TX* dx = static_cast<TX*>(p.y) + i * p.y_stride;
#pragma unroll
      for (int k = 0; k < UPT; ++k) {
        const int c = lane + k * p.tpr;
        if (!mine(k)) break;
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = r * (g[k][j] - m0 - xh[k][j] * m1);
        store_vec(dx + (int64_t)c * VEC, f);
      }
    }
  }
  if (!p.partial) return;
  __syncthreads();  // the weight is done with
  // the block's rows, added in row order
  const int cols = p.tpr * UPT * VEC;
  for (int q = 0; q < rows; ++q) {
    if (row == q) {
#pragma unroll
      for (int k = 0; k < UPT; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int at = (lane + k * p.tpr) * VEC + j;
          s_part[at] = q ? s_part[at] + dw[k][j] : dw[k][j];
          s_part[cols + at] = q ? s_part[cols + at] + db[k][j] : db[k][j];
        }
    }
    __syncthreads();
  }
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.D;
  for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
    out[c] = s_part[c];
    out[p.D + c] = s_part[cols + c];
  }
}

// Wide rows: a row's sums and its dx from three reads; the block's dw and db
// live in its partial row in global memory (no other block touches it).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kWideThreads) norm_back_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(16) float s_red[2][2][32];
  float* out = p.partial ? p.partial + (int64_t)blockIdx.x * 2 * p.D : nullptr;
  if (out)
    for (int c = threadIdx.x; c < 2 * p.D; c += kWideThreads) out[c] = 0.f;
  __syncthreads();
  int flip = 0;
  for (int64_t i = blockIdx.x; i < p.M; i += gridDim.x, flip ^= 1) {
    const TX* x = static_cast<const TX*>(p.x) + i * p.x_stride;
    const TY* gy = static_cast<const TY*>(p.gy) + i * p.gy_stride;
    const float mu = __ldg(p.mean + i), r = __ldg(p.rstd + i);
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
      const float d = to_f32(gy[c]), xh = (to_f32(x[c]) - mu) * r;
      const float g = d * (p.w ? param_at(p.w, p.w_type, c) : 1.0f);
      s[0] += g;
      s[1] = fmaf(g, xh, s[1]);
      if (out) {  // column c is this thread's in every row
        out[c] = fmaf(d, xh, out[c]);
        out[p.D + c] += d;
      }
    }
    if (!p.y) continue;
    row_sum<2>(s, kWideThreads, s_red[flip]);
    const float m0 = s[0] / (float)p.D, m1 = s[1] / (float)p.D;
    TX* dx = static_cast<TX*>(p.y) + i * p.y_stride;
    for (int c = threadIdx.x; c < p.D; c += kWideThreads) {
      const float xh = (to_f32(x[c]) - mu) * r;
      const float g = to_f32(gy[c]) * (p.w ? param_at(p.w, p.w_type, c) : 1.0f);
      dx[c] = from_f32<TX>(r * (g - m0 - xh * m1));
    }
  }
}

// dw and db from the blocks' sums: 32 columns a block, warp k the k-th part of
// the blocks in order, fp64.
__global__ void __launch_bounds__(1024) norm_join_kernel(float* partial, int blocks, int D, int w_type, void* dw,
                                                         void* db) {
  __shared__ double s[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // columns of [dw | db]
  double t = 0.0;
  const int per = (blocks + 31) / 32;
  pdl_wait();
  if (c < 2 * D) {
    const int q1 = min((k + 1) * per, blocks);
#pragma unroll 8
    for (int q = k * per; q < q1; ++q) t += (double)partial[(int64_t)q * 2 * D + c];
  }
  s[k][lane] = t;
  __syncthreads();
  if (k != 0 || c >= 2 * D) return;
  t = 0.0;
  for (int q = 0; q < 32; ++q) t += s[q][lane];
  void* out = c < D ? dw : db;
  const int at = c < D ? c : c - D;
  if (!out) return;
  if (w_type == RECIS_F32) static_cast<float*>(out)[at] = (float)t;
  else if (w_type == RECIS_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn((float)t);
  else static_cast<__half*>(out)[at] = __float2half_rn((float)t);
}

// threads a row: a power of two, with at most `upt` vectors a thread (0: the
// row does not fit a block)
int row_threads(int units, int upt) {
  int t = 1;
  while (t * upt < units && t <= kMaxRowThreads) t *= 2;
  return t <= kMaxRowThreads ? t : 0;
}

// Blocks of `kernel` that all SMs hold at once; asked for once, `cache` is the
// kernel's own (its block size and shared memory may differ: one entry a log2
// of the block's threads).
template <typename K>
int resident_blocks(K kernel, int block, size_t smem, std::atomic<int> (&cache)[16]) {
  int at = 0;
  while ((1 << at) < block) ++at;
  int n = cache[at].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, block, smem) != cudaSuccess || n < 1) n = 1;
    cache[at].store(n, std::memory_order_relaxed);
  }
  return n * kSMs;
}

// Dynamic shared memory beyond the default (48 KB with the kernels' own half KB).
// The limit is the function's, not the launch's, so it is raised once to the most
// that any row takes: a smaller one set for a narrower row would refuse a wide
// row's launch in another host thread.
template <int MOST, typename K>
cudaError_t more_smem(K kernel, std::atomic<uint64_t> (&done)[2]) {
  if constexpr (MOST > 47 * 1024) return allow_smem(kernel, MOST, done);
  else return cudaSuccess;
}

template <typename TX, typename TY, int VEC, int UPT, bool EXACT>
cudaError_t norm_go(const NormParams& p, cudaStream_t s) {
  static std::atomic<int> cache[16];
  auto kernel = norm_kernel<TX, TY, VEC, UPT, EXACT>;
  const int block = std::max(p.tpr, 128), rows = block / p.tpr;
  constexpr bool keep = Params<VEC, UPT, 2>::kKeep;
  const size_t smem = keep ? 0 : (size_t)p.D * 8;  // D is at most kMaxRowThreads * UPT * VEC
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = more_smem<keep ? 0 : kMaxRowThreads * UPT * VEC * 8>(kernel, done);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<int64_t>((p.M + rows - 1) / rows, resident_blocks(kernel, block, smem, cache));
  kernel<<<grid, block, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename TX, typename TY, int UPT>
cudaError_t norm_row_go(const NormParams& p, cudaStream_t s) {
  static std::atomic<int> cache[16];
  auto kernel = norm_row_kernel<TX, TY, UPT>;
  const size_t smem = (size_t)p.D * 8;  // at most 32 KB
  const int grid = (int)std::min<int64_t>((p.M + 7) / 8, resident_blocks(kernel, 256, smem, cache));
  kernel<<<grid, 256, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename TX, typename TY, int VEC>
cudaError_t norm_launch(NormParams p, cudaStream_t s) {
  p.units = p.D / VEC;
  LaunchScope ls("layer_norm", s);
  // A warp a row while it holds in 64 registers a lane, and, where that takes more
  // than 8 vectors a lane, there are rows for every SM (bf16, with a block's threads a
  // row instead: 16384 x 4096 60 and 75 us, 16384 x 2048 34 and 44, 64 x 1024 8.7 and
  // 10.5; 64 x 4096 18.5 and 14.6, 888 x 4096 18.5 and 19).
  if constexpr (VEC == 8) {
    constexpr int most = sizeof(TX) == 2 ? 16 : 8;
    if (p.units > 64 && p.units <= 32 * most && (p.units <= 256 || p.M >= kSMs * 6)) {
      if (p.units <= 128) return norm_row_go<TX, TY, 4>(p, s);
      if (p.units <= 256) return norm_row_go<TX, TY, 8>(p, s);
      return norm_row_go<TX, TY, most>(p, s);
    }
  }
  // Else up to two vectors a thread (single columns: 8), then more threads.  More
  // columns a thread share the sums' shuffles and barriers, fewer leave registers
  // for more rows an SM and more threads for few rows: 16384 x 4096 fp32 takes 135 us
  // at 8 columns, 106 at 16, 112 at 32; 64 x 8192 bf16 16 at 16 and 23 at 32 (16384
  // rows 143 and 126).
  int upt = p.units <= 32 ? 1 : 2;
  if (VEC == 1 && p.units > 64) upt = 8;
  p.tpr = row_threads(p.units, upt);
  if (VEC == 8 && !p.tpr) p.tpr = row_threads(p.units, upt = 4);
  if (!p.tpr) {
    norm_wide_kernel<TX, TY><<<(unsigned)p.M, kWideThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const bool exact = p.tpr * upt == p.units;
  if (upt == 1) return norm_go<TX, TY, VEC, 1, false>(p, s);
  if (upt == 2) return exact ? norm_go<TX, TY, VEC, 2, true>(p, s) : norm_go<TX, TY, VEC, 2, false>(p, s);
  return norm_go<TX, TY, VEC, VEC == 8 ? 4 : 8, false>(p, s);
}

// blocks of the backward (its partial sums' rows): the same for every type
int back_blocks(int64_t M) { return (int)std::min<int64_t>(M, kSMs * 6); }

template <typename TX, typename TY, int VEC, int UPT, bool EXACT>
cudaError_t back_go(const NormParams& p, cudaStream_t s, int* blocks_out) {
  static std::atomic<int> cache[16];
  auto kernel = norm_back_kernel<TX, TY, VEC, UPT, EXACT>;
  const int block = std::max(p.tpr, 256), rows = block / p.tpr;
  const size_t smem = (size_t)2 * p.tpr * UPT * VEC * 4;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = more_smem<2 * kMaxRowThreads * UPT * VEC * 4>(kernel, done);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min<int64_t>(back_blocks(p.M), (p.M + rows - 1) / rows);
  const int grid = (int)std::min<int64_t>(most, resident_blocks(kernel, block, smem, cache));
  *blocks_out = grid;
  kernel<<<grid, block, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename TX, typename TY, int VEC>
cudaError_t back_launch(NormParams p, cudaStream_t s, int* blocks_out) {
  p.units = p.D / VEC;
  LaunchScope ls("layer_norm_backward", s);
  // as the forward, but at most two vectors a thread: it keeps two sums a column
  const int upt = p.units <= 32 ? 1 : VEC == 1 && p.units > 64 ? 8 : 2;
  p.tpr = row_threads(p.units, upt);
  if (!p.tpr) {
    *blocks_out = back_blocks(p.M);
    norm_back_wide_kernel<TX, TY><<<*blocks_out, kWideThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const bool exact = p.tpr * upt == p.units;
  if (upt == 1) return back_go<TX, TY, VEC, 1, false>(p, s, blocks_out);
  if (VEC == 1) return upt == 2 ? back_go<TX, TY, VEC, 2, false>(p, s, blocks_out)
                                : back_go<TX, TY, VEC, VEC == 1 ? 8 : 2, false>(p, s, blocks_out);
  return exact ? back_go<TX, TY, VEC, 2, true>(p, s, blocks_out) : back_go<TX, TY, VEC, 2, false>(p, s, blocks_out);
}

bool norm_sizes_ok(int64_t M, int32_t D) { return M >= 0 && M <= INT32_MAX && D >= 1 && D <= 65536; }

}  // namespace
}  // namespace recis

using namespace recis;

extern "C" recis_status recis_layer_norm(const void* x, int32_t x_type, int64_t x_stride, int64_t M, int32_t D,
                                         const void* weight, const void* bias, int32_t w_type, double eps, void* y,
                                         int32_t y_type, int64_t y_stride, float* mean, float* rstd,
                                         recis_stream_t stream) {
  if (!float_type(x_type) || !float_type(y_type) || !float_type(w_type) || !norm_sizes_ok(M, D) || x_stride < D ||
      y_stride < D || !(eps >= 0.0) || (M > 0 && (!x || !y))) {
    set_error("layer_norm: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  if (misaligned(x, type_bytes(x_type)) || misaligned(y, type_bytes(y_type)) ||
      misaligned(weight, type_bytes(w_type)) || misaligned(bias, type_bytes(w_type)) || misaligned(mean, 4) ||
      misaligned(rstd, 4)) {
    set_error("layer_norm: misaligned array");
    return RECIS_ERR_INVALID_ARG;
  }
  if (M == 0) return RECIS_OK;
  NormParams p = {};
  p.x = x;
  p.w = weight;
  p.b = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.M = M;
  p.x_stride = x_stride;
  p.y_stride = y_stride;
  p.D = D;
  p.w_type = w_type;
  p.eps = (float)eps;
  const bool vec = D % 8 == 0 && rows_aligned16(x, x_stride, x_type) && rows_aligned16(y, y_stride, y_type);
  const cudaError_t e = with_type(x_type, [&](auto a) {
    return with_type(y_type, [&](auto b) {
      using TX = decltype(a);
      using TY = decltype(b);
      return vec ? norm_launch<TX, TY, 8>(p, (cudaStream_t)stream) : norm_launch<TX, TY, 1>(p, (cudaStream_t)stream);
    });
  });
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "layer_norm launch");
}

extern "C" recis_status recis_layer_norm_backward_workspace(int64_t M, int32_t D, int64_t* bytes_out) {
  if (!bytes_out || !norm_sizes_ok(M, D)) {
    set_error("layer_norm_backward_workspace: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  *bytes_out = (int64_t)back_blocks(M) * 2 * D * 4;
  return RECIS_OK;
}

extern "C" recis_status recis_layer_norm_backward(const void* grad_y, int32_t y_type, int64_t grad_y_stride,
                                                  const void* x, int32_t x_type, int64_t x_stride, int64_t M,
                                                  int32_t D, const void* weight, int32_t w_type, const float* mean,
                                                  const float* rstd, void* grad_x, int64_t grad_x_stride,
                                                  void* grad_weight, void* grad_bias, void* workspace,
                                                  int64_t workspace_bytes, recis_stream_t stream) {
  if (!float_type(x_type) || !float_type(y_type) || !float_type(w_type) || !norm_sizes_ok(M, D) || x_stride < D ||
      grad_y_stride < D || (grad_x && grad_x_stride < D) || (M > 0 && (!x || !grad_y || !mean || !rstd))) {
    set_error("layer_norm_backward: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  if (misaligned(x, type_bytes(x_type)) || misaligned(grad_y, type_bytes(y_type)) ||
      misaligned(weight, type_bytes(w_type)) || misaligned(grad_x, type_bytes(x_type)) ||
      misaligned(grad_weight, type_bytes(w_type)) || misaligned(grad_bias, type_bytes(w_type)) || misaligned(mean, 4) ||
      misaligned(rstd, 4) || misaligned(workspace, 256)) {
    set_error("layer_norm_backward: misaligned array");
    return RECIS_ERR_INVALID_ARG;
  }
  const bool sums = grad_weight || grad_bias;
  cudaStream_t s = (cudaStream_t)stream;
  if (M == 0) {
    cudaError_t e = cudaSuccess;
    if (grad_weight) e = cudaMemsetAsync(grad_weight, 0, (size_t)D * type_bytes(w_type), s);
    if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, (size_t)D * type_bytes(w_type), s);
    return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "layer_norm_backward memset");
  }
  if (!sums && !grad_x) return RECIS_OK;
  if (sums && (!workspace || workspace_bytes < (int64_t)back_blocks(M) * 2 * D * 4)) {
    set_error("layer_norm_backward: workspace too small");
    return RECIS_ERR_INVALID_ARG;
  }
  NormParams p = {};
  p.x = x;
  p.w = weight;
  p.gy = grad_y;
  p.y = grad_x;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  p.M = M;
  p.x_stride = x_stride;
  p.gy_stride = grad_y_stride;
  p.y_stride = grad_x_stride;
  p.D = D;
  p.w_type = w_type;
  const bool vec = D % 8 == 0 && rows_aligned16(x, x_stride, x_type) && rows_aligned16(grad_y, grad_y_stride, y_type) &&
                   (!grad_x || rows_aligned16(grad_x, grad_x_stride, x_type));
  int blocks = 0;
  cudaError_t e = with_type(x_type, [&](auto a) {
    return with_type(y_type, [&](auto b) {
      using TX = decltype(a);
      using TY = decltype(b);
      return vec ? back_launch<TX, TY, 8>(p, s, &blocks) : back_launch<TX, TY, 1>(p, s, &blocks);
    });
  });
  if (e != cudaSuccess) return cuda_fail(e, "layer_norm_backward launch");
  if (sums) {
    LaunchScope ls("layer_norm_join", s);
    e = launch_pdl(norm_join_kernel, (unsigned)((2 * D + 31) / 32), 1024, 0, s, p.partial, blocks, D, w_type,
                   grad_weight, grad_bias);
    if (e != cudaSuccess) return cuda_fail(e, "layer_norm_join launch");
  }
  return RECIS_OK;
}
