// Layer norm over the last dimension and its gradients.
//   mean = sum x / W,  rstd = (sum (x - mean)^2 / W + eps)^(-1/2),  xhat = (x - mean) rstd,  y = xhat gamma + beta
//   g = dY gamma,  dX = rstd (g - sum g / W - xhat (sum g xhat) / W),  dgamma = sum_rows dY xhat,  dbeta = sum_rows dY
// Bound by memory: the forward reads X and writes Y once, the backward reads X and dY and writes dX once, with
// each row held in registers between (so the variance is taken over x - mean, not as a difference of
// squares).  A row belongs to a group of threads: 8, 16 or 32 lanes of a warp when it is short, a CTA when
// it is long; thread t of a group holds the same columns of every row it meets, so gamma's and beta's
// gradients are summed in registers over the rows, then over the CTA's groups in shared memory, and one
// partial row per CTA goes to the workspace; a second kernel adds the partial rows in a fixed order.  No
// atomics: the same bits on every run.
#include <cuda_bf16.h>

#include "svg2_device.cuh"
#include "svg2_internal.h"

namespace svg2 {

namespace {

template <class T>
struct NormArgs {
  const T *X, *dY;
  const float *gamma, *beta;      // optional
  const float *mean_in, *rstd_in; // backward
  float *mean, *rstd;             // forward, optional
  T* Y;                           // Y | dX
  float* partial;                 // backward: [gridDim.x][2][W]
  long long rows;
  int W;
  float eps;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f32(*p);
  } else if constexpr (sizeof(T) == 4) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[2 * e] = bf16lo_to_f32(u[e]), v[2 * e + 1] = bf16hi_to_f32(u[e]);
  }
}

template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 4) *p = v[0];
    else *p = __float2bfloat16(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// float32 parameters of a thread's VEC columns
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = __ldg(p);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(p + e));
      v[e] = w.x, v[e + 1] = w.y, v[e + 2] = w.z, v[e + 3] = w.w;
    }
  }
}

// Sum of one value (or two) over a group of G threads: G lanes of a warp, or (G = 0) the whole CTA.
// `turn` alternates the shared buffer between consecutive sums, so one barrier per sum is enough.
template <int G, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* buf, int& turn) {
  constexpr int kWidth = G == 0 ? 32 : G;
#pragma unroll
  for (int o = kWidth / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (G == 0) {
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* b = buf + turn * 64;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) b[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < warps ? b[k * 32 + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[k] = s;
    }
  }
}

// The columns of thread t of a group of n threads: vectors t, t + n, ... of the row.
template <class T, int VEC, int G, int NV, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const NormArgs<T> a) {
  __shared__ float buf[128];
  const int n = G == 0 ? blockDim.x : G;
  const int t = threadIdx.x % n;
  const int nvec = a.W / VEC;
  const long long groups = static_cast<long long>(gridDim.x) * (blockDim.x / n);
  const long long group = static_cast<long long>(blockIdx.x) * (blockDim.x / n) + threadIdx.x / n;
  const float inv_w = 1.f / static_cast<float>(a.W);
  int turn = 0;
  // the trip count is the same for all groups of a CTA: the sums are collective
  for (long long base = 0; base < a.rows; base += groups * R) {
    float x[R][NV][VEC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + group;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        if (row < a.rows && c < nvec) {
          load_vec<T, VEC>(a.X + row * a.W + static_cast<long long>(c) * VEC, x[r][i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[r][i][e] = 0.f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + group;
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0] += x[r][i][e];
      group_sum<G, 1>(s, buf, turn);
      const float mean = s[0] * inv_w;
      s[0] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = t + i * n < nvec;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[r][i][e] = in ? x[r][i][e] - mean : 0.f;
          s[0] = fmaf(x[r][i][e], x[r][i][e], s[0]);
        }
      }
      group_sum<G, 1>(s, buf, turn);
      const float rstd = 1.f / sqrtf(fmaf(s[0], inv_w, a.eps));
      if (row >= a.rows) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        if (c >= nvec) continue;
        float y[VEC], p[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = x[r][i][e] * rstd;
        if (a.gamma != nullptr) {
          load_param<VEC>(a.gamma + c * VEC, p);
#pragma unroll
          for (int e = 0; e < VEC; ++e) y[e] *= p[e];
        }
        if (a.beta != nullptr) {
          load_param<VEC>(a.beta + c * VEC, p);
#pragma unroll
          for (int e = 0; e < VEC; ++e) y[e] += p[e];
        }
        store_vec<T, VEC>(a.Y + row * a.W + static_cast<long long>(c) * VEC, y);
      }
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
    }
  }
}

template <class T, int VEC, int G, int NV, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormArgs<T> a) {
  __shared__ float buf[128];
  __shared__ float acc_s[G == 0 ? 1 : 2 * 8 * 32 * NV * VEC];  // the warps' column sums
  const int n = G == 0 ? blockDim.x : G;
  const int t = threadIdx.x % n;
  const int nvec = a.W / VEC;
  const long long groups = static_cast<long long>(gridDim.x) * (blockDim.x / n);
  const long long group = static_cast<long long>(blockIdx.x) * (blockDim.x / n) + threadIdx.x / n;
  const float inv_w = 1.f / static_cast<float>(a.W);
  int turn = 0;
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dg[i][e] = db[i][e] = 0.f;
  for (long long base = 0; base < a.rows; base += groups * R) {
    float x[R][NV][VEC], g[R][NV][VEC], rstd[R], mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + group;
      const bool live = row < a.rows;
      mean[r] = live ? __ldg(a.mean_in + row) : 0.f;
      rstd[r] = live ? __ldg(a.rstd_in + row) : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        if (live && c < nvec) {
          load_vec<T, VEC>(a.X + row * a.W + static_cast<long long>(c) * VEC, x[r][i]);
          load_vec<T, VEC>(a.dY + row * a.W + static_cast<long long>(c) * VEC, g[r][i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[r][i][e] = mean[r], g[r][i][e] = 0.f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * groups + group;
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        float p[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = 1.f;
        if (a.gamma != nullptr && c < nvec) load_param<VEC>(a.gamma + c * VEC, p);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x[r][i][e] = (x[r][i][e] - mean[r]) * rstd[r];
          dg[i][e] = fmaf(g[r][i][e], x[r][i][e], dg[i][e]);
          db[i][e] += g[r][i][e];
          g[r][i][e] *= p[e];
          s[0] += g[r][i][e];
          s[1] = fmaf(g[r][i][e], x[r][i][e], s[1]);
        }
      }
      group_sum<G, 2>(s, buf, turn);
      if (row >= a.rows) continue;
      const float c1 = s[0] * inv_w, c2 = s[1] * inv_w;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        if (c >= nvec) continue;
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = rstd[r] * (g[r][i][e] - c1 - x[r][i][e] * c2);
        store_vec<T, VEC>(a.Y + row * a.W + static_cast<long long>(c) * VEC, d);
      }
    }
  }
  float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.W;
  if constexpr (G == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * n;
      if (c >= nvec) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        out[c * VEC + e] = dg[i][e];
        out[a.W + c * VEC + e] = db[i][e];
      }
    }
  } else {
    // over the groups of a warp by shuffles, over the 8 warps in shared memory
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
          dg[i][e] += __shfl_xor_sync(0xffffffffu, dg[i][e], o);
          db[i][e] += __shfl_xor_sync(0xffffffffu, db[i][e], o);
        }
        if (lane < G) {
          acc_s[((warp * 2 + 0) * NV + i) * VEC * G + lane * VEC + e] = dg[i][e];
          acc_s[((warp * 2 + 1) * NV + i) * VEC * G + lane * VEC + e] = db[i][e];
        }
      }
    __syncthreads();
    constexpr int kCols = NV * VEC * G;  // column c of the row is entry c: vector c / VEC = lane + i G
    for (int c = threadIdx.x; c < 2 * kCols; c += blockDim.x) {
      const int which = c / kCols, col = c % kCols;
      if (col >= a.W) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += acc_s[(w * 2 + which) * kCols + col];
      out[which * a.W + col] = s;
    }
  }
}

// dgamma, dbeta = the column sums of the partial rows, 32 columns per CTA: warp w adds rows w, w + 32, ...,
// then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partial, int parts, int W,
                                                           float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;  // of 2 W columns
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < 2 * W) {
    int r = warp;
    for (; r + 96 < parts; r += 128)
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] += __ldg(partial + static_cast<size_t>(r + 32 * u) * 2 * W + col);
    for (; r < parts; r += 32) v[0] += __ldg(partial + static_cast<size_t>(r) * 2 * W + col);
  }
  s[warp][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (warp == 0 && col < 2 * W) {
    float t = 0.f;
    for (int w = 0; w < 32; ++w) t += s[w][lane];
    float* out = col < W ? dgamma : dbeta;
    if (out != nullptr) out[col < W ? col : col - W] = t;
  }
}

template <class T, int VEC, int G, int NV, int R, int MAXT = 256>
cudaError_t run_norm(const NormArgs<T>& a, bool bwd, int threads, int max_parts, int* parts, cudaStream_t s) {
  const int per_cta = G == 0 ? 1 : threads / G;
  // as many CTAs as are resident at once (every group then meets the same number of rows, within one pass)
  int resident = 0;
  cudaError_t e = bwd ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, norm_bwd_kernel<T, VEC, G, NV, R, MAXT>, threads, 0)
                      : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, norm_fwd_kernel<T, VEC, G, NV, R, MAXT>, threads, 0);
  if (e != cudaSuccess) return e;
  const long long want = (a.rows + static_cast<long long>(per_cta) * R - 1) / (static_cast<long long>(per_cta) * R);
  long long grid = static_cast<long long>(kNormSms) * (resident > 0 ? resident : 1);
  if (grid > want) grid = want;
  if (bwd && grid > max_parts) grid = max_parts;
  *parts = static_cast<int>(grid);
  if (bwd) norm_bwd_kernel<T, VEC, G, NV, R, MAXT><<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
  else norm_fwd_kernel<T, VEC, G, NV, R, MAXT><<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <class T, int VEC>
cudaError_t pick_norm(const NormArgs<T>& a, bool bwd, int max_parts, int* parts, cudaStream_t s) {
  const int nvec = a.W / VEC;
  // a row of up to 128 vectors belongs to lanes of one warp, a longer one to a CTA
  if constexpr (VEC > 1) {
    if (nvec <= 8) return run_norm<T, VEC, 8, 1, 2>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 16) return run_norm<T, VEC, 16, 1, 2>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 32) return run_norm<T, VEC, 32, 1, 2>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 64) return run_norm<T, VEC, 32, 2, 1>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 256) return run_norm<T, VEC, 0, 1, 1>(a, bwd, (nvec + 31) / 32 * 32, max_parts, parts, s);
    // (at most 8192 columns: 1024 vectors of bf16, 2048 of float32)
    return run_norm<T, VEC, 0, 2, 1, VEC == 8 ? 512 : 1024>(a, bwd, ((nvec + 1) / 2 + 31) / 32 * 32, max_parts, parts, s);
  } else {
    if (nvec <= 32) return run_norm<T, 1, 32, 1, 2>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 128) return run_norm<T, 1, 32, 4, 1>(a, bwd, 256, max_parts, parts, s);
    if (nvec <= 1024) return run_norm<T, 1, 0, 4, 1>(a, bwd, ((nvec + 3) / 4 + 31) / 32 * 32, max_parts, parts, s);
    return run_norm<T, 1, 0, 8, 1, 1024>(a, bwd, ((nvec + 7) / 8 + 31) / 32 * 32, max_parts, parts, s);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class T>
cudaError_t run_typed(const NormCall& n, bool bwd, cudaStream_t s) {
  NormArgs<T> a{};
  a.X = static_cast<const T*>(n.X);
  a.dY = static_cast<const T*>(n.dY);
  a.gamma = n.gamma;
  a.beta = n.beta;
  a.mean_in = a.mean = n.mean;
  a.rstd_in = a.rstd = n.rstd;
  a.Y = static_cast<T*>(n.Y);
  a.partial = n.partial;
  a.rows = n.rows;
  a.W = n.width;
  a.eps = n.eps;
  constexpr int kVec = 16 / sizeof(T);
  // 16-byte accesses where every row starts on a 16-byte boundary, else element by element
  const bool vec = n.width % kVec == 0 && aligned16(n.X) && aligned16(n.dY) && aligned16(n.Y) && aligned16(n.gamma) &&
                   aligned16(n.beta);
  int parts = 0;
  const int max_parts = norm_max_parts(n.rows);
  cudaError_t e = vec ? pick_norm<T, kVec>(a, bwd, max_parts, &parts, s) : pick_norm<T, 1>(a, bwd, max_parts, &parts, s);
  if (e == cudaSuccess && bwd && (n.dgamma != nullptr || n.dbeta != nullptr)) {
    norm_reduce_kernel<<<(2 * n.width + 31) / 32, 1024, 0, s>>>(n.partial, parts, n.width, n.dgamma, n.dbeta);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

cudaError_t launch_norm(const NormCall& n, bool f32, bool bwd, cudaStream_t s) {
  return f32 ? run_typed<float>(n, bwd, s) : run_typed<__nv_bfloat16>(n, bwd, s);
}

}  // namespace svg2
