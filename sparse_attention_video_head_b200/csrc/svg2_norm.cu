// Layer norm over the last dimension and its gradients.
//   mean = sum x / W,  rstd = (sum (x - mean)^2 / W + eps)^(-1/2),  xhat = (x - mean) rstd,  y = xhat gamma + beta
//   g = dY gamma,  dX = rstd (g - sum g / W - xhat (sum g xhat) / W),  dgamma = sum_rows dY xhat,  dbeta = sum_rows dY
// Bound by memory: the forward reads X and writes Y once, the backward reads X and dY and writes dX once, with
// each row held in registers between (so the variance is taken over x - mean, not as a difference of squares).
//
// A row belongs to a group of threads: 8, 16 or 32 lanes of a warp when it is short, a CTA when it is long.
// Every thread copies its own 16-byte vectors of the next rows into its own slots of a shared-memory ring
// (cp.async) while it works on the current one, so reads stay in flight through the row sums without
// registers or barriers.  A row that does not start on a 16-byte boundary is covered by aligned vectors
// all the same: its first and last vector are partly outside the row and masked.  A group's rows are a
// multiple of 8 apart, so they all start at the same place in a vector and a thread holds the same
// columns of each: gamma and beta are read once, and their gradients are summed in registers over the rows, then over
// the CTA in shared memory, and one partial row per CTA goes to the workspace; a second kernel adds the
// partial rows in a fixed order.  No atomics: the same bits on every run.
#include <cuda_bf16.h>

#include <algorithm>

#include "svg2_device.cuh"
#include "svg2_internal.h"

namespace svg2 {

namespace {

// Up to this many partial values are added by the CTA that comes last, more by a kernel of their own.
constexpr long long kNormFusedValues = 32768;

template <class T>
struct NormArgs {
  const T *X, *dY;
  const float *gamma, *beta;       // optional
  const float *mean_in, *rstd_in;  // backward
  float *mean, *rstd;              // forward, optional
  T* Y;                            // Y | dX
  float* partial;                  // backward: [gridDim.x][2][W]
  float *dgamma, *dbeta;           // backward, optional
  uint32_t* arrived;               // FUSED: CTAs whose partial row is written
  long long rows;
  int W;
  int x_mis;               // X's elements past a 16-byte boundary
  bool dy_same, y_same;    // dY, Y start at the same place in a vector as X: 16-byte accesses fit
  float eps;
};

template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// A vector as float pairs (the arithmetic runs on pairs: one instruction for two values).
__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = make_float2(bf16lo_to_f32(u[e]), bf16hi_to_f32(u[e]));
}
__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[2]) {
  v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
  v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[4]) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                    pack_bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[2]) {
  return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
}
template <int P>
__device__ __forceinline__ float element(const float2 (&v)[P], int e) { return (e & 1) ? v[e >> 1].y : v[e >> 1].x; }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

// Sums of K values over a group of G threads: G lanes of a warp, or (G = 0) the whole CTA.
// `turn` alternates the shared buffer between consecutive sums, so one barrier per sum is enough.
template <int G, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* buf, int& turn) {
  static_assert(K <= 8, "the shared buffer holds two sums of 8 values from 32 warps");
  constexpr int kWidth = G == 0 ? 32 : G;
#pragma unroll
  for (int o = kWidth / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (G == 0) {
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* b = buf + turn * 256;
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

// Where a thread works: vectors t, t + n, ... of rows first, first + stride, ...; `off` elements of the first
// vector lie before the row (the same for all its rows).
template <class T, int G>
struct Place {
  int t, n, off, nvec;
  long long first, stride;
  __device__ __forceinline__ Place(const NormArgs<T>& a) {
    constexpr int V = kVec<T>;
    n = G == 0 ? blockDim.x : G;
    t = threadIdx.x % n;
    if constexpr (G == 0) {
      first = blockIdx.x;
      stride = gridDim.x;
    } else {  // the groups of a warp are 8 rows apart, the 8 warps of a CTA take the rows between
      constexpr int kPerWarp = 32 / G;
      first = (static_cast<long long>(blockIdx.x) * kPerWarp + (threadIdx.x & 31) / G) * 8 + (threadIdx.x >> 5);
      stride = static_cast<long long>(gridDim.x) * kPerWarp * 8;
    }
    off = static_cast<int>((a.x_mis + first * a.W) % V);
    nvec = (off + a.W + V - 1) / V;
  }
  // first column of vector i of this thread (may be negative or reach past W)
  __device__ __forceinline__ int col(int i) const { return (t + i * n) * kVec<T> - off; }
  __device__ __forceinline__ bool has(int i) const { return t + i * n < nvec; }
};

// Starts the copy of the vector at column c of a row into this thread's slot; zeros where `in` is false.  EDGE:
// rows may start or end inside a vector.
template <class T, bool EDGE>
__device__ __forceinline__ void fetch_vec(uint4* slot, const T* X, bool same, bool in, long long row, int c,
                                          const NormArgs<T>& a) {
  constexpr int V = kVec<T>;
  const long long e0 = row * a.W + c;
  if constexpr (!EDGE) {
    cp_async16_zfill(smem_u32(slot), X + (in ? e0 : 0), in);
  } else if (!in || (same && e0 >= 0 && e0 + V <= a.rows * a.W)) {
    cp_async16_zfill(smem_u32(slot), X + (in ? e0 : 0), in);
  } else {  // the tensor's ends, or another alignment than X's: only the row's own elements
    T* s = reinterpret_cast<T*>(slot);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e >= 0 && c + e < a.W) s[e] = X[e0 + e];
  }
}

// The part of a vector that lies inside its row, the same for all rows of a thread: elements [lo, hi).
struct Span {
  int lo, hi;
};

// Bits of the elements inside the span, to clear what a neighbouring row left in the vector.
template <class T>
__device__ __forceinline__ uint4 span_bits(Span p) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[k] = (k >= p.lo && k < p.hi) ? 0xffffffffu : 0u;
    } else {
      w[k] = ((2 * k >= p.lo && 2 * k < p.hi) ? 0xffffu : 0u) | ((2 * k + 1 >= p.lo && 2 * k + 1 < p.hi) ? 0xffff0000u : 0u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 operator&(uint4 a, uint4 b) { return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w); }

template <class T, bool EDGE>
__device__ __forceinline__ void put_vec(T* Y, bool same, long long row, int c, Span in, const float2 (&v)[kVec<T> / 2],
                                        int W) {
  constexpr int V = kVec<T>;
  T* p = Y + row * W + c;
  if (!EDGE || (same && in.lo == 0 && in.hi == V)) {
    *reinterpret_cast<uint4*>(p) = pack(v);
  } else if (sizeof(T) == 2 && same && (in.lo == 0 || in.hi == V)) {
    // the row's first or last vector: its 1 to 7 elements as at most one store each of 2, 4 and 8 bytes
    const uint4 w = pack(v);
    char* q = reinterpret_cast<char*>(p);
    if (in.hi == V) {
      const int h = V - in.lo;
      if (h & 1) *reinterpret_cast<uint16_t*>(q + 2 * in.lo) = static_cast<uint16_t>((h > 4 ? (h > 6 ? w.x : w.y) : (h > 2 ? w.z : w.w)) >> 16);
      if (h & 2) *reinterpret_cast<uint32_t*>(q + (h & 4 ? 4 : 12)) = h & 4 ? w.y : w.w;
      if (h & 4) *reinterpret_cast<uint2*>(q + 8) = make_uint2(w.z, w.w);
    } else {
      const int h = in.hi;
      if (h & 4) *reinterpret_cast<uint2*>(q) = make_uint2(w.x, w.y);
      if (h & 2) *reinterpret_cast<uint32_t*>(q + (h & 4 ? 8 : 0)) = h & 4 ? w.z : w.x;
      if (h & 1) *reinterpret_cast<uint16_t*>(q + 2 * (h - 1)) = static_cast<uint16_t>(h > 4 ? (h > 6 ? w.w : w.z) : (h > 2 ? w.y : w.x));
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e >= in.lo && e < in.hi) store_one(p + e, element(v, e));
  }
}

// float32 parameters of a thread's columns (`none` where there are none)
template <int P>
__device__ __forceinline__ void load_param(const float* p, int c, int W, float none, float2 (&v)[P]) {
  auto one = [&](int i) { return (p != nullptr && i >= 0 && i < W) ? __ldg(p + i) : none; };
#pragma unroll
  for (int e = 0; e < P; ++e) v[e] = make_float2(one(c + 2 * e), one(c + 2 * e + 1));
}

template <class T, bool EDGE, int G, int NV, int R, int STAGES, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const NormArgs<T> a) {
  constexpr int V = kVec<T>, P = V / 2;
  extern __shared__ uint4 ring[];  // [STAGES][R][NV][blockDim.x]
  __shared__ float buf[512];
  const Place<T, G> at(a);
  const float inv_w = 1.f / static_cast<float>(a.W);
  int turn = 0;
  auto slot = [&](int stage, int r, int i) { return ring + ((stage * R + r) * NV + i) * blockDim.x + threadIdx.x; };
  auto fetch = [&](long long base, int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * at.stride + at.first;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        fetch_vec<T, EDGE>(slot(stage, r, i), a.X, true, row < a.rows && at.has(i), row, at.col(i), a);
    }
    cp_async_commit();
  };
  const long long step = at.stride * R;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s * step, s);
  float2 ga[NV][P], be[NV][P];  // of this thread's columns
  float2 keep[NV][P];            // 1 inside the row, 0 outside (EDGE)
  Span span[NV];
  uint4 bits[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    span[i] = Span{max(0, -at.col(i)), min(V, a.W - at.col(i))};
    bits[i] = span_bits<T>(span[i]);
#pragma unroll
    for (int e = 0; e < P; ++e)
      keep[i][e] = make_float2(2 * e >= span[i].lo && 2 * e < span[i].hi ? 1.f : 0.f,
                               2 * e + 1 >= span[i].lo && 2 * e + 1 < span[i].hi ? 1.f : 0.f);
    load_param(a.gamma, at.col(i), a.W, 1.f, ga[i]);
    load_param(a.beta, at.col(i), a.W, 0.f, be[i]);
  }
  int stage = 0;
  // the trip count is the same for all groups of a CTA: the sums are collective
  for (long long base = 0; base < a.rows; base += step) {
    fetch(base + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    cp_async_wait<STAGES - 1>();
    float2 x[R][NV][P];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack(EDGE ? *slot(stage, r, i) & bits[i] : *slot(stage, r, i), x[r][i]);
#pragma unroll
        for (int e = 0; e < P; ++e) t = add2(t, x[r][i][e]);
      }
      s[r] = t.x + t.y;
    }
    group_sum<G, R>(s, buf, turn);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv_w;
      const float2 neg = make_float2(-mean[r], -mean[r]);
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < P; ++e) x[r][i][e] = add2(x[r][i][e], neg);
        if (EDGE || at.has(i))
#pragma unroll
          for (int e = 0; e < P; ++e) t = fma2(x[r][i][e], EDGE ? mul2(x[r][i][e], keep[i][e]) : x[r][i][e], t);
      }
      s[r] = t.x + t.y;
    }
    group_sum<G, R>(s, buf, turn);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * at.stride + at.first;
      const float rstd = rsqrtf(fmaf(s[r], inv_w, a.eps));
      const float2 r2 = make_float2(rstd, rstd);
      if (row < a.rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!at.has(i)) continue;
          float2 y[P];
#pragma unroll
          for (int e = 0; e < P; ++e) y[e] = fma2(mul2(x[r][i][e], r2), ga[i][e], be[i][e]);
          put_vec<T, EDGE>(a.Y, a.y_same, row, at.col(i), span[i], y, a.W);
        }
        if (at.t == 0) {
          if (a.mean != nullptr) a.mean[row] = mean[r];
          if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// FUSED: the CTA that comes last adds up the partial rows (a kernel of its own for that: its code cost the main loop of
// the others 5 to 9 %).
template <class T, bool EDGE, int G, int NV, int R, int STAGES, int MAXT, bool FUSED>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormArgs<T> a) {
  constexpr int V = kVec<T>, P = V / 2;
  // [STAGES][R][2][NV][blockDim.x], then gamma of each thread's columns [NV][V / 4][blockDim.x]; at the end the
  // warps' column sums [8][2][W]
  extern __shared__ uint4 ring[];
  __shared__ float buf[512];
  const Place<T, G> at(a);
  const float inv_w = 1.f / static_cast<float>(a.W);
  int turn = 0;
  auto slot = [&](int stage, int r, int k, int i) {
    return ring + (((stage * R + r) * 2 + k) * NV + i) * blockDim.x + threadIdx.x;
  };
  auto gamma_slot = [&](int i, int q) {
    return reinterpret_cast<float4*>(ring + STAGES * R * 2 * NV * blockDim.x + (i * (V / 4) + q) * blockDim.x + threadIdx.x);
  };
  auto fetch = [&](long long base, int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * at.stride + at.first;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = row < a.rows && at.has(i);
        fetch_vec<T, EDGE>(slot(stage, r, 0, i), a.X, true, in, row, at.col(i), a);
        fetch_vec<T, EDGE>(slot(stage, r, 1, i), a.dY, a.dy_same, in, row, at.col(i), a);
      }
    }
    cp_async_commit();
  };
  const long long step = at.stride * R;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s * step, s);
  float2 dg[NV][P], db[NV][P];
  Span span[NV];
  uint4 bits[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    span[i] = Span{max(0, -at.col(i)), min(V, a.W - at.col(i))};
    bits[i] = span_bits<T>(span[i]);
    float2 p[P];
    load_param(a.gamma, at.col(i), a.W, 1.f, p);
#pragma unroll
    for (int q = 0; q < V / 4; ++q) *gamma_slot(i, q) = make_float4(p[2 * q].x, p[2 * q].y, p[2 * q + 1].x, p[2 * q + 1].y);
#pragma unroll
    for (int e = 0; e < P; ++e) dg[i][e] = db[i][e] = make_float2(0.f, 0.f);
  }
  int stage = 0;
  float mean[R], rstd[R];  // of the next rows, read ahead
  auto stats = [&](long long base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * at.stride + at.first;
      mean[r] = row < a.rows ? __ldg(a.mean_in + row) : 0.f;
      rstd[r] = row < a.rows ? __ldg(a.rstd_in + row) : 0.f;
    }
  };
  stats(0);
  for (long long base = 0; base < a.rows; base += step) {
    fetch(base + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    float m[R], rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = mean[r], rs[r] = rstd[r];
    stats(base + step);
    cp_async_wait<STAGES - 1>();
    float2 x[R][NV][P], g[R][NV][P];
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 neg = make_float2(-m[r], -m[r]), r2 = make_float2(rs[r], rs[r]);
      float2 t0 = make_float2(0.f, 0.f), t1 = t0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack(EDGE ? *slot(stage, r, 0, i) & bits[i] : *slot(stage, r, 0, i), x[r][i]);
        // (dY is 0 outside the row: nothing is added there)
        unpack(EDGE ? *slot(stage, r, 1, i) & bits[i] : *slot(stage, r, 1, i), g[r][i]);
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const float4 p4 = *gamma_slot(i, q);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int e = 2 * q + u;
            x[r][i][e] = mul2(add2(x[r][i][e], neg), r2);
            dg[i][e] = fma2(g[r][i][e], x[r][i][e], dg[i][e]);
            db[i][e] = add2(db[i][e], g[r][i][e]);
            g[r][i][e] = mul2(g[r][i][e], u == 0 ? make_float2(p4.x, p4.y) : make_float2(p4.z, p4.w));
            t0 = add2(t0, g[r][i][e]);
            t1 = fma2(g[r][i][e], x[r][i][e], t1);
          }
        }
      }
      s[2 * r] = t0.x + t0.y;
      s[2 * r + 1] = t1.x + t1.y;
    }
    group_sum<G, 2 * R>(s, buf, turn);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = base + r * at.stride + at.first;
      if (row >= a.rows) continue;
      const float c1 = -s[2 * r] * inv_w, c2 = -s[2 * r + 1] * inv_w;
      const float2 c12 = make_float2(c1, c1), c22 = make_float2(c2, c2), r2 = make_float2(rs[r], rs[r]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!at.has(i)) continue;
        float2 d[P];
#pragma unroll
        for (int e = 0; e < P; ++e) d[e] = mul2(r2, fma2(x[r][i][e], c22, add2(g[r][i][e], c12)));
        put_vec<T, EDGE>(a.Y, a.y_same, row, at.col(i), span[i], d, a.W);
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.W;
  if constexpr (G == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.col(i);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e >= 0 && c + e < a.W) {
          out[c + e] = element(dg[i], e);
          out[a.W + c + e] = element(db[i], e);
        }
    }
  } else {
    // over the groups of a warp by shuffles (they hold the same columns), over the 8 warps in shared memory
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* cols = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.col(i);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = element(dg[i], e), v = element(db[i], e);
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
          u += __shfl_xor_sync(0xffffffffu, u, o);
          v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        if (lane < G && c + e >= 0 && c + e < a.W) {
          cols[(warp * 2 + 0) * a.W + c + e] = u;
          cols[(warp * 2 + 1) * a.W + c + e] = v;
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.W; c += blockDim.x) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += cols[w * 2 * a.W + c];
      out[c] = s;
    }
  }
  if constexpr (!FUSED) return;
  // row by row in order, whichever CTA it is; the counter is left at zero for the next call
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int c = threadIdx.x; c < 2 * a.W; c += blockDim.x) {
    float* to = c < a.W ? a.dgamma : a.dbeta;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int r = 0;
    for (; r + 4 <= static_cast<int>(gridDim.x); r += 4)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += __ldcg(a.partial + static_cast<size_t>(r + u) * 2 * a.W + c);
    for (; r < static_cast<int>(gridDim.x); ++r) s[0] += __ldcg(a.partial + static_cast<size_t>(r) * 2 * a.W + c);
    if (to != nullptr) to[c < a.W ? c : c - a.W] = (s[0] + s[1]) + (s[2] + s[3]);
  }
  if (threadIdx.x == 0) *a.arrived = 0u;
}

// Rows of odd widths, many and short.  kVec rows of W elements are W whole 16-byte vectors wherever the tensor starts on
// one, so a warp copies that many rows at a time into its own shared memory, two stages, works on them there by
// single elements (lane l has columns l, l + 32, ...) and writes the results back over them, and to memory as whole vectors.
// Bound by its instructions for bf16 (0.35 to 0.63 of the copy bandwidth forward, 0.42 to 0.75 backward) and by memory for
// float32 (0.62 to 0.91).  In us, forward / backward, against the kernels above: bf16 2000000 x 77 237 / 302 (356 / 374), 1626016 x
// 123 239 / 294 (546 / 580), 391389 x 511 196 / 362 (432 / 636); float32 784313 x 255 294 / 428 (503 / 1049).
template <class T, int K, bool BWD>
__global__ void __launch_bounds__(128) norm_odd_kernel(const NormArgs<T> a) {
  constexpr int V = kVec<T>, NB = BWD ? 2 : 1, RU = K <= 4 ? 4 : (K <= 8 || !BWD ? 2 : 1);  // RU rows at a time
  extern __shared__ uint4 ring[];  // [warps][2 stages][X, dY][W]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, W = a.W;
  uint4* mine = ring + static_cast<size_t>(warp) * 2 * NB * W;
  const long long tiles = (a.rows + V - 1) / V, step = static_cast<long long>(gridDim.x) * warps;
  const float inv_w = 1.f / static_cast<float>(W);
  auto fetch = [&](long long tile, int stage) {
    if (tile < tiles) {
      const long long e0 = tile * V * W;
      uint4* to = mine + stage * NB * W;
      if (tile * V + V <= a.rows) {
        for (int v = lane; v < W; v += 32) {
          cp_async16_zfill(smem_u32(to + v), a.X + e0 + v * V, true);
          if (BWD) cp_async16_zfill(smem_u32(to + W + v), a.dY + e0 + v * V, true);
        }
      } else {  // the last rows: fewer than V
        const int n = static_cast<int>(a.rows - tile * V) * W;
        for (int e = lane; e < n; e += 32) {
          reinterpret_cast<T*>(to)[e] = a.X[e0 + e];
          if (BWD) reinterpret_cast<T*>(to + W)[e] = a.dY[e0 + e];
        }
      }
    }
    cp_async_commit();
  };
  auto load = [](T v) { return static_cast<float>(v); };
  long long tile = static_cast<long long>(blockIdx.x) * warps + warp;
  fetch(tile, 0);
  float ga[K], be[K], dg[BWD ? K : 1], db[BWD ? K : 1];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = lane + 32 * k;
    ga[k] = a.gamma != nullptr && c < W ? __ldg(a.gamma + c) : 1.f;
    be[k] = !BWD && a.beta != nullptr && c < W ? __ldg(a.beta + c) : 0.f;
    if (BWD) dg[BWD ? k : 0] = db[BWD ? k : 0] = 0.f;
  }
  // backward: lane r holds mean and rstd of row r of the next tile
  float mean_n = 0.f, rstd_n = 0.f;
  auto stats = [&](long long t) {
    const long long row = t * V + lane;
    const bool has = lane < V && row < a.rows;
    mean_n = has ? __ldg(a.mean_in + row) : 0.f;
    rstd_n = has ? __ldg(a.rstd_in + row) : 0.f;
  };
  if (BWD) stats(tile);
  int stage = 0, turn = 0;
  for (; tile < tiles; tile += step) {
    fetch(tile + step, stage ^ 1);
    const float mean_t = mean_n, rstd_t = rstd_n;
    if (BWD) stats(tile + step);
    cp_async_wait<1>();
    __syncwarp();
    uint4* vec = mine + stage * NB * W;
    T* xs = reinterpret_cast<T*>(vec);
    const T* gs = reinterpret_cast<const T*>(vec + W);
    const int rows = static_cast<int>(min(static_cast<long long>(V), a.rows - tile * V));
    for (int r = 0; r < rows; r += RU) {
      float x[RU][K], s[BWD ? 2 * RU : RU];
      if constexpr (!BWD) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          s[u] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            x[u][k] = r + u < rows && lane + 32 * k < W ? load(xs[(r + u) * W + lane + 32 * k]) : 0.f;
            s[u] += x[u][k];
          }
        }
        group_sum<32, RU>(s, nullptr, turn);
        float mean[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          mean[u] = s[u] * inv_w;
          s[u] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            x[u][k] = lane + 32 * k < W ? x[u][k] - mean[u] : 0.f;
            s[u] = fmaf(x[u][k], x[u][k], s[u]);
          }
        }
        group_sum<32, RU>(s, nullptr, turn);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          if (r + u >= rows) continue;
          const float rstd = rsqrtf(fmaf(s[u], inv_w, a.eps));
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (lane + 32 * k < W) store_one(xs + (r + u) * W + lane + 32 * k, fmaf(x[u][k] * rstd, ga[k], be[k]));
          if (lane == 0) {
            if (a.mean != nullptr) a.mean[tile * V + r + u] = mean[u];
            if (a.rstd != nullptr) a.rstd[tile * V + r + u] = rstd;
          }
        }
      } else {
        float g[RU][K], rs[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const float m = __shfl_sync(0xffffffffu, mean_t, (r + u) & (V - 1));
          rs[u] = __shfl_sync(0xffffffffu, rstd_t, (r + u) & (V - 1));
          s[2 * u] = s[2 * u + 1] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const bool in = r + u < rows && lane + 32 * k < W;
            const int e = (r + u) * W + lane + 32 * k;
            x[u][k] = in ? (load(xs[e]) - m) * rs[u] : 0.f;
            const float dy = in ? load(gs[e]) : 0.f;
            dg[k] = fmaf(dy, x[u][k], dg[k]);
            db[k] += dy;
            g[u][k] = dy * ga[k];
            s[2 * u] += g[u][k];
            s[2 * u + 1] = fmaf(g[u][k], x[u][k], s[2 * u + 1]);
          }
        }
        group_sum<32, 2 * RU>(s, nullptr, turn);
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          if (r + u >= rows) continue;
          const float c1 = -s[2 * u] * inv_w, c2 = -s[2 * u + 1] * inv_w;
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (lane + 32 * k < W) store_one(xs + (r + u) * W + lane + 32 * k, rs[u] * fmaf(x[u][k], c2, g[u][k] + c1));
        }
      }
    }
    __syncwarp();
    T* out = a.Y + tile * V * W;
    if (rows == V) {
      for (int v = lane; v < W; v += 32) reinterpret_cast<uint4*>(out)[v] = vec[v];
    } else {
      for (int e = lane; e < rows * W; e += 32) out[e] = xs[e];
    }
    __syncwarp();  // (the next copies into this stage come after every lane's reads)
    stage ^= 1;
  }
  cp_async_wait<0>();
  if constexpr (BWD) {  // the warps' column sums, added in order
    float* cols = reinterpret_cast<float*>(ring);  // [warps][2][W]
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (lane + 32 * k < W) {
        cols[(warp * 2 + 0) * W + lane + 32 * k] = dg[k];
        cols[(warp * 2 + 1) * W + lane + 32 * k] = db[k];
      }
    __syncthreads();
    float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * W;
    for (int c = threadIdx.x; c < 2 * W; c += blockDim.x) {
      float s = 0.f;
      for (int w = 0; w < warps; ++w) s += cols[w * 2 * W + c];
      out[c] = s;
    }
  }
}

// Below, a warp's lanes are mostly idle (bf16 2000000 x 37: 208 us against 178; float32 x 21: 197 against 96); above, two
// stages of so many rows leave few warps resident.
constexpr int kNormOddFrom = 65, kNormOddTo = 512;

template <class T, bool BWD>
cudaError_t run_norm_odd(const NormArgs<T>& a, int max_parts, int* parts, cudaStream_t s) {
  auto* kernel = a.W <= 96    ? norm_odd_kernel<T, 3, BWD>
                 : a.W <= 128 ? norm_odd_kernel<T, 4, BWD>
                 : a.W <= 192 ? norm_odd_kernel<T, 6, BWD>
                 : a.W <= 256 ? norm_odd_kernel<T, 8, BWD>
                 : a.W <= 384 ? norm_odd_kernel<T, 12, BWD>
                              : norm_odd_kernel<T, 16, BWD>;
  const int warps = a.W <= 256 ? 4 : 2;
  const int smem = warps * 2 * (BWD ? 2 : 1) * a.W * 16;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  int resident = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, 32 * warps, smem);
  if (e != cudaSuccess) return e;
  const long long tiles = (a.rows + kVec<T> - 1) / kVec<T>;
  long long grid = std::min((tiles + warps - 1) / warps, static_cast<long long>(kNormSms) * std::max(1, resident));
  if (BWD) grid = std::min(grid, static_cast<long long>(max_parts));
  *parts = static_cast<int>(grid);
  kernel<<<static_cast<unsigned>(grid), 32 * warps, smem, s>>>(a);
  return cudaGetLastError();
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

template <class T, bool BWD, bool EDGE, int G, int NV, int R, int STAGES, int MAXT>
cudaError_t run_norm(const NormArgs<T>& a, int threads, int max_parts, int* parts, cudaStream_t s) {
  constexpr int V = kVec<T>;
  auto* kernel = BWD ? norm_bwd_kernel<T, EDGE, G, NV, R, STAGES, MAXT, false> : norm_fwd_kernel<T, EDGE, G, NV, R, STAGES, MAXT>;
  const int per_cta = G == 0 ? 1 : threads / G;
  size_t smem = static_cast<size_t>(STAGES) * R * (BWD ? 2 : 1) * NV * threads * 16;
  if (BWD) smem += static_cast<size_t>(NV) * V * threads * 4;
  if (BWD && G != 0) smem = std::max(smem, static_cast<size_t>(16) * a.W * 4);
  cudaError_t e = cudaSuccess;
  long long grid = (a.rows + per_cta - 1) / per_cta;
  const bool fused = BWD && grid <= kNormSms && grid * 2 * a.W <= kNormFusedValues;
  if (fused) kernel = norm_bwd_kernel<T, EDGE, G, NV, R, STAGES, MAXT, true>;
  // (48 KB, less the static buffer, need no permission)
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (grid > kNormSms) {  // as many CTAs as are resident at once
    int resident = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    const long long most = static_cast<long long>(kNormSms) * std::max(1, std::min(resident, kNormMaxPerSm));
    if (grid > most) grid = most;
  }
  if (BWD && grid > max_parts) grid = max_parts;
  if (EDGE && G == 0 && grid < a.rows) grid = std::max(8LL, grid / 8 * 8);  // a CTA's rows are a multiple of 8 apart
  *parts = static_cast<int>(grid);
  if (fused) *parts = 0;
  kernel<<<static_cast<unsigned>(grid), threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <class T, bool BWD, bool EDGE>
cudaError_t pick_norm(const NormArgs<T>& a, int max_parts, int* parts, cudaStream_t s) {
  constexpr int V = kVec<T>;
  // vectors that cover a row, wherever it starts
  const int nvec = EDGE ? (V - 1 + a.W + V - 1) / V : a.W / V;
  auto cta = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
  // Rows at a time (R) and ring stages (S) are the fastest of a sweep over R in 1, 2, 4, S in 2, 3, 4 and, for a CTA
  // per row, 1 to 5 vectors a thread: more rows share a barrier, more registers leave fewer CTAs resident.
  // bf16, 3024000 x 128: forward 254 us (R = 2, S = 2) against 299 to 309 for the others, backward 367 us (R = 1, S = 4)
  // against 391 to 423; 75600 x 5120: forward 241 us (5 vectors, R = 2) against 247 to 371, backward 418 us
  // (5 vectors, R = 1) against 424 to 553; 200000 x 1024: 135 and 218 us (2 vectors, R = 4) against 141 to 165 and
  // 219 to 272.  Copying the same bytes takes 237, 355, 237, 355, 125 and 188 us.
  constexpr int R1 = BWD ? 1 : 2, S1 = BWD ? 4 : 2;
  if (nvec <= 8) return run_norm<T, BWD, EDGE, 8, 1, R1, S1, 256>(a, 256, max_parts, parts, s);
  if (nvec <= 16) return run_norm<T, BWD, EDGE, 16, 1, R1, S1, 256>(a, 256, max_parts, parts, s);
  if (nvec <= 32) return run_norm<T, BWD, EDGE, 32, 1, R1, S1, 256>(a, 256, max_parts, parts, s);
  if (nvec <= 64) return run_norm<T, BWD, EDGE, 32, 2, 1, BWD ? 3 : 2, 256>(a, 256, max_parts, parts, s);
  if (nvec <= 256) {
    if constexpr (BWD && EDGE) return run_norm<T, BWD, EDGE, 0, 2, 1, 4, 128>(a, cta(2), max_parts, parts, s);
    else if constexpr (V == 8) return run_norm<T, BWD, EDGE, 0, 2, 4, 2, 128>(a, cta(2), max_parts, parts, s);
    else return run_norm<T, BWD, EDGE, 0, 1, 4, 2, 256>(a, cta(1), max_parts, parts, s);
  }
  if (nvec <= 1024) return run_norm<T, BWD, EDGE, 0, 5, BWD ? 1 : 2, BWD ? 3 : 2, 224>(a, cta(5), max_parts, parts, s);
  // (at most 8192 columns: 1025 vectors of bf16, 2049 of float32)
  return run_norm<T, BWD, EDGE, 0, 4, 1, 2, V == 8 ? 288 : 544>(a, cta(4), max_parts, parts, s);
}

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
  a.dgamma = n.dgamma;
  a.dbeta = n.dbeta;
  a.arrived = n.arrived;
  auto mis = [](const void* p) { return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)); };
  a.x_mis = mis(n.X);
  a.dy_same = mis(n.dY) == a.x_mis;
  a.y_same = mis(n.Y) == a.x_mis;
  int parts = 0;
  const int max_parts = norm_max_parts(n.rows);
  const bool edge = a.W % kVec<T> != 0 || a.x_mis != 0 || !a.y_same || (bwd && !a.dy_same);
  // many odd rows that start together on 16 bytes
  const bool odd = edge && a.x_mis == 0 && a.y_same && (!bwd || a.dy_same) && a.W >= kNormOddFrom && a.W <= kNormOddTo &&
                   a.rows >= 4LL * kNormSms * kVec<T>;
  cudaError_t e = odd ? (bwd ? run_norm_odd<T, true>(a, max_parts, &parts, s) : run_norm_odd<T, false>(a, max_parts, &parts, s))
                  : bwd ? (edge ? pick_norm<T, true, true>(a, max_parts, &parts, s)
                              : pick_norm<T, true, false>(a, max_parts, &parts, s))
                      : (edge ? pick_norm<T, false, true>(a, max_parts, &parts, s)
                              : pick_norm<T, false, false>(a, max_parts, &parts, s));
  if (e == cudaSuccess && parts > 0 && bwd && (n.dgamma != nullptr || n.dbeta != nullptr)) {
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
