// Gradients of the dense and the variable-block sparse attention on tcgen05 tensor cores.
//
// With s_ij = scale q_i.k_j, P_ij = exp(s_ij - lse_i) (the forward's probabilities, recomputed from its
// log-sum-exp, so no maximum is needed) and delta_i = dO_i.O_i:
//   dV = P^T dO,   dS = P o (dO V^T - delta),   dK = scale dS^T Q,   dQ = scale dS K.
// dK, dV sum over queries and dQ over keys, so the work is cut into two kinds of unit, both with 128
// resident rows and a stream of 128-row tiles, and every output row has one owner: no atomics, the
// same bits on every run, no float32 copy of dQ in memory.  The price is that S and dP are computed
// twice (7 products per tile pair where one pass with atomic dQ sums would take 5).
//   key unit    K, V of 128 rows of one K cluster stay in shared memory; Q, dO of the Q clusters that
//               keep it stream by.  S^T = K Q^T, dP^T = V dO^T; P^T and dS^T go back to TMEM as the A
//               operands of dV += P^T dO and dK += dS^T Q.
//   query unit  Q, dO of 128 rows of one Q cluster stay; K, V of its kept clusters stream by.
//               S = Q K^T, dP = dO V^T; dS goes back to TMEM as the A operand of dQ += dS K.
// The streams are packed as in the forward: the kept clusters' rows back to back, so ragged cluster
// edges cost no padding; rows past the stream's end are zeros.
//   warps 0-7   P and dS: TMEM lanes = resident rows, warps 0-3 the tile's columns 0-63, 4-7 64-127
//   warp 8      TMEM allocator and MMA issuer
//   warps 9-11  (9 alone when dense) range table, then the tiles' producers
// P and dS are rounded to bf16 for the products (as P is in the forward); both stay float32 until then.
// A row of dS sums to zero, so dQ does not depend on what all keys have in common; the rounded dS, with delta
// from a bf16 O, sums to some r_i instead, and dQ would carry scale r_i times that common part, which
// in a trained K is often its largest.  The query unit therefore sums the dS values it hands over and
// subtracts scale r_i c, c = the mean of the keys that the row keeps (any c is right in exact arithmetic): on keys
// with a mean of four standard deviations the error of dQ falls from 1.0e-2 to 2.6e-3 of its norm.  A mean over other
// keys too would let large ones among them into rows that do not keep them (one cluster of 40 that is 300 away: dQ off by half
// its norm), so the sparse call has a mean for every Q cluster.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "svg2_device.cuh"
#include "svg2_internal.h"

namespace svg2 {

namespace {

// 12 warps in three warpgroups: 8 for P and dS, then the MMA and producer warps.
constexpr int kBwdThreads = 384;
// Register split after set-up (setmaxnreg): 256 x 176 + 128 x 152 = 64512 = 384 x 168, the launch's
// allocation under __launch_bounds__(384, 1).  The one split in steps of 8 at which neither side spills
// (168: the P and dS loop does; 184: the MMA warp's descriptors do).
constexpr int kBwdLaunchRegs = 168, kBwdSoftmaxRegs = 176, kBwdOtherRegs = 152;
static_assert(256 * kBwdSoftmaxRegs + (kBwdThreads - 256) * kBwdOtherRegs <= kBwdThreads * kBwdLaunchRegs,
              "register split");
constexpr int kBwdMmaWarp = 8, kBwdProducerWarp = 9;
constexpr int kBwdMaxRanges = 1024;
constexpr uint32_t kGatherSleep = 32;
constexpr float kLog2e = 1.4426950408889634f;
// Of every 16 column pairs, this many get 2^x from the cubic on the FMA pipe, the rest from the MUFU.  Dense: P and
// dS follow one another in the same warps, so the exponentials' time counts in full (2 x 75600 x 128: 15.0 ms with 8
// in both kinds of unit, 15.3 to 15.6 with 4 or 10 in one of them).  Sparse: the three gathering warps issue from the same
// schedulers, and the cubic's instructions cost more than the MUFU saves (2 x 75600 x 128: 6.12 ms with 0, 6.22 with
// 2, 6.26 with 4, 6.45 with 6, 6.59 with 8; 8 x 12480 in 64 / 256 clusters: 1.88 against 2.03 ms with 8).
constexpr int kBwdCubicDense = 8, kBwdCubicSparse = 0;

template <int D>
constexpr uint32_t bwd_tile_bytes() { return 128u * D * 2u; }
// One more step of the S and dP products, 16 deep, adds what depends on the streamed row alone (key unit) or masks pairs
// (MULTI units), so that the warps that compute P and dS read nothing but TMEM: their loads from shared memory
// wait behind the products' operand reads.  The resident side A holds ones in columns 0-2 and in column 4 + c for
// the rows of the unit's cluster c; the streamed side B holds
//   S, columns 0-2   -lse / scale as three bf16 (24 bits), so that S' = S - lse / scale      (key unit)
//   S, column 4 + c  the penalty -3.4e38 where cluster c does not keep the streamed row        (MULTI)
//   dP, columns 0-2  -delta as three bf16, so that dP' = dP - delta                             (key unit)
// and zeros elsewhere.  Both [128, 16], K-major without swizzle: the first 8 columns of all rows, 16 bytes each, then
// the other 8.
constexpr uint32_t kStepBytes = 4096, kStepPlane = 2048;
constexpr int kBwdMaxSegments = 12;
constexpr uint32_t kSegPenalty = 0xff7fu;  // bf16 -3.39e38

// Stages of the streamed tiles: four tiles fit at d = 128.  T1 waits from its S product to the unit's last product
// of the tile, T2 only from dP (to dV), so three and one let T1 arrive a period early: 8 x 12480 x 128 takes 1.75 ms
// against 1.92 with two of each.  (At d = 64 more would fit; four of each gained nothing.)
constexpr int kStages1 = 3, kStages2 = 1, kStreamTiles = kStages1 + kStages2;
constexpr uint32_t kBarBytes = 384;  // barriers, and what else a CTA shares

template <int D>
constexpr uint32_t bwd_smem() {
  return (2 + kStreamTiles) * bwd_tile_bytes<D>() + 1024 /*align*/ + 2048 /*row sums*/ + 4096 /*range starts*/ +
         4096 + 64 /*range offsets*/ + 2048 /*range segments*/ + (1 + kStreamTiles) * kStepBytes /*A, B of S and dP by stage*/ +
         kBarBytes;
}
static_assert(bwd_smem<128>() <= 227 * 1024, "shared memory");

// Column 4 + c of a row's S operand: the penalty where bit c of `keep` is clear.
__device__ __forceinline__ void store_seg(uint8_t* b, int row, uint32_t keep) {
  uint32_t w[6];
#pragma unroll
  for (int k = 0; k < 6; ++k)
    w[k] = ((keep >> (2 * k)) & 1u ? 0u : kSegPenalty) | ((keep >> (2 * k + 1)) & 1u ? 0u : kSegPenalty << 16);
  *reinterpret_cast<uint2*>(b + row * 16 + 8) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint4*>(b + kStepPlane + row * 16) = make_uint4(w[2], w[3], w[4], w[5]);
}
// v as the sum of three bf16 (the first alone when it is not finite), then five zeros
__device__ __forceinline__ uint4 three_bf16(float v) {
  const uint32_t hi = pack_bf16x2(v, 0.f) & 0xffffu;
  const float r1 = v - __uint_as_float(hi << 16);
  const uint32_t mid = pack_bf16x2(r1, 0.f) & 0xffffu;
  const uint32_t lo = pack_bf16x2(r1 - __uint_as_float(mid << 16), 0.f) & 0xffffu;
  const bool finite = fabsf(__uint_as_float(hi << 16)) < INFINITY;
  return make_uint4(finite ? hi | (mid << 16) : hi, finite ? lo : 0u, 0u, 0u);
}

// Streams of up to this many tiles hand P and dS over as two bf16 numbers each (the rounding, and the rest) and take a
// product more for each; one-tile streams also take delta as sum_j P_ij dP_ij instead of from the bf16 O
// (the key unit only when it holds every key, dense N <= 128).  Short rows average fewer rounding errors and often
// hold like keys, and there the products are not what takes the time: over random short rows (2 to 512 keys)
// the worst error of dQ and dK falls from 5.8e-3 and 3.0e-2 to 4.9e-3 and 2.1e-3 of their norms.
constexpr int kBwdSplitTiles = 4;
// Query units with streams up to this long do so for the second chunk of every tile (template SPLIT = 1; 2: both
// chunks): dQ is then 2.1 to 2.2e-3 of its norm off instead of 2.45 to 2.6e-3 (1.66e-3 is its own rounding), for 0 to 2 %
// of the gradients' time on 6 x 1333 x 64 and 1 x 4096 x 64 sparse, 7 to 14 % on 24 x 4096 x 64 and 8 x 2500 x 128.  Longer
// streams, where the products are all of the time, stay at 2.4 to 2.5e-3.
constexpr int kBwdHalfSplitTiles = 32;

struct BwdMaps {  // Q, K, V, dO by [plane, row, column]: boxes of 128 rows x 64 columns, 128-byte swizzle
  CUtensorMap m[4];
};

struct BwdArgs {
  const int32_t *q_off, *k_off;     // null: dense
  const uint32_t *keepers, *kept;   // the selection as bits, by K cluster and by Q cluster
  const BwdUnit *k_units, *q_units;                    // [BH, per_head]
  const int32_t *perm_q, *perm_k;
  const float *neg_lse2, *neg_delta;                   // [BH, N] -lse log2(e), -delta, by permuted row
  const uint4 *lse_step, *delta_step;                  // [BH, N] three_bf16 of -lse / scale, of -delta
  const float* center;                                 // dense [BH, D], sparse [BH, nQ, D]
  const __nv_bfloat16 *Q, *K, *V, *dO;                 // the tensors of the maps
  __nv_bfloat16 *dQ, *dK, *dV;
  int BH, N, nQ, nK, k_per_head, q_per_head;
  float scale;
  DeviceStatus* st;
  const uint64_t* wait_budget;
};

struct BwdBars {
  uint64_t res_full, t1_full[kStages1], t2_full[kStages2], t1_empty[kStages1], t2_empty[kStages2], s_full[2], p_full[2], dp_full, ds_full[2], o_full,
      mma_done;
  uint32_t tmem_base;
  int32_t L;
  uint8_t seg[128];  // sparse query unit: each row's cluster, counted from the unit's first
};
static_assert(sizeof(BwdBars) <= kBarBytes, "shared memory");


// ------------------------------------------------------------------------------------------------
// delta_i = dO_i . O_i and the scaled log-sum-exp, by permuted row; with perm, dO's rows in permuted
// order too.  D / 8 lanes per row, 16 bytes each: bound by the reads of O and dO.  The first CTAs take
// the mean of up to kMeanRows evenly spaced K rows each, of a plane (dense) or of a K cluster.
// ------------------------------------------------------------------------------------------------
constexpr int kMeanRows = 512;
// From this many rows per K cluster on a CTA takes a cluster's mean, below a warp does (plain means, gradients of 24 x 4096 x 128
// in 1024 clusters: 1490 us with warps, 1537 with CTAs; 1 x 4096 x 64 in 32: 71.2 with warps, 66.8 with CTAs).
constexpr int kMeanWide = 64;

// Keys far from the others that a row's softmax gives nothing must not move what its dQ subtracts either: with 10 % of
// the keys 300 away and of no weight the plain mean put dQ off by 7e-2 of its norm, 2.4e-3 now.  So the values within one standard
// deviation of the mean are averaged again, column by column (of two groups the smaller one lies past that), and where the
// plain mean is further from theirs than twice their own standard deviation, theirs counts.  (Nothing here knows the weights: a
// group that is taken for far and has weight costs its rows up to twice the error.)
struct MeanSums {  // of a column; first pass: sum, sum of squares, number; second: the same of x - mean, of those within reach
  float a, b, n;
};
__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) < INFINITY ? x : 0.f; }
__device__ __forceinline__ float first_mean(MeanSums s) { return s.n > 0.f ? finite_or_0(s.a / s.n) : 0.f; }
__device__ __forceinline__ float mean_reach(MeanSums s, float mean) {
  const float var = s.b / fmaxf(s.n, 1.f) - mean * mean;
  return var < INFINITY ? sqrtf(fmaxf(var, 0.f)) : INFINITY;
}
// x with weight w; a NaN or infinity stays with the rows that keep its key
__device__ __forceinline__ void add_within(MeanSums& s, float x, float mean, float reach, float w) {
  x -= mean;
  if (fabsf(x) <= reach && fabsf(x) < INFINITY) {
    s.a = fmaf(w, x, s.a);
    s.b = fmaf(w * x, x, s.b);
    s.n += w;
  }
}
__device__ __forceinline__ float settle_mean(float plain, float mean, MeanSums s) {
  if (!(s.n > 0.f)) return plain;
  const float off = s.a / s.n, d = plain - (mean + off);
  return d * d > 4.f * (s.b / s.n - off * off) ? finite_or_0(mean + off) : plain;
}

// floor(t n / S) without a 64-bit division
__device__ __forceinline__ int spaced_row(int t, int n, int S) {
  return t * (n / S) + static_cast<int>(static_cast<unsigned>(t * (n % S)) / static_cast<unsigned>(S));
}
template <class F>
__device__ __forceinline__ void each_value(uint4 w, F&& take) {  // take(column of eight, value)
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    take(2 * e, bf16lo_to_f32(u[e]));
    take(2 * e + 1, bf16hi_to_f32(u[e]));
  }
}

// The mean of up to kMeanRows evenly spaced rows of the n >= 1 from row0 on, by a CTA; kMeanSample of them stand for
// all where the values within reach are looked for.
constexpr int kMeanSample = 64;

template <int D>
__device__ __forceinline__ void mean_wide(const uint4* __restrict__ K, long long row0, int n, float* __restrict__ mean) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes, kPicks = kMeanSample / kGroups;
  constexpr int kPer = 256 / D;  // threads per column in the end
  __shared__ float part[kGroups][D];
  __shared__ uint4 sample[kMeanSample][kLanes];
  const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int S = min(n, kMeanRows), each = (S + kGroups - 1) / kGroups;  // a group's rows follow one another
  const int t0 = group * each, t1 = min(S, t0 + each);
#pragma unroll
  for (int k = 0; k < kPicks; ++k) {
    const int i = k * each / kPicks, t = t0 + i;
    const bool is = t < t1 && (k == 0 || i > (k - 1) * each / kPicks);
    sample[k * kGroups + group][sub] = is ? __ldg(K + (row0 + spaced_row(t, n, S)) * kLanes + sub)
                                          : make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);  // NaN: none
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
  for (int t = t0; t < t1; ++t)
    each_value(__ldg(K + (row0 + spaced_row(t, n, S)) * kLanes + sub), [&](int e, float x) { acc[e] += finite_or_0(x); });
#pragma unroll
  for (int e = 0; e < 8; ++e) part[group][sub * 8 + e] = acc[e];
  __syncthreads();
  const int col = threadIdx.x / kPer, h = threadIdx.x % kPer;  // a column's threads are neighbours
  auto over_threads = [&](float v) {
#pragma unroll
    for (int o = 1; o < kPer; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  auto total = [&](MeanSums s) { return MeanSums{over_threads(s.a), over_threads(s.b), over_threads(s.n)}; };
  float plain = 0.f, v[kMeanSample / kPer];
#pragma unroll
  for (int g = 0; g < kGroups / kPer; ++g) plain += part[g * kPer + h][col];
  plain = finite_or_0(over_threads(plain) / static_cast<float>(S));
  const __nv_bfloat16* values = reinterpret_cast<const __nv_bfloat16*>(sample);
  MeanSums s{0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < kMeanSample / kPer; ++r) {
    v[r] = __bfloat162float(values[(r * kPer + h) * D + col]);
    add_within(s, v[r], 0.f, INFINITY, 1.f);
  }
  s = total(s);
  const float m = first_mean(s), reach = mean_reach(s, m);
  s = MeanSums{0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < kMeanSample / kPer; ++r) add_within(s, v[r], m, reach, 1.f);
  s = total(s);
  if (h == 0) mean[col] = settle_mean(plain, m, s);
}

// The same by a warp, for few rows: all of the up to kMeanRows are looked at twice.
template <int D>
__device__ __forceinline__ void mean_warp(const uint4* __restrict__ K, long long row0, int n, float* __restrict__ mean) {
  constexpr int kLanes = D / 8, kGroups = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, S = min(n, kMeanRows);
  MeanSums s[8];
  float m[8], reach[8];
  auto pass = [&](auto&& take) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = MeanSums{0.f, 0.f, 0.f};
#pragma unroll 4
    for (int t = lane / kLanes; t < S; t += kGroups)
      each_value(__ldg(K + (row0 + spaced_row(t, n, S)) * kLanes + sub), take);
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[e].a += __shfl_xor_sync(0xffffffffu, s[e].a, o);
        s[e].b += __shfl_xor_sync(0xffffffffu, s[e].b, o);
        s[e].n += __shfl_xor_sync(0xffffffffu, s[e].n, o);
      }
  };
  pass([&](int e, float x) { add_within(s[e], x, 0.f, INFINITY, 1.f); });
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = first_mean(s[e]);
    reach[e] = mean_reach(s[e], m[e]);
  }
  if (S > 2) pass([&](int e, float x) { add_within(s[e], x, m[e], reach[e], 1.f); });
  if (lane < kLanes)
#pragma unroll
    for (int e = 0; e < 8; ++e) mean[sub * 8 + e] = S > 2 ? settle_mean(m[e], m[e], s[e]) : m[e];
}

// Rows of cluster i by its plane's offsets; malformed ones hold none.
__device__ __forceinline__ int cluster_rows(const int32_t* off, int i, int N) {
  const int start = off[i], n = off[i + 1] - start;
  return start < 0 || n <= 0 || start > N - n ? 0 : n;
}

__host__ __device__ __forceinline__ unsigned mean_ctas_of(int BH, int n, bool wide) {
  const unsigned count = static_cast<unsigned>(BH) * n;
  return wide ? count : (count + 7) / 8;
}

template <int D>
__global__ void __launch_bounds__(256, 4) bwd_prep_kernel(const uint4* __restrict__ O, const uint4* __restrict__ dO,
                                                       const float* __restrict__ lse, const int32_t* __restrict__ perm,
                                                       const uint4* __restrict__ K, int N, long long rows,
                                                       int BH, float* __restrict__ neg_lse2,
                                                       float* __restrict__ neg_delta, uint4* __restrict__ lse_step,
                                                       uint4* __restrict__ delta_step, float inv_scale,
                                                       uint4* __restrict__ dOp, const int32_t* __restrict__ k_off,
                                                       int nK, bool wide, float* __restrict__ means,
                                                       DeviceStatus* st) {
  // means: of BH planes (k_off null), or of their nK clusters each, by a CTA or (wide false) by a warp
  const unsigned mean_ctas = mean_ctas_of(BH, k_off != nullptr ? nK : 1, wide);
  if (blockIdx.x < mean_ctas) {
    const unsigned i = wide ? blockIdx.x : blockIdx.x * 8 + threadIdx.x / 32;
    int bh = i, start = 0, n = N;
    if (k_off != nullptr) {
      if (i >= static_cast<unsigned>(BH) * nK) return;
      bh = i / nK;
      const int j = i % nK;
      const int32_t* off = k_off + static_cast<size_t>(bh) * (nK + 1);
      start = off[j];
      n = cluster_rows(off, j, N);
      if (n == 0) return;  // (its mean is not read)
    }
    const long long row0 = static_cast<long long>(bh) * N + start;
    float* mean = means + static_cast<size_t>(i) * D;
    if (wide) mean_wide<D>(K, row0, n, mean);
    else mean_warp<D>(K, row0, n, mean);
    return;
  }
  constexpr int kLanes = D / 8, kPerWarp = 32 / kLanes, kUnroll = 2;
  const int sub = threadIdx.x % kLanes;
  const unsigned total = static_cast<unsigned>(rows);  // below 2^31
  const unsigned step = (gridDim.x - mean_ctas) * 8u * kPerWarp;
  // every lane of a warp takes part in the shuffles: rows past the end only skip their memory
  for (unsigned r0 = ((blockIdx.x - mean_ctas) * 8u + threadIdx.x / 32) * kPerWarp; r0 < total; r0 += kUnroll * step) {
    uint4 o[kUnroll], g[kUnroll];
    float l[kUnroll];
    unsigned src[kUnroll];
    bool valid[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const unsigned r = r0 + u * step + (threadIdx.x % 32) / kLanes;
      valid[u] = r < total;
      src[u] = r;
      if (valid[u] && perm != nullptr) {
        const int t = perm[r];
        SVG2_DEBUG_CHECK(t >= 0 && t < N, st, kWhereGather, r, t);
        valid[u] = t >= 0 && t < N;  // a bad entry has no output row, so no gradient either
        src[u] = r / static_cast<unsigned>(N) * static_cast<unsigned>(N) + t;
      }
      l[u] = r < total && sub == 0 ? lse[r] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      o[u] = g[u] = make_uint4(0, 0, 0, 0);
      if (valid[u]) {
        o[u] = O[static_cast<size_t>(src[u]) * kLanes + sub];
        g[u] = dO[static_cast<size_t>(src[u]) * kLanes + sub];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const unsigned r = r0 + u * step + (threadIdx.x % 32) / kLanes;
      float acc = 0.f;
      const uint32_t ow[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc = fmaf(bf16lo_to_f32(ow[e]), bf16lo_to_f32(gw[e]), acc);
        acc = fmaf(bf16hi_to_f32(ow[e]), bf16hi_to_f32(gw[e]), acc);
      }
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
      if (r >= total) continue;
      if (dOp != nullptr) dOp[static_cast<size_t>(r) * kLanes + sub] = g[u];
      if (sub == 0) {
        const bool empty = l[u] == -INFINITY;  // a row without keys: P = 0 (and it is in no stream)
        neg_lse2[r] = empty ? -INFINITY : -l[u] * kLog2e;
        neg_delta[r] = -acc;
        lse_step[r] = three_bf16(empty ? 0.f : -l[u] * inv_scale);
        delta_step[r] = three_bf16(-acc);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// The sparse plan, one CTA per (b,h): the selection as bits both ways, and the units of both kinds.  A K
// cluster listed twice for one Q cluster, or an index out of range, latches SVG2_ERR_DEVICE_BOUNDS: the
// gradient kernel then does nothing.
//
// A unit costs as many tiles as its stream is long, however few of its 128 rows are used, and clusters
// rarely end on a multiple of 128.  So what is left of a cluster after its full tiles shares a unit with the
// rows that follow; the joint stream is the union of the clusters' streams, and the pairs that a row's own
// cluster does not keep are masked.
// ------------------------------------------------------------------------------------------------

// One warp packs clusters [c0, c1) into units, lane w holding word w of the clusters' bits; lane 0 calls
// emit(i, unit) in order.
//
// A unit takes t rows of the next cluster where that shortens the streams, in words of the clusters' bits.  It adds what
// the cluster's stream has beyond the unit's, and a quarter (kMaskCost / 16) of the joint stream where the unit is
// the first time of several clusters, of the addition later: the masking, and a last wave with fewer and longer units.
// It saves a unit of the cluster's own stream if the cluster needs one less (the room that is left counts a third of
// that, for the rows to come); if not, half of what t of a unit's 128 rows cost.  Gradients in us with a cost of 0, 2, 4, 6
// sixteenths: 2 x 75600 in 100 / 500 clusters, 28 % kept, 6784, 6379, 5803, 6026 (5884 without sharing); 8 x 12480 in 64 / 256,
// 60 %: 2016, 1886, 1883, 2057 (2330); 3 x 20000 in 300 / 300, 30 %: 1432, 1429, 1173, 1146 (1154); with the room counted, 4 x
// 16000 in 400 / 64, 40 %: 1344 -> 1201.
constexpr int kMaskCost = 4;

template <class Emit>
__device__ __forceinline__ void pack_units(const int32_t* off, const uint32_t* bits, int W, int c0, int c1, int N,
                                          Emit&& emit) {
  const int lane = threadIdx.x & 31;
  int count = 0;
  int first = 0, row0 = 0, rows = 0, last = 0;  // the unit that can still take rows (rows = 0: none)
  uint32_t joint = 0u;                          // what any of its clusters keeps or is kept by
  int end = off[c0];
  for (int j = c0; j < c1; ++j) {
    const uint32_t mine = lane < W ? bits[j * W + lane] : 0u;
    int start = end;
    end = off[j + 1];
    int left = end - start;
    if (start < 0 || left <= 0 || start > N - left) continue;  // empty, or malformed offsets
    if (rows > 0 && rows < 128 && row0 + rows == start && j - first < kBwdMaxSegments) {
      const int t = min(128 - rows, left);
      const int added = __reduce_add_sync(0xffffffffu, __popc(mine & ~joint));
      const int all = __reduce_add_sync(0xffffffffu, __popc(mine | joint));
      const int mask = kMaskCost * (last > first ? added : all);
      const int own = __reduce_add_sync(0xffffffffu, __popc(mine));
      const int gain = ((left - t + 127) >> 7) < ((left + 127) >> 7) ? 16 * own + own * (128 - rows - t) / 24
                                                                           : t * all / 16;
      if (16 * added + mask < gain) {
        rows += t;
        last = j;
        joint |= mine;
        start += t;
        left -= t;
      }
    }
    if (left > 0) {
      if (rows > 0) {
        if (lane == 0) emit(count, BwdUnit{first, row0, rows, last - first + 1});
        ++count;
      }
      for (; left >= 128; start += 128, left -= 128) {
        if (lane == 0) emit(count, BwdUnit{j, start, 128, 1});
        ++count;
      }
      first = last = j;
      row0 = start;
      rows = left;
      joint = mine;
    }
  }
  if (rows > 0) {
    if (lane == 0) emit(count, BwdUnit{first, row0, rows, last - first + 1});
  }
}

constexpr int kPlanRun = 32;  // clusters that one warp packs; units do not cross runs (at most 31 units of a plane)
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr size_t kPlanSmem = 200 * 1024;  // the selection's bits both ways, if they fit
// Up to this much of it two CTAs fit an SM, and those of the kept keys' means go beside the planning ones, with four
// warps per Q cluster (8 x 12480 in 64 / 256 clusters: both 33 us, 45 with two warps, 73 with one).  Otherwise they have a launch
// of their own, a warp per Q cluster (24 x 4096 in 1024 / 1024: 165 us, 204 with four warps).
constexpr int kCenterWarps = 4;
constexpr size_t kPlanBesideSmem = 96 * 1024;

__device__ __forceinline__ void columns(float4 v, float (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
__device__ __forceinline__ void columns(float2 v, float (&x)[2]) { x[0] = v.x, x[1] = v.y; }

// The mean of the keys that a Q cluster keeps, from the means of the K clusters (settled as for the rows of one): W
// warps per Q cluster, row = plane nQ + cluster, each with every W-th 32 of its list, d / 32 columns per lane.  0 for a
// cluster that keeps none.  W > 1: all threads of a CTA call it; part: [warps][P][32 lanes].
template <class V, int P, int W>  // V: the vector of P columns
__device__ __forceinline__ void center_cluster(const int32_t* __restrict__ k_off, const int32_t* __restrict__ sel_count,
                                               const int32_t* __restrict__ sel_idx, int N, int nQ, int nK, int rows,
                                               int row, const float* __restrict__ cluster_mean,
                                               float* __restrict__ center, MeanSums* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warp0 = warp / W * W;
  const bool has = row < rows;
  const int bh = has ? row / nQ : 0, cnt = has ? min(max(sel_count[row], 0), nK) : 0;
  const int32_t* off = k_off + static_cast<size_t>(bh) * (nK + 1);
  const int32_t* list = sel_idx + static_cast<size_t>(has ? row : 0) * nK;
  const V* means = reinterpret_cast<const V*>(cluster_mean) + static_cast<size_t>(bh) * nK * 32 + lane;
  MeanSums s[P];
  auto pass = [&](auto&& take) {  // take(column, its cluster mean, the cluster's rows); s: the sums over all warps
#pragma unroll
    for (int p = 0; p < P; ++p) s[p] = MeanSums{0.f, 0.f, 0.f};
    for (int e0 = 32 * (warp - warp0); e0 < cnt; e0 += 32 * W) {
      int j = e0 + lane < cnt ? list[e0 + lane] : -1;
      const int n = j >= 0 && j < nK ? cluster_rows(off, j, N) : 0;
      if (n == 0) j = -1;
      for (int t0 = 0; t0 < min(32, cnt - e0); t0 += 8)
#pragma unroll
        for (int t = t0; t < t0 + 8; ++t) {
          const int k = __shfl_sync(0xffffffffu, j, t);
          const float w = static_cast<float>(__shfl_sync(0xffffffffu, n, t));
          const V m = k >= 0 ? __ldg(means + static_cast<size_t>(k) * 32) : V{};
          float x[P];
          columns(m, x);
#pragma unroll
          for (int p = 0; p < P; ++p) take(p, x[p], w);
        }
    }
    if constexpr (W > 1) {
      __syncthreads();  // (the sums of the pass before have been read)
#pragma unroll
      for (int p = 0; p < P; ++p) part[(warp * P + p) * 32 + lane] = s[p];
      __syncthreads();
#pragma unroll
      for (int p = 0; p < P; ++p) {
        s[p] = MeanSums{0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const MeanSums o = part[((warp0 + w) * P + p) * 32 + lane];
          s[p].a += o.a, s[p].b += o.b, s[p].n += o.n;
        }
      }
    }
  };
  float mean[P], reach[P], c[P];
  pass([&](int p, float x, float w) { add_within(s[p], x, 0.f, INFINITY, w); });
#pragma unroll
  for (int p = 0; p < P; ++p) {
    mean[p] = first_mean(s[p]);
    reach[p] = mean_reach(s[p], mean[p]);
  }
  pass([&](int p, float x, float w) { add_within(s[p], x, mean[p], reach[p], w); });
  if (!has || warp != warp0) return;
  V* out = reinterpret_cast<V*>(center) + static_cast<size_t>(row) * 32 + lane;
#pragma unroll
  for (int p = 0; p < P; ++p) c[p] = settle_mean(mean[p], mean[p], s[p]);
  if constexpr (P == 4) *out = make_float4(c[0], c[1], c[2], c[3]);
  else *out = make_float2(c[0], c[1]);
}

template <int W>
__device__ __forceinline__ void center_row(const int32_t* k_off, const int32_t* sel_count, const int32_t* sel_idx, int N,
                                           int nQ, int nK, int d, int rows, int row, const float* cluster_mean, float* center,
                                           MeanSums* part) {
  if (d == 128) center_cluster<float4, 4, W>(k_off, sel_count, sel_idx, N, nQ, nK, rows, row, cluster_mean, center, part);
  else center_cluster<float2, 2, W>(k_off, sel_count, sel_idx, N, nQ, nK, rows, row, cluster_mean, center, part);
}

__global__ void __launch_bounds__(256)
    bwd_center_kernel(const int32_t* __restrict__ k_off, const int32_t* __restrict__ sel_count,
                      const int32_t* __restrict__ sel_idx, int N, int nQ, int nK, int d, int rows,
                      const float* __restrict__ cluster_mean, float* __restrict__ center) {
  center_row<1>(k_off, sel_count, sel_idx, N, nQ, nK, d, rows, blockIdx.x * 8 + threadIdx.x / 32, cluster_mean, center, nullptr);
}

// The first BH CTAs make the plans, others (if any) the means of the kept keys.
__global__ void __launch_bounds__(kPlanThreads)
    bwd_plan_kernel(const int32_t* __restrict__ q_off, const int32_t* __restrict__ k_off,
                    const int32_t* __restrict__ sel_count, const int32_t* __restrict__ sel_idx, int N, int nQ, int nK,
                    uint32_t* keepers, uint32_t* kept, bool kept_in_smem, BwdUnit* __restrict__ k_units,
                    int k_per_head, BwdUnit* __restrict__ q_units, int q_per_head, int BH, int d,
                    const float* __restrict__ cluster_mean, float* __restrict__ center, DeviceStatus* st) {
  extern __shared__ uint32_t k_bits[];  // [nK, WQ], then [nQ, WK] if it fits, else [32 warps][WK]
  __shared__ int32_t k_offsets[kMaxClustersAssign + 1], q_offsets[kMaxClustersAssign + 1];
  __shared__ uint32_t k_rows[kPlanWarps], q_rows[kPlanWarps];  // the clusters that have rows
  if (static_cast<int>(blockIdx.x) >= BH) {
    center_row<kCenterWarps>(k_off, sel_count, sel_idx, N, nQ, nK, d, BH * nQ,
                             (blockIdx.x - BH) * (kPlanWarps / kCenterWarps) + threadIdx.x / (32 * kCenterWarps), cluster_mean,
                             center, reinterpret_cast<MeanSums*>(k_bits));
    return;
  }
  const int WQ = (nQ + 31) / 32, WK = (nK + 31) / 32;
  const int bh = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int w = threadIdx.x; w < nK * WQ; w += kPlanThreads) k_bits[w] = 0u;
  BwdUnit* ku = k_units + static_cast<size_t>(bh) * k_per_head;
  BwdUnit* qu = q_units + static_cast<size_t>(bh) * q_per_head;
  for (int i = threadIdx.x; i < k_per_head; i += kPlanThreads) ku[i] = BwdUnit{0, 0, 0, 0};
  for (int i = threadIdx.x; i < q_per_head; i += kPlanThreads) qu[i] = BwdUnit{0, 0, 0, 0};
  for (int i = threadIdx.x; i <= nK; i += kPlanThreads) k_offsets[i] = k_off[static_cast<size_t>(bh) * (nK + 1) + i];
  for (int i = threadIdx.x; i <= nQ; i += kPlanThreads) q_offsets[i] = q_off[static_cast<size_t>(bh) * (nQ + 1) + i];
  __syncthreads();
  {
    static_assert(kMaxClustersAssign <= kPlanThreads, "a thread per cluster");
    const int c = threadIdx.x;
    const uint32_t k = __ballot_sync(0xffffffffu, c < nK && cluster_rows(k_offsets, c, N) > 0);
    const uint32_t q = __ballot_sync(0xffffffffu, c < nQ && cluster_rows(q_offsets, c, N) > 0);
    if (lane == 0) k_rows[warp] = k, q_rows[warp] = q;
  }
  __syncthreads();
  uint32_t* kept_g = kept + static_cast<size_t>(bh) * nQ * WK;
  uint32_t* q_bits_s = k_bits + nK * WQ;
  for (int i = warp; i < nQ; i += kPlanWarps) {
    const size_t row = static_cast<size_t>(bh) * nQ + i;
    uint32_t* mine = q_bits_s + (kept_in_smem ? i : warp) * WK;
    for (int w = lane; w < WK; w += 32) mine[w] = 0u;
    __syncwarp();
    int cnt = sel_count[row];
    if (cnt < 0 || cnt > nK) {
      if (lane == 0) raise_status(st, kStatusDeviceBounds, kWherePlan, i, cnt);
      cnt = 0;
    }
    for (int e0 = lane; e0 < cnt; e0 += 256) {  // eight loads in flight
      int j[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) j[u] = e0 + 32 * u < cnt ? __ldg(sel_idx + row * nK + e0 + 32 * u) : -1;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (e0 + 32 * u >= cnt) break;
        const uint32_t bit = 1u << (i & 31);
        if (j[u] < 0 || j[u] >= nK || (atomicOr(&k_bits[j[u] * WQ + (i >> 5)], bit) & bit) != 0u)
          raise_status(st, kStatusDeviceBounds, kWherePlan, i, j[u]);
        else
          atomicOr(&mine[j[u] >> 5], 1u << (j[u] & 31));
      }
    }
    __syncwarp();
    // Clusters without rows keep nothing and are kept by nothing: a unit may span an empty cluster, whose part of the
    // selection would lengthen its stream, and the packing counts bits.
    const bool has = (q_rows[i >> 5] >> (i & 31)) & 1u;
    for (int w = lane; w < WK; w += 32) kept_g[i * WK + w] = mine[w] = has ? mine[w] & k_rows[w] : 0u;
    __syncwarp();
  }
  __syncthreads();
  for (int w = threadIdx.x; w < nK * WQ; w += kPlanThreads) {
    const int j = w / WQ;
    const bool has = (k_rows[j >> 5] >> (j & 31)) & 1u;
    keepers[static_cast<size_t>(bh) * nK * WQ + w] = k_bits[w] = has ? k_bits[w] & q_rows[w - j * WQ] : 0u;
  }
  __syncthreads();
  // units: a run's go from the slot that the runs before it cannot reach (a run of n clusters and m rows has at
  // most n + m / 128), the slots between stay empty
  const int runs_k = (nK + kPlanRun - 1) / kPlanRun, runs_q = (nQ + kPlanRun - 1) / kPlanRun;
  const uint32_t* q_bits = kept_in_smem ? q_bits_s : kept_g;
  for (int r = warp; r < runs_k + runs_q; r += kPlanWarps) {
    const bool k = r < runs_k;
    const int c0 = (k ? r : r - runs_k) * kPlanRun;
    const int32_t* off = k ? k_offsets : q_offsets;
    const int base = min(max(off[c0], 0), N) / 128 + c0, most = k ? k_per_head : q_per_head;
    BwdUnit* out = k ? ku : qu;
    pack_units(off, k ? k_bits : q_bits, k ? WQ : WK, c0, min(k ? nK : nQ, c0 + kPlanRun), N,
               [&](int i, const BwdUnit& u) {
                 if (base + i < most) out[base + i] = u;
               });
  }
  for (int i = threadIdx.x; i < nK; i += kPlanThreads) SVG2_DEBUG_CHECK(k_offsets[i] >= 0 && k_offsets[i + 1] >= k_offsets[i] && k_offsets[i + 1] <= N, st, kWherePlan, i, k_offsets[i]);
  for (int i = threadIdx.x; i < nQ; i += kPlanThreads) SVG2_DEBUG_CHECK(q_offsets[i] >= 0 && q_offsets[i + 1] >= q_offsets[i] && q_offsets[i + 1] <= N, st, kWherePlan, i, q_offsets[i]);
}

// ------------------------------------------------------------------------------------------------
// One unit.  KV: a key unit (dK, dV), else a query unit (dQ).  R1, R2: resident tiles (K, V | Q, dO);
// T1, T2: streamed tiles (Q, dO | K, V).
// ------------------------------------------------------------------------------------------------
// TMEM columns: S (the query unit alternates between two slots), dP, and the accumulators.  P and dS
// (bf16) overwrite their S and dP: column half h puts its 64 values at the half's first 32 columns, which
// only its own warps have read.
template <bool KV>
struct BwdTmem {
  static constexpr uint32_t s1 = 128;                 // query unit: second S slot
  static constexpr uint32_t acc1 = 128;               // key unit: dV
  static constexpr uint32_t dp = 256, acc2 = 384;     // acc2: dK | dQ
};

template <int D, bool DENSE, bool KV, int SPLIT, bool MULTI>
__device__ __forceinline__ void bwd_unit(const BwdMaps& maps, const BwdArgs& a, const BwdUnit un, const int bh,
                                         uint8_t* smem, BwdBars* bars, float* stats, const int32_t* r_start,
                                         const int32_t* r_cum, const uint16_t* r_seg, uint8_t* step_s, float* scratch, const long long wb) {
  constexpr uint32_t kTile = bwd_tile_bytes<D>();
  constexpr int kHalves = D / 64;   // 128-byte swizzle atoms across a row
  constexpr int kSteps = D / 16;    // instructions of one S or dP product
  using Tm = BwdTmem<KV>;
  constexpr int S1 = kStages1, S2 = kStages2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = bars->tmem_base;
  const int L = bars->L;
  const int T = (L + 127) / 128;
  DeviceStatus* st = a.st;
  const uint32_t r1 = smem_u32(smem), r2 = r1 + kTile, t1 = r1 + 2 * kTile, t2 = t1 + S1 * kTile;

  if (warp == kBwdMmaWarp) {
    if (elect_one() && T > 0) {
      const uint32_t id_s = idesc_bf16_f32(128, 128, 0);  // both operands K-major
      const uint32_t id_o = idesc_bf16_f32(128, D, 1);    // B = a streamed tile read row-major (MN-major)
      // D[slot] = R x T^T, contraction over d, and the step's columns (B at `step`, 0: none)
      const uint32_t step_a = smem_u32(step_s), step_b = step_a + kStepBytes;  // B of S by stage of T1, then of dP by stage of T2
      auto product = [&](uint32_t d_tmem, uint32_t ra, uint32_t tb, uint32_t step) {
        const uint64_t da = sdesc_sw128(ra, 16, 1024), db = sdesc_sw128(tb, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const uint64_t off = static_cast<uint64_t>(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
          mma_ss(d_tmem, da + off, db + off, id_s, ks > 0 ? 1u : 0u);
        }
        if (step != 0u)
          mma_ss(d_tmem, sdesc_plain(step_a, kStepPlane, 128), sdesc_plain(step, kStepPlane, 128), id_s, 1u);
      };
      auto s_step = [&](int stage) { return KV || MULTI ? step_b + stage * kStepBytes : 0u; };
      auto dp_step = [&](int stage) { return KV ? step_b + (S1 + stage) * kStepBytes : 0u; };
      // acc (+)= X T with X (P or dS, bf16) in TMEM, contraction over the tile's 128 rows, in the two chunks in
      // which X is handed over: rows 0-31 and 64-95, then 32-63 and 96-127
      auto accumulate = [&](uint32_t acc, uint32_t x, uint32_t tb, int chunk, bool add) {
        const uint64_t db = sdesc_sw128(tb, 16384, 1024);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int ks = 2 * chunk + (u & 1) + (u >> 1) * 4;
          mma_ts(acc, x + (ks >> 2) * 64 + (ks & 3) * 8, db + static_cast<uint64_t>((ks * 16 * 128) >> 4), id_o,
                 (add || u > 0) ? 1u : 0u);
        }
      };
      auto wait = [&](uint64_t* bar, int phase) {
        return mbar_wait(smem_u32(bar), phase & 1, st, kWhereAttnBwdMma, wb);
      };
      auto wait_tile = [&](uint64_t* bar, int phase) {
        const bool landed = wait(bar, phase);
        if (!DENSE) fence_proxy_async_smem();  // rows gathered by cp.async, segments stored (generic proxy)
        return landed;
      };
      bool ok = wait(&bars->res_full, 0) && wait_tile(&bars->t1_full[0], 0);
      if (ok) {
        tc_fence_after();
        product(tmem, r1, t1, s_step(0));
        mma_commit(smem_u32(&bars->s_full[0]));
        ok = wait_tile(&bars->t2_full[0], 0);
      }
      if (ok) {
        tc_fence_after();
        product(tmem + Tm::dp, r2, t2, dp_step(0));
        mma_commit(smem_u32(&bars->dp_full));
        if (!KV) mma_commit(smem_u32(&bars->t2_empty[0]));
      }
      // stage and phase of tile j + 1 (c1, c2: of tile j)
      int c1 = 0, c2 = 0, g1 = S1 > 1 ? 1 : 0, g2 = S2 > 1 ? 1 : 0, ph1 = S1 > 1 ? 0 : 1, ph2 = S2 > 1 ? 0 : 1;
      for (int j = 0; j < T && ok; ++j) {
        const bool more = j + 1 < T;
        if constexpr (KV) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (ok) ok = wait(&bars->p_full[c], j);
            if (!ok) break;
            tc_fence_after();
            accumulate(tmem + Tm::acc1, tmem, t2 + c2 * kTile, c, j > 0 || c > 0);  // dV += P^T dO
            if constexpr (SPLIT == 2) accumulate(tmem + Tm::acc1, tmem + 32, t2 + c2 * kTile, c, true);
          }
          if (!ok) break;
          mma_commit(smem_u32(&bars->t2_empty[c2]));
        }
        if (more) {
          // key unit: the products run in issue order, so S(j+1) overwrites P(j) only after dV has read it;
          // query unit: the other slot, whose S(j-1) was read before dS(j-1) was handed over
          ok = wait_tile(&bars->t1_full[g1], ph1);
          if (!ok) break;
          tc_fence_after();
          const int slot = KV ? 0 : (j + 1) & 1;
          product(tmem + slot * Tm::s1, r1, t1 + g1 * kTile, s_step(g1));
          mma_commit(smem_u32(&bars->s_full[slot]));
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (ok) ok = wait(&bars->ds_full[c], j);
          if (!ok) break;
          tc_fence_after();
          accumulate(tmem + Tm::acc2, tmem + Tm::dp, t1 + c1 * kTile, c, j > 0 || c > 0);  // dK += dS^T Q | dQ += dS K
          if (SPLIT > 1 - c) accumulate(tmem + Tm::acc2, tmem + Tm::dp + 32, t1 + c1 * kTile, c, true);
        }
        if (!ok) break;
        mma_commit(smem_u32(&bars->t1_empty[c1]));
        if (more) {
          ok = wait_tile(&bars->t2_full[g2], ph2);
          if (!ok) break;
          tc_fence_after();
          product(tmem + Tm::dp, r2, t2 + g2 * kTile, dp_step(g2));
          mma_commit(smem_u32(&bars->dp_full));
          if (!KV) mma_commit(smem_u32(&bars->t2_empty[g2]));
        }
        c1 = g1;
        c2 = g2;
        if (++g1 == S1) g1 = 0, ph1 ^= 1;
        if (++g2 == S2) g2 = 0, ph2 ^= 1;
      }
      if (ok) mma_commit(smem_u32(&bars->o_full));
      mma_commit(smem_u32(&bars->mma_done));
      mbar_wait(smem_u32(&bars->mma_done), 0, nullptr, kWhereAttnBwdMma, kWaitBudgetCycles / 8);
    }
  } else if (warp == kBwdProducerWarp || (!DENSE && warp > kBwdProducerWarp)) {
    // ---------------- resident and streamed tiles ----------------
    // A tile that is one contiguous piece comes by TMA: every dense tile (its rows past the plane's end are
    // zero-filled), and a sparse one inside a range.  A sparse tile of several pieces is gathered with
    // 16-byte cp.async copies by warps 9 to 11 (rows 0-47, 48-87, 88-127): as TMA boxes, one run per piece,
    // the single issuing thread took 1.6 times the tile's products at 49 rows per cluster.
    const int pw = warp - kBwdProducerWarp;
    const bool leader = pw == 0 && elect_one();
    const CUtensorMap* m1 = &maps.m[KV ? 0 : 1];
    const CUtensorMap* m2 = &maps.m[KV ? 3 : 2];
    if (leader && T > 0) {
      const uint32_t bar = smem_u32(&bars->res_full);
      mbar_arrive_expect_tx(bar, 2 * kTile);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        tma_load_3d(r1 + h * 16384, &maps.m[KV ? 1 : 0], h * 64, un.row0, bh, bar);
        tma_load_3d(r2 + h * 16384, &maps.m[KV ? 2 : 3], h * 64, un.row0, bh, bar);
      }
    }
    auto tma_tile = [&](const CUtensorMap* m, uint32_t dst, uint32_t bar, int row, uint32_t more_bytes) {
      mbar_arrive_expect_tx(bar, kTile + more_bytes);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) tma_load_3d(dst + h * 16384, m, h * 64, row, bh, bar);
    };
    const size_t plane = static_cast<size_t>(bh) * a.N;
    const uint32_t step_b = smem_u32(step_s) + kStepBytes;  // B of S by stage of T1, then of dP by stage of T2
    int n1 = 0, n2 = 0;  // tiles requested of each streamed operand
    bool ok = true;
    // `round`: how often the stage was filled before
    auto wait_empty = [&](uint64_t* bar, int round) {
      return round == 0 || __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(bar), (round - 1) & 1, st,
                                                                   kWhereAttnBwdProducer, DENSE ? 100 : kGatherSleep, wb));
    };
    int g1 = 0, g2 = 0, round1 = 0, round2 = 0;  // stage of tile j and its round
    if constexpr (DENSE) {
      for (int j = 0; j < T; ++j) {
        const uint32_t b1 = smem_u32(&bars->t1_full[g1]), b2 = smem_u32(&bars->t2_full[g2]);
        // the rows' step operands: as many as the plane still has (columns past it are masked)
        const uint32_t bytes = KV ? min(128, a.N - j * 128) * 16u : 0u;
        ok = wait_empty(&bars->t1_empty[g1], round1);
        if (!ok) break;
        if (leader) {
          tma_tile(m1, t1 + g1 * kTile, b1, j * 128, bytes);
          if (KV) bulk_load(step_b + g1 * kStepBytes, a.lse_step + plane + j * 128, bytes, b1);
        }
        n1 = j + 1;
        ok = wait_empty(&bars->t2_empty[g2], round2);
        if (!ok) break;
        if (leader) {
          tma_tile(m2, t2 + g2 * kTile, b2, j * 128, bytes);
          if (KV) bulk_load(step_b + (S1 + g2) * kStepBytes, a.delta_step + plane + j * 128, bytes, b2);
        }
        n2 = j + 1;
        if (++g1 == S1) g1 = 0, ++round1;
        if (++g2 == S2) g2 = 0, ++round2;
      }
    } else {
      constexpr int CPR = D / 8;           // 16-byte chunks per row
      constexpr int RPI = 32 / CPR;        // rows per warp instruction
      constexpr int kIters = 48 / RPI;     // at most this many instructions per tile and operand
      constexpr int kPeriod = 8 / RPI;     // the row's place in its 8-row swizzle group repeats this often
      const int wr0 = pw == 0 ? 0 : (pw == 1 ? 48 : 88), nrw = pw == 0 ? 48 : 40;
      const int chunk = lane % CPR, sub = lane / CPR;
      uint32_t xo[kPeriod];  // this thread's byte offset within a tile, less it * RPI * 128
#pragma unroll
      for (int k = 0; k < kPeriod; ++k)
        xo[k] = (chunk >> 3) * 16384 + (wr0 + sub) * 128 + (((chunk & 7) ^ ((k * RPI + sub) & 7)) << 4);
      const __nv_bfloat16* s1 = (KV ? a.Q : a.K) + plane * D + chunk * 8;
      const __nv_bfloat16* s2 = (KV ? a.dO : a.V) + plane * D + chunk * 8;
      int e0 = 0, e1 = 0, et = 0;  // ranges of this lane's two stream positions and of the tile's first
      auto src_row = [&](int p, int& e) {
        if (p >= L) return -1;
        while (r_cum[e + 1] <= p) ++e;
        return r_start[e] + (p - r_cum[e]);
      };
      for (int j = 0; j < T; ++j) {
        const uint32_t b1 = smem_u32(&bars->t1_full[g1]), b2 = smem_u32(&bars->t2_full[g2]);
        const int ra = src_row(j * 128 + wr0 + lane, e0), rb = src_row(j * 128 + wr0 + 32 + lane, e1);
        while (r_cum[et + 1] <= j * 128) ++et;
        const bool whole = r_cum[et + 1] >= j * 128 + 128;
        const int first = r_start[et] + (j * 128 - r_cum[et]);
        int rows_it[kIters];
        if (!whole) {
#pragma unroll
          for (int it = 0; it < kIters; ++it)
            if (it * RPI < nrw) rows_it[it] = __shfl_sync(0xffffffffu, it * RPI < 32 ? ra : rb, (it * RPI + sub) & 31);
        }
        auto gather = [&](uint32_t dst, const __nv_bfloat16* src) {
#pragma unroll
          for (int it = 0; it < kIters; ++it) {
            if (it * RPI >= nrw) break;
            const int r = rows_it[it];
            cp_async16_zfill(dst + xo[it % kPeriod] + it * RPI * 128, src + static_cast<size_t>(max(r, 0)) * D, r >= 0);
          }
        };
        ok = wait_empty(&bars->t1_empty[g1], round1);
        if (!ok) break;
        if (whole) {
          if (leader) tma_tile(m1, t1 + g1 * kTile, b1, first, 0u);
        } else {
          if (leader) mbar_arrive(b1);
          gather(t1 + g1 * kTile, s1);
        }
        // a stream row's step operand: of the query (key unit), then its segments (MULTI; 8 bytes hold the three bf16)
        auto row_step = [&](uint32_t dst, const uint4* src, int c, int r) {
          const uint4* from = src + plane + max(r, 0);
          if (MULTI) cp_async8_zfill(dst + c * 16, from, r >= 0);
          else cp_async16_zfill(dst + c * 16, from, r >= 0);
        };
        if constexpr (KV) {
          row_step(step_b + g1 * kStepBytes, a.lse_step, wr0 + lane, ra);
          if (32 + lane < nrw) row_step(step_b + g1 * kStepBytes, a.lse_step, wr0 + 32 + lane, rb);
        }
        cp_async_mbar_arrive(b1);
        if constexpr (MULTI) {  // (plain stores: an arrival of their own orders them)
          auto segs = [&](int c, int r, int e) {
            if (r >= 0) store_seg(step_s + (1 + g1) * kStepBytes, c, r_seg[e]);
          };
          segs(wr0 + lane, ra, e0);
          if (32 + lane < nrw) segs(wr0 + 32 + lane, rb, e1);
          fence_proxy_async_smem();
        }
        mbar_arrive(b1);
        n1 = j + 1;
        ok = wait_empty(&bars->t2_empty[g2], round2);
        if (!ok) break;
        if (whole) {
          if (leader) tma_tile(m2, t2 + g2 * kTile, b2, first, 0u);
        } else {
          if (leader) mbar_arrive(b2);
          gather(t2 + g2 * kTile, s2);
        }
        if constexpr (KV) {
          row_step(step_b + (S1 + g2) * kStepBytes, a.delta_step, wr0 + lane, ra);
          if (32 + lane < nrw) row_step(step_b + (S1 + g2) * kStepBytes, a.delta_step, wr0 + 32 + lane, rb);
        }
        cp_async_mbar_arrive(b2);
        n2 = j + 1;
        if (++g1 == S1) g1 = 0, ++round1;
        if (++g2 == S2) g2 = 0, ++round2;
      }
    }
    // Every copy has landed before the CTA leaves, also when some agent gave up: the last phase of each
    // stage's barrier is awaited here (older phases are complete, or the stage would not have been reused).
    cp_async_wait<0>();
    if (leader && T > 0) {
      const long long drain = kWaitBudgetCycles / 8;
      mbar_wait(smem_u32(&bars->res_full), 0, nullptr, kWhereAttnBwdProducer, drain);
      for (int g = 0; g < S1; ++g)
        if (const int fills = (n1 + S1 - 1 - g) / S1; fills > 0)
          mbar_wait(smem_u32(&bars->t1_full[g]), (fills - 1) & 1, nullptr, kWhereAttnBwdProducer, drain);
      for (int g = 0; g < S2; ++g)
        if (const int fills = (n2 + S2 - 1 - g) / S2; fills > 0)
          mbar_wait(smem_u32(&bars->t2_full[g]), (fills - 1) & 1, nullptr, kWhereAttnBwdProducer, drain);
    }
  } else if (warp < 8) {
    // ---------------- P and dS, then the unit's rows of the gradients ----------------
    const int half = warp >> 2;  // columns 64 half .. 64 half + 63 of every tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sl2 = a.scale * kLog2e;
    const float2 scl = make_float2(sl2, sl2);
    const size_t plane = static_cast<size_t>(bh) * a.N;
    float nl_row = 0.f, nd_row = 0.f;
    if (!KV && row < un.nrows) {
      nl_row = a.neg_lse2[plane + un.row0 + row];
      nd_row = a.neg_delta[plane + un.row0 + row];
    }
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase & 1, st, kWhereAttnBwdSoftmax, wb));
    };
    const bool exact_delta = SPLIT == 2 && T == 1 && (!KV || (DENSE && a.N <= 128));
    auto all_softmax_warps = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    auto hand_over = [&](uint64_t* bar) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(bar));
    };
    float2 r_sum = make_float2(0.f, 0.f);  // query unit: this half's sum of the row's rounded dS
    bool ok = true;
    // Every tile goes in two chunks of 32 columns: the loads of the second run under the first's arithmetic, and
    // the MMA warp starts on the first while the second is computed.
    for (int j = 0; j < T; ++j) {
      ok = KV ? wait(&bars->s_full[0], j) : wait(&bars->s_full[j & 1], j >> 1);
      const uint32_t t_s = tmem + lane_off + (KV ? 0u : (j & 1) * Tm::s1) + half * 64;
      const uint32_t t_dp = tmem + lane_off + Tm::dp + half * 64;
      uint32_t sv[64];
      float2 p[32];
      if (ok) {
        tc_fence_after();
        tmem_ld32p(t_s, sv);
        tmem_wait_ld();
        tmem_ld32p(t_s + 32, sv + 32);
        if constexpr (KV && SPLIT == 2) tmem_wait_ld();  // (the rests of P's first chunk go where S's second chunk is)
        const int valid = L - j * 128 - half * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 1) tmem_wait_ld();
          if (valid < 64) {  // past the stream's end: P = 0, or 2^-126 by the cubic (times rows of zeros)
#pragma unroll
            for (int e = 32 * c; e < 32 * c + 32; ++e)
              if (e >= valid) sv[e] = __float_as_uint(-INFINITY);
          }
          // P = 2^(s log2(e) - lse log2(e)); in a key unit S' holds the lse already
#pragma unroll
          for (int e = 16 * c; e < 16 * c + 16; ++e) {
            const float2 x = make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1]));
            const float2 t = KV ? mul2(x, scl) : fma2(x, scl, make_float2(nl_row, nl_row));
            // A NaN query (or lse) is a NaN column of a key unit: only P brings it to dV.  In a query unit it is the whole row,
            // which has MUFU columns, and a NaN key makes dS K one whatever its P.  (2 x 75600: 15.35 ms, 15.20 without
            // the NaN form.)
            p[e] = ((e & 15) >= 16 - (DENSE ? kBwdCubicDense : kBwdCubicSparse)) ? (KV ? exp2_cubic2_nan(t) : exp2_cubic2(t))
                                                                                   : make_float2(fast_exp2(t.x), fast_exp2(t.y));
          }
          if constexpr (KV) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = pack_bf16x2(p[16 * c + e].x, p[16 * c + e].y);
            tmem_st16(t_s + 16 * c, pk);
            if constexpr (SPLIT == 2) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                pk[e] = pack_bf16x2(p[16 * c + e].x - bf16lo_to_f32(pk[e]), p[16 * c + e].y - bf16hi_to_f32(pk[e]));
              tmem_st16(t_s + 32 + 16 * c, pk);
            }
            hand_over(&bars->p_full[c]);
          }
        }
        ok = wait(&bars->dp_full, j);  // (does not depend on this tile's P)
      }
      if (!ok) {
        if (exact_delta) {  // (the warps that got further meet here)
          all_softmax_warps();
          if constexpr (KV) all_softmax_warps();
        }
        break;
      }
      tc_fence_after();
      tmem_ld32p(t_dp, sv);
      tmem_wait_ld();
      tmem_ld32p(t_dp + 32, sv + 32);
      if constexpr (SPLIT == 2) tmem_wait_ld();  // (the second halves of dS go where dP's second chunk is)
      if (exact_delta) {
        // delta_i = sum_j P_ij dP_ij in float32 (key unit: what is missing in dP' = dP - delta)
        if constexpr (KV) {  // over the lanes and the four warps: this CTA holds every key of the plane
          float x[32];
          const bool key = row < un.nrows;  // (the rows past it have a dP' too)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 lo = p[i >> 1], hi = p[16 + (i >> 1)];
            const float a0 = key ? ((i & 1) ? lo.y : lo.x) * __uint_as_float(sv[i]) : 0.f;
            const float a1 = key ? ((i & 1) ? hi.y : hi.x) * __uint_as_float(sv[32 + i]) : 0.f;
            const bool up = (lane & 16) != 0;
            x[i] = (up ? a1 : a0) + __shfl_xor_sync(0xffffffffu, up ? a0 : a1, 16);
          }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < 2 * o; ++i) {
              const bool up = (lane & o) != 0;
              const float keep = up ? x[i + 2 * o] : x[i];
              x[i] = keep + __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 2 * o], o);
            }
          float* red = scratch + (warp & 3) * 128 + half * 64 + 2 * lane;  // lane l ends with columns 2l, 2l + 1
          red[0] = x[0];
          red[1] = x[1];
          all_softmax_warps();
          if (half == 0) {
            const float* c = scratch + row;
            stats[128 + row] = -((c[0] + c[128]) + (c[256] + c[384]));
          }
          all_softmax_warps();
        } else {  // over the row's two halves
          float2 x = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x = fma2(p[e], make_float2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), x);
          stats[256 + half * 128 + row] = x.x + x.y;
          all_softmax_warps();
          nd_row = -(stats[256 + row] + stats[384 + row]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (c == 1) tmem_wait_ld();
        uint32_t hi[16], lo[SPLIT != 0 ? 16 : 1];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = 16 * c + e;
          float2 x = make_float2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1]));
          if constexpr (!KV) x = add2(x, make_float2(nd_row, nd_row));
          else if constexpr (SPLIT == 2)
            if (exact_delta) x = add2(x, *reinterpret_cast<const float2*>(stats + 128 + half * 64 + 2 * k));
          const float2 ds = mul2(p[k], x);
          hi[e] = pack_bf16x2(ds.x, ds.y);
          if (SPLIT > 1 - c) lo[SPLIT != 0 ? e : 0] = pack_bf16x2(ds.x - bf16lo_to_f32(hi[e]), ds.y - bf16hi_to_f32(hi[e]));
        }
        tmem_st16(t_dp + 16 * c, hi);
        if constexpr (SPLIT != 0)
          if (SPLIT > 1 - c) tmem_st16(t_dp + 32 + 16 * c, lo);
        hand_over(&bars->ds_full[c]);
        if constexpr (!KV) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            r_sum = add2(r_sum, make_float2(bf16lo_to_f32(hi[e]), bf16hi_to_f32(hi[e])));
            if (SPLIT > 1 - c) r_sum = add2(r_sum, make_float2(bf16lo_to_f32(lo[SPLIT != 0 ? e : 0]), bf16hi_to_f32(lo[SPLIT != 0 ? e : 0])));
          }
        }
      }
    }
    float r_row = 0.f;
    if constexpr (!KV) {  // both halves' sums of the row
      stats[half * 128 + row] = r_sum.x + r_sum.y;
      all_softmax_warps();
      r_row = stats[row] + stats[128 + row];
    }
    if (ok && T > 0) ok = wait(&bars->o_full, 0);
    if (ok) {
      tc_fence_after();
      // key unit: warps 0-3 write dV, warps 4-7 dK; query unit: each half of the columns of dQ
      const int32_t* perm = KV ? a.perm_k : a.perm_q;
      __nv_bfloat16* out = KV ? (half == 0 ? a.dV : a.dK) : a.dQ;
      const float f = KV && half == 0 ? 1.f : a.scale;
      constexpr int kChunks = KV ? D / 32 : D / 64;  // 32-column chunks per warp
      const int c0 = KV ? 0 : half * kChunks;
      const uint32_t t_o = tmem + lane_off + (KV && half == 0 ? Tm::acc1 : Tm::acc2);
      int tk = -1;
      if (row < un.nrows) {
        tk = perm != nullptr ? __ldg(perm + plane + un.row0 + row) : un.row0 + row;
        SVG2_DEBUG_CHECK(tk >= 0 && tk < a.N, st, kWhereAttnBwdSoftmax, un.row0 + row, tk);
        if (tk < 0 || tk >= a.N) tk = -1;  // an invalid permutation entry is skipped
      }
      uint4* dst = reinterpret_cast<uint4*>(out + (plane + (tk < 0 ? 0 : tk)) * D);
      size_t group = bh;  // whose center: the plane's, or the row's Q cluster's
      if constexpr (!KV && !DENSE) group = static_cast<size_t>(bh) * a.nQ + un.cluster + bars->seg[row];
#pragma unroll 1
      for (int c = c0; c < c0 + kChunks; ++c) {
        uint32_t v[32];
        if (T > 0) {
          tmem_ld32(t_o + c * 32, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if constexpr (!KV) {
          const float4* mean4 = reinterpret_cast<const float4*>(a.center + group * D + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 m = __ldg(mean4 + e);
            v[4 * e + 0] = __float_as_uint(fmaf(-r_row, m.x, __uint_as_float(v[4 * e + 0])));
            v[4 * e + 1] = __float_as_uint(fmaf(-r_row, m.y, __uint_as_float(v[4 * e + 1])));
            v[4 * e + 2] = __float_as_uint(fmaf(-r_row, m.z, __uint_as_float(v[4 * e + 2])));
            v[4 * e + 3] = __float_as_uint(fmaf(-r_row, m.w, __uint_as_float(v[4 * e + 3])));
          }
        }
        if (tk >= 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(v[8 * e + 0]) * f, __uint_as_float(v[8 * e + 1]) * f);
            w.y = pack_bf16x2(__uint_as_float(v[8 * e + 2]) * f, __uint_as_float(v[8 * e + 3]) * f);
            w.z = pack_bf16x2(__uint_as_float(v[8 * e + 4]) * f, __uint_as_float(v[8 * e + 5]) * f);
            w.w = pack_bf16x2(__uint_as_float(v[8 * e + 6]) * f, __uint_as_float(v[8 * e + 7]) * f);
            dst[c * 4 + e] = w;
          }
        }
      }
    }
  }
}

// The ranges of plane rows that a unit's stream is made of (warp 9): the clusters kept by any of the
// unit's, their start rows, the exclusive prefix of their lengths and which of the unit's clusters keep them.
__device__ __forceinline__ void build_ranges(const BwdArgs& a, const BwdUnit un, int bh, bool kv, int32_t* r_start,
                                             int32_t* r_cum, uint16_t* r_seg, BwdBars* bars) {
  const int lane = threadIdx.x & 31;
  const int rows = kv ? a.nK : a.nQ, cols = kv ? a.nQ : a.nK, W = (cols + 31) / 32;
  const uint32_t* bits = (kv ? a.keepers : a.kept) + (static_cast<size_t>(bh) * rows + un.cluster) * W;
  const int32_t* off = (kv ? a.q_off : a.k_off) + static_cast<size_t>(bh) * (cols + 1);
  uint32_t any = 0u;
  if (lane < W)
    for (int s = 0; s < un.nseg; ++s) any |= bits[s * W + lane];
  const int mine = __popc(any);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int cnt = __shfl_sync(0xffffffffu, incl, 31);
  for (int e = incl - mine; any != 0u; ++e, any &= any - 1) r_start[e] = lane * 32 + __ffs(any) - 1;
  __syncwarp();
  int run = 0;
  for (int b = 0; b < cnt; b += 32) {
    int s0 = 0, len = 0;
    if (b + lane < cnt) {
      const int i = r_start[b + lane];
      s0 = off[i];
      len = off[i + 1] - s0;
      if (s0 < 0 || len < 0 || s0 > a.N - len) s0 = len = 0;  // malformed offsets hold no rows
      uint32_t seg = 0u;
      for (int s = 0; s < un.nseg; ++s) seg |= ((bits[s * W + (i >> 5)] >> (i & 31)) & 1u) << s;
      r_seg[b + lane] = static_cast<uint16_t>(seg);
    }
    int sum = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (b + lane < cnt) {
      r_start[b + lane] = s0;
      r_cum[b + lane] = run + sum - len;
    }
    run += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) {
    r_cum[cnt] = run;
    bars->L = run;
  }
}

// Dense attention with long and with short streams, and the sparse plan, are kernels of their own: each holds
// only the unit variants that it can meet, which keeps the hot loops' registers free of spills.
enum class BwdKind { kDense, kDenseMid, kDenseShort, kSparse };

template <int D, BwdKind KIND>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_bwd_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs a) {
  if (__syncthreads_or(status_set(a.st))) return;  // the whole CTA, or none of it
  // key units first (they are the longer ones), then query units
  const int nk = a.BH * a.k_per_head;
  const bool kv = static_cast<int>(blockIdx.x) < nk;
  const int idx = kv ? blockIdx.x : blockIdx.x - nk;
  const int per = kv ? a.k_per_head : a.q_per_head;
  const int bh = idx / per, u = idx % per;
  constexpr bool dense = KIND != BwdKind::kSparse;
  BwdUnit un;
  if (dense) un = BwdUnit{0, u * 128, min(128, a.N - u * 128), 1};
  else un = (kv ? a.k_units : a.q_units)[idx];
  if constexpr (!dense) {  // (malformed offsets can make two runs of the plan write one slot)
    un.nrows = min(un.nrows, a.N - un.row0);
    un.nseg = min(un.nseg, (kv ? a.nK : a.nQ) - un.cluster);
  }
  if (un.nrows <= 0) return;
  const long long wb = effective_wait_budget(a.wait_budget);

  constexpr uint32_t kTile = bwd_tile_bytes<D>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* stats = reinterpret_cast<float*>(smem + (2 + kStreamTiles) * kTile);  // sums over rows' halves, or columns
  int32_t* r_start = reinterpret_cast<int32_t*>(stats + 512);
  int32_t* r_cum = r_start + kBwdMaxRanges;  // kBwdMaxRanges + 1 entries
  uint16_t* r_seg = reinterpret_cast<uint16_t*>(r_cum + kBwdMaxRanges + 16);
  uint8_t* step_s = reinterpret_cast<uint8_t*>(r_seg + kBwdMaxRanges);  // A, then B of S and of dP by stage
  BwdBars* bars = reinterpret_cast<BwdBars*>(step_s + (1 + kStreamTiles) * kStepBytes);
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->res_full), 1);
    // the TMA bytes (or the leader's arrival); when sparse, each producer lane's own copies and, for T1, plain stores
    for (int i = 0; i < kStages1; ++i) {
      mbar_init(smem_u32(&bars->t1_full[i]), dense ? 1 : 193);
      mbar_init(smem_u32(&bars->t1_empty[i]), 1);
    }
    for (int i = 0; i < kStages2; ++i) {
      mbar_init(smem_u32(&bars->t2_full[i]), dense ? 1 : 97);
      mbar_init(smem_u32(&bars->t2_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->p_full[i]), 8);
      mbar_init(smem_u32(&bars->ds_full[i]), 8);
    }
    mbar_init(smem_u32(&bars->dp_full), 1);
    mbar_init(smem_u32(&bars->o_full), 1);
    mbar_init(smem_u32(&bars->mma_done), 1);
    fence_mbar_init();
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (kv || !dense) {  // the step operands: A, and zeros in B
    if (warp < 4) {
      const int row = threadIdx.x;
      int seg = 0;  // this row's cluster among the unit's
      if constexpr (!dense) {
        const int32_t* off = kv ? a.k_off + static_cast<size_t>(bh) * (a.nK + 1) : a.q_off + static_cast<size_t>(bh) * (a.nQ + 1);
        while (seg + 1 < un.nseg && off[un.cluster + seg + 1] <= un.row0 + row) ++seg;
        bars->seg[row] = static_cast<uint8_t>(seg);
      }
      uint32_t w[8] = {0x3f803f80u, 0x3f80u};
#pragma unroll
      for (int k = 0; k < 6; ++k) w[2 + k] = seg == 2 * k ? 0x3f80u : (seg == 2 * k + 1 ? 0x3f800000u : 0u);
      *reinterpret_cast<uint4*>(step_s + row * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(step_s + kStepPlane + row * 16) = make_uint4(w[4], w[5], w[6], w[7]);
    } else if (warp < 8) {
#pragma unroll
      for (int k = 0; k < 2 * kStreamTiles; ++k)
        *reinterpret_cast<uint4*>(step_s + kStepBytes + (k * 128 + threadIdx.x - 128) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == kBwdProducerWarp) {
    if (!dense) build_ranges(a, un, bh, kv, r_start, r_cum, r_seg, bars);
    else if ((threadIdx.x & 31) == 0) bars->L = a.N;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwdOtherRegs) : "memory");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwdSoftmaxRegs) : "memory");
  float* scratch = reinterpret_cast<float*>(r_start);
#define SVG2_BWD_UNIT(KV, SPLIT, MULTI) \
  bwd_unit<D, dense, KV, SPLIT, MULTI>(maps, a, un, bh, smem, bars, stats, r_start, r_cum, r_seg, step_s, scratch, wb)
  if constexpr (dense) {
    constexpr int kSplitQ = KIND == BwdKind::kDenseShort ? 2 : (KIND == BwdKind::kDenseMid ? 1 : 0);
    if (kv) SVG2_BWD_UNIT(true, KIND == BwdKind::kDenseShort ? 2 : 0, false);
    else SVG2_BWD_UNIT(false, kSplitQ, false);
  } else {
    const bool split = bars->L <= kBwdSplitTiles * 128, multi = un.nseg > 1;
    if (kv) {
      if (split) SVG2_BWD_UNIT(true, 2, true);  // (with one cluster its mask drops nothing)
      else if (multi) SVG2_BWD_UNIT(true, 0, true);
      else SVG2_BWD_UNIT(true, 0, false);
    } else {
      if (split) SVG2_BWD_UNIT(false, 2, true);
      else if (bars->L <= kBwdHalfSplitTiles * 128) SVG2_BWD_UNIT(false, 1, true);
      else if (multi) SVG2_BWD_UNIT(false, 0, true);
      else SVG2_BWD_UNIT(false, 0, false);
    }
  }
#undef SVG2_BWD_UNIT
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdMmaWarp) {
    tc_fence_after();
    tmem_dealloc(bars->tmem_base, 512);
  }
}

template <int D>
cudaError_t launch_bwd(const BwdInputs& in, int BH, int N, int nQ, int nK, float scale, const BwdScratch& sc,
                       DeviceStatus* st, const uint64_t* wait_budget, cudaStream_t s) {
  const bool dense = in.sel_idx == nullptr;
  const long long rows = static_cast<long long>(BH) * N;
  constexpr int kRows = 256 / (D / 8);  // rows per CTA pass
  const unsigned grid = static_cast<unsigned>(rows / kRows + 1 < 148 * 16 ? rows / kRows + 1 : 148 * 16);
  const bool wide = dense || N >= kMeanWide * nK;
  bwd_prep_kernel<D><<<grid + mean_ctas_of(BH, dense ? 1 : nK, wide), 256, 0, s>>>(static_cast<const uint4*>(in.O), static_cast<const uint4*>(in.dO),
                                               in.lse, in.perm_q, static_cast<const uint4*>(in.K), N, rows,
                                               BH, sc.neg_lse2, sc.neg_delta,
                                               sc.lse_step, sc.delta_step, 1.f / scale,
                                               in.perm_q != nullptr ? static_cast<uint4*>(sc.dOp) : nullptr,
                                               dense ? nullptr : in.k_off, nK, wide, dense ? sc.center : sc.cluster_mean, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  BwdArgs a{};
  a.BH = BH;
  a.N = N;
  a.nQ = nQ;
  a.nK = nK;
  a.k_per_head = dense ? (N + 127) / 128 : bwd_max_units_per_head(N, nK);
  a.q_per_head = dense ? (N + 127) / 128 : bwd_max_units_per_head(N, nQ);
  if (!dense) {
    const size_t k_bytes = static_cast<size_t>(nK) * ((nQ + 31) / 32) * 4, row = static_cast<size_t>((nK + 31) / 32) * 4;
    const bool fits = k_bytes + nQ * row <= kPlanSmem;
    e = cudaFuncSetAttribute(bwd_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPlanSmem));
    if (e != cudaSuccess) return e;
    const size_t bits_smem = k_bytes + (fits ? nQ : kPlanWarps) * row;
    const bool beside = bits_smem <= kPlanBesideSmem;
    const size_t plan_smem = beside ? std::max(bits_smem, kPlanWarps * D * sizeof(MeanSums)) : bits_smem;
    const int clusters = BH * nQ;
    constexpr int kPerCta = kPlanWarps / kCenterWarps;
    if (!beside) {
      bwd_center_kernel<<<static_cast<unsigned>((clusters + 7) / 8), 256, 0, s>>>(in.k_off, in.sel_count, in.sel_idx, N, nQ, nK, D,
                                                                              clusters, sc.cluster_mean, sc.center);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    bwd_plan_kernel<<<static_cast<unsigned>(BH + (beside ? (clusters + kPerCta - 1) / kPerCta : 0)), kPlanThreads, plan_smem, s>>>(
        in.q_off, in.k_off, in.sel_count, in.sel_idx, N, nQ, nK, sc.keepers, sc.kept, fits, sc.k_units, a.k_per_head,
        sc.q_units, a.q_per_head, BH, D, sc.cluster_mean, sc.center, st);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  a.q_off = in.q_off;
  a.k_off = in.k_off;
  a.keepers = sc.keepers;
  a.kept = sc.kept;
  a.k_units = sc.k_units;
  a.q_units = sc.q_units;
  a.perm_q = in.perm_q;
  a.perm_k = in.perm_k;
  a.neg_lse2 = sc.neg_lse2;
  a.neg_delta = sc.neg_delta;
  a.center = sc.center;
  a.lse_step = sc.lse_step;
  a.delta_step = sc.delta_step;
  a.dQ = static_cast<__nv_bfloat16*>(in.dQ);
  a.dK = static_cast<__nv_bfloat16*>(in.dK);
  a.dV = static_cast<__nv_bfloat16*>(in.dV);
  a.scale = scale;
  a.st = st;
  a.wait_budget = wait_budget;
  alignas(64) BwdMaps maps;
  const void* base[4] = {in.Q, in.K, in.V, in.perm_q != nullptr ? sc.dOp : in.dO};
  for (int t = 0; t < 4 && e == cudaSuccess; ++t)
    e = make_tmap_bf16_3d(&maps.m[t], base[t], D, N, BH, D * 2, static_cast<uint64_t>(N) * D * 2, 128);
  a.Q = static_cast<const __nv_bfloat16*>(base[0]);
  a.K = static_cast<const __nv_bfloat16*>(base[1]);
  a.V = static_cast<const __nv_bfloat16*>(base[2]);
  a.dO = static_cast<const __nv_bfloat16*>(base[3]);
  if (e != cudaSuccess) return e;
  auto* kernel = !dense ? attn_bwd_kernel<D, BwdKind::kSparse>
                 : N <= kBwdSplitTiles * 128  ? attn_bwd_kernel<D, BwdKind::kDenseShort>
                 : N <= kBwdHalfSplitTiles * 128 ? attn_bwd_kernel<D, BwdKind::kDenseMid>
                                              : attn_bwd_kernel<D, BwdKind::kDense>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bwd_smem<D>());
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(BH) * (a.k_per_head + a.q_per_head);
  kernel<<<static_cast<unsigned>(units), kBwdThreads, bwd_smem<D>(), s>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd(const BwdInputs& in, int BH, int N, int d, int nQ, int nK, float scale,
                            const BwdScratch& sc, DeviceStatus* st, const uint64_t* wait_budget, cudaStream_t s) {
  return d == 128 ? launch_bwd<128>(in, BH, N, nQ, nK, scale, sc, st, wait_budget, s)
                  : launch_bwd<64>(in, BH, N, nQ, nK, scale, sc, st, wait_budget, s);
}

}  // namespace svg2
