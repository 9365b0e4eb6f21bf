// Layer norm over rows, forward and backward (include/bmoe_norm.h).
//
// Both passes are bound by HBM: a few operations per element read once and
// written once.  A row is held in registers between its loads and its stores:
// TPR threads (one wave up to 2048 columns in groups of 8, else a whole workgroup)
// hold NV groups of consecutive elements each, group v of thread t being group t +
// TPR v of the row, so every load is contiguous over the wave.  One wave per row
// needs no LDS and no barrier.  Workgroups loop over rows, which keeps gamma, beta
// and the backward's column sums of the thread's columns in registers.
#include "step_ops.hpp"

#include <type_traits>

namespace bmoe {

// Sum over a wave's 64 lanes, the same value in every lane (fixed order).
__device__ __forceinline__ float ln_wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Sums of N values over the TPR threads of a row, the same in each of them: over
// each wave, then every wave adds the waves' sums.  Two sets of those in turn, so one
// barrier a sum is enough: who writes a set again is past the barrier of the sum
// between, which every wave reaches only after its reads of the set.
template <int TPR>
struct LnRed {
  float2 sums[2][TPR > 64 ? TPR / 64 : 1];
};
template <int TPR, int N>
__device__ __forceinline__ void ln_row_sum(float (&v)[N], LnRed<TPR>& red, int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = ln_wave_sum(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float2* r = red.sums[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = make_float2(v[0], v[N - 1]);
    __syncthreads();
    const float2 u = r[threadIdx.x % W];
    v[0] = u.x;
    if constexpr (N == 2) v[1] = u.y;
#pragma unroll
    for (int m = 1; m < W; m <<= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], m);
  }
}

// How a row is cut into groups of consecutive elements: 8 at 16-byte alignment in a
// width that they divide (LN_WHOLE), 8 at any alignment with the last group's
// elements one by one (LN_ANY), 2 (LN_PAIR) or 1 (LN_SINGLE).
enum LnCut { LN_WHOLE, LN_ANY, LN_PAIR, LN_SINGLE };
constexpr int ln_elems(int cut) { return cut <= LN_ANY ? 8 : cut == LN_PAIR ? 2 : 1; }

// The group from element i on, n elements (or more) before the row's end.
template <int ACT, int CUT>
__device__ __forceinline__ void ln_load(const void* p, size_t i, int n, float* v) {
  typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
  typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
  if constexpr (CUT == LN_WHOLE) {
    load8<ACT>(p, i, v);
  } else if constexpr (CUT == LN_PAIR && ACT == ACT_BF16) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i);
    v[0] = bf16lo(u);
    v[1] = bf16hi(u);
  } else if constexpr (CUT == LN_PAIR) {
    const float2 u = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
    v[0] = u.x;
    v[1] = u.y;
  } else if constexpr (CUT == LN_SINGLE) {
    v[0] = load1<ACT>(p, i);
  } else if (n < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? load1<ACT>(p, i + j) : 0.f;
  } else if constexpr (ACT == ACT_BF16) {
    const u32x4_any_t u = *reinterpret_cast<const u32x4_any_t*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16lo(u[k]);
      v[2 * k + 1] = bf16hi(u[k]);
    }
  } else {
    const f32x4_any_t* q = reinterpret_cast<const f32x4_any_t*>(static_cast<const float*>(p) + i);
    const f32x4_any_t lo = q[0], hi = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = lo[k];
      v[4 + k] = hi[k];
    }
  }
}

template <int ACT, int CUT>
__device__ __forceinline__ void ln_store(void* p, size_t i, int n, const float* v) {
  // results go past L2, which the rows to come need (streamed stores: 122 ->
  // 119 us at 32768 x 2048 bf16, 12.9 -> 11.7 us at 8192 x 1024; streamed loads
  // lose where the producer left its rows in the last-level cache: 15.7 us).  With a
  // pass behind that reads y, streamed and plain stores: 161 and 165 us at 32768 x
  // 2048, 19.3 and 18.1 at 8192 x 1024.  Groups that share lines are stored plainly.
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
  typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));
  if constexpr (CUT == LN_PAIR && ACT == ACT_BF16) {
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + i) = pack_bf16x2(v[0], v[1]);
  } else if constexpr (CUT == LN_PAIR) {
    *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = make_float2(v[0], v[1]);
  } else if constexpr (CUT == LN_SINGLE && ACT == ACT_BF16) {
    static_cast<uint16_t*>(p)[i] = uint16_t(pack_bf16x2(v[0], v[0]));
  } else if constexpr (CUT == LN_SINGLE) {
    static_cast<float*>(p)[i] = v[0];
  } else if (CUT == LN_ANY && n < 8) {
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      if (j >= n) continue;
      if constexpr (ACT == ACT_BF16) static_cast<uint16_t*>(p)[i + j] = uint16_t(pack_bf16x2(v[j], v[j]));
      else static_cast<float*>(p)[i + j] = v[j];
    }
  } else if constexpr (ACT == ACT_BF16) {
    const u32x4_t u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (CUT == LN_WHOLE) __builtin_nontemporal_store(u, reinterpret_cast<u32x4_t*>(q));
    else *reinterpret_cast<u32x4_any_t*>(q) = u;
  } else {
    const f32x4_t lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    float* q = static_cast<float*>(p) + i;
    if constexpr (CUT == LN_WHOLE) {
      __builtin_nontemporal_store(lo, reinterpret_cast<f32x4_t*>(q));
      __builtin_nontemporal_store(hi, reinterpret_cast<f32x4_t*>(q) + 1);
    } else {
      reinterpret_cast<f32x4_any_t*>(q)[0] = lo;
      reinterpret_cast<f32x4_any_t*>(q)[1] = hi;
    }
  }
}

// The values as the activation dtype stores them.
template <int ACT, int E>
__device__ __forceinline__ void ln_round(float* v) {
  if constexpr (ACT == ACT_BF16) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = float(__bf16(v[j]));
  }
}

// Waves per SIMD that the kernels' registers leave room for: the row itself, and
// per column gamma and beta (forward) or gamma and two sums (backward).  A grid of
// exactly the workgroups that run at a time loses no partial last round: 32768 x
// 2048 forward 111 us with 3 per CU (as many as fit), 146 with 4, 122 with 8 and
// 125 with one per 4 rows.
constexpr int ln_fwd_waves(int e, int nv) { return e * nv >= 32 ? 3 : e * nv >= 16 ? (e == 8 ? 5 : 4) : 8; }
constexpr int ln_threads(int tpr) { return tpr > 256 ? tpr : 256; }

template <int ACT, int CUT, int TPR, int NV>
__global__ __launch_bounds__(ln_threads(TPR), TPR > 512 ? 4 : ln_fwd_waves(ln_elems(CUT), NV)) void ln_fwd_kernel(LnFwdArgs a) {
#pragma clang fp contract(off)  // what a row is centred by is the mean as rounded
  constexpr int E = ln_elems(CUT), RPW = TPR > 256 ? 1 : 256 / TPR;  // rows per workgroup
  __shared__ LnRed<TPR> red;
  int turn = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int groups = (a.width + E - 1) / E;
  const float inv = 1.0f / float(a.width);
  float ga[NV][E], be[NV][E];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int g = t + TPR * v;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      ga[v][j] = 1.f;
      be[v][j] = 0.f;
    }
    if (g < groups && a.gamma) ln_load<ACT_F32, CUT>(a.gamma, size_t(g) * E, a.width - E * g, ga[v]);
    if (g < groups && a.beta) ln_load<ACT_F32, CUT>(a.beta, size_t(g) * E, a.width - E * g, be[v]);
  }
  for (int row = blockIdx.x * RPW + sub; row < a.rows; row += gridDim.x * RPW) {
    const size_t at = size_t(row) * a.width;
    float x[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v;
#pragma unroll
      for (int j = 0; j < E; ++j) x[v][j] = 0.f;
      if (g < groups) ln_load<ACT, CUT>(a.x, at + size_t(g) * E, a.width - E * g, x[v]);
    }
    if (a.res) {
      float r[NV][E];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int g = t + TPR * v;
#pragma unroll
        for (int j = 0; j < E; ++j) r[v][j] = 0.f;
        if (g < groups) ln_load<ACT, CUT>(a.res, at + size_t(g) * E, a.width - E * g, r[v]);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int g = t + TPR * v;
#pragma unroll
        for (int j = 0; j < E; ++j) x[v][j] += r[v][j];
        ln_round<ACT, E>(x[v]);
        if (g < groups) ln_store<ACT, CUT>(a.sum, at + size_t(g) * E, a.width - E * g, x[v]);
      }
    }
    float s[1] = {0.f};  // in parts of the mean, which no finite row's sum of leaves fp32
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) s[0] = fmaf(x[v][j], inv, s[0]);
    ln_row_sum<TPR>(s, red, turn);
    float mean = s[0], before = 0.f, d = 0.f, var = 0.f, unit = 1.f;
    // x -= by, the sum of its squares and, in `whole` passes, its own mean
    auto centre = [&](float by, auto whole) {
      constexpr bool W = decltype(whole)::value;
      float q[W ? 2 : 1] = {};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int in = a.width - E * (t + TPR * v);  // past the row everything stays 0
#pragma unroll
        for (int j = 0; j < E; ++j) {
          x[v][j] -= (CUT == LN_ANY ? j < in : in > 0) ? by : 0.f;
          if constexpr (W) q[1] = fmaf(x[v][j], inv, q[1]);
          q[0] = fmaf(x[v][j], x[v][j], q[0]);
        }
      }
      ln_row_sum<TPR>(q, red, turn);
      var = q[0] * inv;
      if constexpr (W) d = q[1];
    };
    centre(mean, std::false_type{});
    // The mean as summed is off by that sum's roundings: by as much as a row far
    // from 0 varies, or by all that a constant row does.  A row further from 0 than
    // it varies takes what is missing, d, from its centred values' own mean, and is
    // centred once more where that is not small against what it varies by.  One whose
    // squares leave fp32 (deviations of 1e19 / sqrt(width) and more) goes on times
    // 2^-80, one whose squares vanish in it, with an eps that does not cover them,
    // times 2^96.  (8192 x 4096 bf16: 23.3 us, 26.0 for rows 5 deviations from 0; with d in
    // every row in place of this branch 24.6; cached inputs.)
    const bool large = !(var < __builtin_inff()), small = var + a.eps < 0x1p-100f;
    if (large || small || !(mean * mean <= var)) {
      if (large || small) {
        unit = large ? 0x1p-80f : 0x1p96f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < E; ++j) x[v][j] *= unit;
      }
      centre(0.f, std::true_type{});
      if (!(d * d <= 0x1p-12f * var)) {
        before = d;
        centre(d, std::true_type{});
      }
    }
    mean += (before + d) * (unit == 1.f ? 1.f : unit < 1.f ? 0x1p80f : 0x1p-96f);
    var = fmaf(-d, d, var);
    const float rstd = 1.0f / sqrtf((var < 0.f ? 0.f : var) + a.eps * unit * unit);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v;
      float y[E];
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = fmaf((x[v][j] - d) * rstd, ga[v][j], be[v][j]);
      if (g < groups) ln_store<ACT, CUT>(a.y, at + size_t(g) * E, a.width - E * g, y);
    }
    if (t == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd * unit;
    }
  }
}

// dgamma and dbeta of 16 columns over all rows, by one workgroup of NT threads:
// NT / 16 groups of lanes that take the rows g, g + NT / 16, ... each, their sums
// added in order.  8 columns read more lines twice (512 x 4096 fp32 15.9 us in
// place of 11.4, 333 x 1000 4.2 of 4.5).
constexpr int LN_COLS = 16;
template <int ACT, int DACT, int NT>
__device__ __forceinline__ void ln_columns(const LnBwdArgs& a, int block) {
  constexpr int G = NT / LN_COLS;
  __shared__ float2 sm[G][LN_COLS + 1];
  const int col = threadIdx.x % LN_COLS, grp = threadIdx.x / LN_COLS, c = block * LN_COLS + col;
  float dg = 0.f, db = 0.f;
  if (c < a.width) {
#pragma unroll 8
    for (int r = grp; r < a.rows; r += G) {
      const size_t at = size_t(r) * a.width + c;
      const float dy = load1<DACT>(a.dy, at);
      dg = fmaf(dy, (load1<ACT>(a.s, at) - a.mean[r]) * a.rstd[r], dg);
      db += dy;
    }
  }
  sm[grp][col] = make_float2(dg, db);
  __syncthreads();
  if (grp == 0 && c < a.width) {
    dg = db = 0.f;
#pragma unroll
    for (int w = 0; w < G; ++w) {
      dg += sm[w][col].x;
      db += sm[w][col].y;
    }
    a.dgamma[c] = dg;
    a.dbeta[c] = db;
  }
}

// Backward.  With SUMS each thread keeps its columns' sums of dy xhat and dy over
// the rows of its workgroup; at the end the workgroup adds its waves' sums in
// order (through LDS) and writes one partial row [dgamma | dbeta].  Without, the
// workgroups behind a.row_blocks, if any, take the columns' sums from the inputs
// again.
template <int ACT, int DACT, int CUT, int TPR, int NV, bool SUMS>
__global__ __launch_bounds__(ln_threads(TPR)) void ln_bwd_kernel(LnBwdArgs a) {
  constexpr int E = ln_elems(CUT), RPW = TPR > 256 ? 1 : 256 / TPR;
  if constexpr (!SUMS) {
    if (int(blockIdx.x) >= a.row_blocks) {
      ln_columns<ACT, DACT, ln_threads(TPR)>(a, int(blockIdx.x) - a.row_blocks);
      return;
    }
  }
  __shared__ LnRed<TPR> red;
  int turn = 0;
  __shared__ float cols[SUMS && RPW > 1 ? RPW : 1][SUMS && RPW > 1 ? TPR * NV * E : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int groups = (a.width + E - 1) / E;
  const float inv = 1.0f / float(a.width);
  float ga[NV][E], dg[NV][E], db[NV][E];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int g = t + TPR * v;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      ga[v][j] = 1.f;
      dg[v][j] = db[v][j] = 0.f;
    }
    if (g < groups && a.gamma) ln_load<ACT_F32, CUT>(a.gamma, size_t(g) * E, a.width - E * g, ga[v]);
  }
  for (int row = blockIdx.x * RPW + sub; row < a.rows; row += a.row_blocks * RPW) {
    const size_t at = size_t(row) * a.width;
    float x[NV][E], d[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v;
#pragma unroll
      for (int j = 0; j < E; ++j) x[v][j] = d[v][j] = 0.f;
      if (g < groups) {
        ln_load<ACT, CUT>(a.s, at + size_t(g) * E, a.width - E * g, x[v]);
        ln_load<DACT, CUT>(a.dy, at + size_t(g) * E, a.width - E * g, d[v]);
      }
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c[2] = {0.f, 0.f};  // sums of v and v xhat
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      // past the row dy is zero and xhat is made zero, so that
      // an infinite rstd or mean reaches no other column
      const int in = a.width - E * (t + TPR * v);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[v][j] = (CUT == LN_ANY ? j < in : in > 0) ? (x[v][j] - mean) * rstd : 0.f;
        const float dy = d[v][j];
        if constexpr (SUMS) {
          dg[v][j] = fmaf(dy, x[v][j], dg[v][j]);
          db[v][j] += dy;
        }
        d[v][j] = dy * ga[v][j];
        c[0] += d[v][j];
        c[1] = fmaf(d[v][j], x[v][j], c[1]);
      }
    }
    ln_row_sum<TPR>(c, red, turn);
    const float c1 = c[0] * inv, c2 = c[1] * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v;
      if (g < groups) {
        float o[E];
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = rstd * (d[v][j] - c1 - x[v][j] * c2);
        if (a.d_sum) {
          float r[E];
          ln_load<ACT, CUT>(a.d_sum, at + size_t(g) * E, a.width - E * g, r);
#pragma unroll
          for (int j = 0; j < E; ++j) o[j] += r[j];
        }
        ln_store<ACT, CUT>(a.dx, at + size_t(g) * E, a.width - E * g, o);
      }
    }
  }
  if constexpr (SUMS) {
    float* out = a.part + size_t(blockIdx.x) * 2 * a.width;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (RPW == 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int g = t + TPR * v;
          if (g < groups)
#pragma unroll
            for (int j = 0; j < E; ++j)
              if (CUT != LN_ANY || E * g + j < a.width) out[size_t(k) * a.width + size_t(g) * E + j] = k ? db[v][j] : dg[v][j];
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < E; ++j) cols[sub][(t + TPR * v) * E + j] = k ? db[v][j] : dg[v][j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += 256) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < RPW; ++w) s += cols[w][c];
          out[size_t(k) * a.width + c] = s;
        }
      }
    }
  }
}

// Column sums of the P partial rows: 16 columns per workgroup, 64 groups of
// lanes that take the rows p, p + 64, ... each, their sums added in order (8 rows
// per thread at 512 partial rows, all loads in flight at once).
__global__ __launch_bounds__(1024) void ln_colsum_kernel(const float* part, float* dgamma, float* dbeta, int P,
                                                         int width) {
  __shared__ float sm[64][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col, n = 2 * width;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int p = grp; p < P; p += 64) s += part[size_t(p) * n + c];
  }
  sm[grp][col] = s;
  __syncthreads();
  if (threadIdx.x < 128) {  // eight sums of eight groups, then those
    const int k = threadIdx.x >> 4;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sm[8 * k + w][col];
    sm[8 * k][col] = s;
  }
  __syncthreads();
  if (threadIdx.x < 16 && c < n) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sm[8 * w][col];
    if (c < width) dgamma[c] = s;
    else dbeta[c - width] = s;
  }
}

namespace {

bool ln_aligned(const void* p, size_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

// Threads per row and groups per thread for a row of `groups` groups.
struct LnShape {
  int tpr, nv;
};
LnShape ln_shape(int cut, int groups) {
  if (cut <= LN_ANY) {
    if (groups <= 64) return {64, 1};
    if (groups <= 128) return {64, 2};
    if (groups <= 256) return {64, 4};
    if (groups <= 512) return {256, 2};
    if (groups <= 1024) return {512, 2};
    return {1024, 2};
  }
  if (cut == LN_PAIR) {
    if (groups <= 128) return {64, 2};
    if (groups <= 512) return {64, 8};
    if (groups <= 2048) return {256, 8};
    return {1024, 8};
  }
  return groups <= 256 ? LnShape{64, 4} : LnShape{64, 16};  // 512 at most
}

// whole, pair: what alignment and width allow.  Wide rows of any alignment take 16
// bytes at a time (forward and gradient in us, so and by pairs or singles: 8220 x 1443
// bf16 25 and 41, 55 and 81; 16384 x 2047 bf16 71 and 121, 172 and 264; 5000 x 4099
// fp32 72 and 100, 77 and 168), narrow ones lose by the last group's single accesses
// (20000 x 255 bf16 19 and 49, 15 and 35), as do fp32's pairs in the forward (4096 x
// 2046 26 and 22) and above 4096 in the gradient (3000 x 8190 118 and 110).
int ln_cut(int width, bool whole, bool pair, bool keep_pairs) {
  if (whole) return LN_WHOLE;
  if (pair && (width <= 512 || keep_pairs)) return LN_PAIR;
  return width > 512 ? LN_ANY : pair ? LN_PAIR : LN_SINGLE;
}

constexpr int LN_CUS = 256;  // of a whole MI355X

template <int ACT, int CUT, int TPR, int NV>
hipError_t fwd_go(const LnFwdArgs& a, hipStream_t s) {
  constexpr int RPW = TPR > 256 ? 1 : 256 / TPR, waves = TPR > 512 ? 4 : ln_fwd_waves(ln_elems(CUT), NV);
  constexpr int most = LN_CUS * (waves * 256 / ln_threads(TPR));
  const int blocks = (a.rows + RPW - 1) / RPW;
  hipLaunchKernelGGL((ln_fwd_kernel<ACT, CUT, TPR, NV>), dim3(unsigned(blocks < most ? blocks : most)),
                     dim3(ln_threads(TPR)), 0, s, a);
  return hipGetLastError();
}

template <int ACT, int DACT, int CUT, int TPR, int NV>
hipError_t bwd_go(LnBwdArgs a, hipStream_t s) {
  const dim3 threads(ln_threads(TPR));
  if (a.part) {
    hipLaunchKernelGGL((ln_bwd_kernel<ACT, DACT, CUT, TPR, NV, true>), dim3(unsigned(a.row_blocks)), threads, 0, s, a);
    return hipGetLastError();
  }
  int columns = a.dgamma ? (a.width + LN_COLS - 1) / LN_COLS : 0;
  if (columns && (a.dx == a.s || a.dx == a.dy)) {  // in place: the columns first
    const int rows = a.row_blocks;
    a.row_blocks = 0;
    hipLaunchKernelGGL((ln_bwd_kernel<ACT, DACT, CUT, TPR, NV, false>), dim3(unsigned(columns)), threads, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.row_blocks = rows;
    columns = 0;
  }
  const int grid = a.row_blocks + columns;
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL((ln_bwd_kernel<ACT, DACT, CUT, TPR, NV, false>), dim3(unsigned(grid)), threads, 0, s, a);
  return hipGetLastError();
}

#define LN_SHAPES_8(GO, CUT)                 \
  if (sh.tpr == 1024) return GO(CUT, 1024, 2); \
  if (sh.tpr == 512) return GO(CUT, 512, 2);   \
  if (sh.tpr == 256) return GO(CUT, 256, 2);   \
  if (sh.nv == 4) return GO(CUT, 64, 4);       \
  if (sh.nv == 2) return GO(CUT, 64, 2);       \
  return GO(CUT, 64, 1);

#define LN_SHAPES(GO)                                                       \
  const int e = ln_elems(cut);                                              \
  const LnShape sh = ln_shape(cut, (a.width + e - 1) / e);                  \
  if (cut == LN_WHOLE) { LN_SHAPES_8(GO, LN_WHOLE) }                        \
  if (cut == LN_ANY) { LN_SHAPES_8(GO, LN_ANY) }                            \
  if (cut == LN_PAIR) {                                                     \
    if (sh.tpr == 1024) return GO(LN_PAIR, 1024, 8);                        \
    if (sh.tpr == 256) return GO(LN_PAIR, 256, 8);                          \
    return sh.nv == 8 ? GO(LN_PAIR, 64, 8) : GO(LN_PAIR, 64, 2);            \
  }                                                                         \
  return sh.nv == 16 ? GO(LN_SINGLE, 64, 16) : GO(LN_SINGLE, 64, 4);

template <int ACT>
hipError_t fwd_act(const LnFwdArgs& a, int cut, hipStream_t s) {
#define LN_GO(C, T, V) fwd_go<ACT, C, T, V>(a, s)
  LN_SHAPES(LN_GO)
#undef LN_GO
}

template <int ACT, int DACT>
hipError_t bwd_act(const LnBwdArgs& a, int cut, hipStream_t s) {
#define LN_GO(C, T, V) bwd_go<ACT, DACT, C, T, V>(a, s)
  LN_SHAPES(LN_GO)
#undef LN_GO
}

}  // namespace

// Rows' workgroups of the backward: what runs at a time with the sums of a whole row
// of 2048 in registers, two per CU (32768 x 2048 136 us with 512, 163 with 768, 143 with
// 1024; narrower rows' registers leave room for more, which would have to pay for their
// partial rows), no more than there are groups of 4 rows.
static int ln_bwd_blocks(int rows) {
  const int need = (rows + 3) / 4;
  return need < 512 ? need : 512;
}

// Whether one launch takes the columns' sums too, from inputs read twice, in place
// of partial rows and a second launch.  Long columns and inputs beyond the L2s lose
// (us on the GPU, one launch and two, fp32: 333 x 1000 4.5 and 6.3, 1024 x 512 6.9
// and 6.8, 512 x 4096 11.4 and 14.8, 1024 x 2048 10.7 and 13.2; 1024 x 4096 19.1 and
// 17.7, 2048 x 512 12.4 and 8.1; the host needs 9.5 and 12.5 a call).
static bool ln_bwd_once(int rows, int width) { return rows <= 1024 && size_t(rows) * width <= size_t(1) << 21; }

size_t ln_bwd_workspace(int rows, int width) { return ln_bwd_once(rows, width) ? 0 : size_t(ln_bwd_blocks(rows)) * 2 * width * 4; }

hipError_t launch_ln_fwd(const LnFwdArgs& a, int act, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const size_t two = act == ACT_BF16 ? 4 : 8;
  auto all = [&](size_t b, size_t f) {
    return ln_aligned(a.x, b) && ln_aligned(a.res, b) && ln_aligned(a.sum, b) && ln_aligned(a.y, b) &&
           ln_aligned(a.gamma, f) && ln_aligned(a.beta, f);
  };
  const int cut = ln_cut(a.width, a.width % 8 == 0 && all(16, 16), a.width % 2 == 0 && all(two, 8), act == ACT_F32);
  return act == ACT_BF16 ? fwd_act<ACT_BF16>(a, cut, s) : fwd_act<ACT_F32>(a, cut, s);
}

hipError_t launch_ln_bwd(LnBwdArgs a, int act, int dact, hipStream_t s) {
  const size_t two = act == ACT_BF16 ? 4 : 8, dtwo = dact == ACT_BF16 ? 4 : 8;
  auto all = [&](size_t b, size_t d, size_t f) {
    return ln_aligned(a.s, b) && ln_aligned(a.d_sum, b) && ln_aligned(a.dx, b) && ln_aligned(a.dy, d) &&
           ln_aligned(a.gamma, f);
  };
  const int cut = ln_cut(a.width, a.width % 8 == 0 && all(16, 16, 16), a.width % 2 == 0 && all(two, dtwo, 8), a.width > 4096);
  a.row_blocks = ln_bwd_blocks(a.rows);
  if (!a.dgamma || ln_bwd_once(a.rows, a.width)) a.part = nullptr;
  const hipError_t e = act == ACT_BF16
                           ? (dact == ACT_BF16 ? bwd_act<ACT_BF16, ACT_BF16>(a, cut, s) : bwd_act<ACT_BF16, ACT_F32>(a, cut, s))
                           : bwd_act<ACT_F32, ACT_F32>(a, cut, s);
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(ln_colsum_kernel, dim3(unsigned((2 * a.width + 15) / 16)), dim3(1024), 0, s, a.part, a.dgamma,
                     a.dbeta, a.row_blocks, a.width);
  return hipGetLastError();
}

}  // namespace bmoe
