// Rows in registers: what the norms' kernels (layer_norm.hip, block_norm.hip) share.
//
// TPR threads hold a row, NV groups of consecutive elements each, group v of thread t
// being group t + TPR v of the row, so every load is contiguous over the wave.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace bmoe {

// Sum over the LANES lanes of a wave that share a row, the same value in each of them
// (the tree of exchanges with the lanes 1, 2, 4, .. away, within the register file).
template <int CTRL>
__device__ __forceinline__ float ln_dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int LANES>
__device__ __forceinline__ float ln_wave_sum(float v) {
  static_assert(LANES == 16 || LANES == 32 || LANES == 64, "rows of lanes");
  v = ln_dpp_add<0xB1>(v);    // quad_perm 1 0 3 2
  v = ln_dpp_add<0x4E>(v);    // quad_perm 2 3 0 1
  v = ln_dpp_add<0x141>(v);   // row_half_mirror: the other four of eight
  v = ln_dpp_add<0x140>(v);   // row_mirror: the other eight of sixteen
  if constexpr (LANES >= 32) {
    const auto u = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(u[0]) + __uint_as_float(u[1]);
  }
  if constexpr (LANES == 64) {
    const auto u = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(u[0]) + __uint_as_float(u[1]);
  }
  return v;
}

// Sums of N values over the TPR threads of a row, the same in each of them: over
// each wave, then every wave adds the waves' sums (TPR a power of two).  Two sets of those in turn, so one
// barrier a sum is enough: who writes a set again is past the barrier of the sum
// between, which every wave reaches only after its reads of the set.
template <int TPR>
struct LnRed {
  float2 sums[2][TPR > 64 ? TPR / 64 : 1];
};
template <int TPR, int N>
__device__ __forceinline__ void ln_row_sum(float (&v)[N], LnRed<TPR>& red, int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = ln_wave_sum<(TPR < 64 ? TPR : 64)>(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float2* r = red.sums[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x % TPR / 64] = make_float2(v[0], v[N - 1]);
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

// The mean of a row, which is centred by it in place, and 1 / its deviation: with x the
// row on return, its normed values are (x - off) rstd, its 1 / deviation is rstd unit.
struct LnStats {
  float mean, off, rstd, unit;
};
// on(v, j): whether x[v][j] is the row's; what is not is 0 and stays it.
template <int TPR, int NV, int E, typename On>
__device__ __forceinline__ LnStats ln_centre(float (&x)[NV][E], int width, float eps, LnRed<TPR>& red, int& turn, On&& on) {
#pragma clang fp contract(off)  // what a row is centred by is the mean as rounded
  const float inv = 1.0f / float(width);
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
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[v][j] -= on(v, j) ? by : 0.f;
        if constexpr (W) q[1] = fmaf(x[v][j], inv, q[1]);
        q[0] = fmaf(x[v][j], x[v][j], q[0]);
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
  const bool large = !(var < __builtin_inff()), small = var + eps < 0x1p-100f;
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
  return {mean, d, 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps * unit * unit), unit};
}

}  // namespace bmoe
