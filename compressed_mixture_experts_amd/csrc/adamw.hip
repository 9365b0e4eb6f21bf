// AdamW step over many tensors (include/bmoe_adamw.h).
//
// Bound by HBM: 28 bytes a value with fp32 moments and gradients, 16 with moments in 8
// bits, some 15 operations for the step and 60 for the codes.  One launch takes up to
// AW_TENSORS tensors, whose description travels in the kernel's arguments: no table in
// memory, so nothing is copied before the launch and a captured step holds all of it.  A
// workgroup takes a run of one tensor's values, 1024 at a time, four consecutive ones
// per thread, so that a wave's 256 values are one block of the 8-bit form: its largest
// value needs no LDS and no barrier.
#include "step_ops.hpp"

#include <algorithm>

namespace bmoe {

constexpr int AW_M_TOP = 13, AW_V_TOP = 29;     // octaves of the codes below a block's largest value
constexpr uint32_t AW_M_NAN = 127, AW_V_NAN = 255;

struct AwLaunch {
  AwTensor t[AW_TENSORS];
  uint32_t start[AW_TENSORS];   // first workgroup of each tensor
  int32_t count, run;           // tensors; values a workgroup takes (a multiple of 1024)
  AwScalars s;
};
static_assert(sizeof(AwLaunch) <= 4096, "kernel arguments");

__device__ __forceinline__ uint32_t aw_mix(uint32_t h) {
  h = (h ^ (h >> 15)) * 0x6A09E667u;
  h = (h ^ (h >> 13)) * 0x3C6EF373u;
  return h ^ (h >> 16);
}

// The larger of two pairs of 16-bit numbers, from another lane of the wave by DPP.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
template <int CTRL>
__device__ __forceinline__ uint32_t aw_max2(uint32_t x) {
  const uint32_t y = uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xF, 0xF, false));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, x), __builtin_bit_cast(u16x2_t, y)));
}
// Over the wave, the same in every lane (scalar).  Rows of 16 lanes first, then lane 15
// of each row into the next and lane 31 into the upper half; lanes without a source take 0.
__device__ __forceinline__ uint32_t aw_wave_max2(uint32_t x) {
  x = aw_max2<0xB1>(x);    // quad_perm 1 0 3 2
  x = aw_max2<0x4E>(x);    // quad_perm 2 3 0 1
  x = aw_max2<0x141>(x);   // row_half_mirror
  x = aw_max2<0x140>(x);   // row_mirror
  x = aw_max2<0x142>(x);   // row_bcast 15
  x = aw_max2<0x143>(x);   // row_bcast 31
  return uint32_t(__builtin_amdgcn_readlane(int(x), 63));
}

// Codes are fp32's own: with code c as the exponent's low bits and the mantissa's upper
// three, c << 20, octaves, steps and the even steps below the lowest octave (fp32's
// subnormal values) are all there, times 2^-129 of a code's lowest place.  So a code and
// its value are a scaling and a shift apart (5 and 9 operations a value in place of 8
// and 20: 333 -> 310 us for 100 M values).  `by`: top - 126 - e, the scaling to codes.
__device__ __forceinline__ float aw_value(uint32_t c, int by) { return __builtin_amdgcn_ldexpf(__uint_as_float(c << 20), -by); }
// The code of a finite x >= 0, rounded up with probability equal to what is cut off (r: 16
// random bits).
__device__ __forceinline__ uint32_t aw_code(float x, int by, uint32_t r) {
  return (__float_as_uint(__builtin_amdgcn_ldexpf(x, by)) + (r << 4)) >> 20;
}
__device__ __forceinline__ float aw_m(uint32_t c, int by) {
  const float m = aw_value(c & 127u, by);
  return (c & 127u) == AW_M_NAN ? __builtin_nanf("") : __uint_as_float(__float_as_uint(m) | (c & 128u) << 24);
}
__device__ __forceinline__ float aw_v(uint32_t c, int by) { return c == AW_V_NAN ? __builtin_nanf("") : aw_value(c, by); }
__device__ __forceinline__ int aw_by(int field, int top) { return top + 1 - field; }   // field: the stored byte, e + 127

// Exponents as stored: of the largest finite value, between -126 and 127.  (A field of
// 0 is that of values below 2^-126, which take the lowest exponent.)
__device__ __forceinline__ int aw_exp_field(float x) {
  const int f = int(__float_as_uint(x) >> 23 & 255u);
  return f == 255 ? 0 : f;
}

struct AwBlock {
  float p[4], g[4], m[4], v[4];
  uint32_t cm, cv;
  int em, ev;
};

template <bool EIGHT>
__device__ __forceinline__ void aw_load(const AwTensor& t, int64_t i, int in, bool vec, AwBlock& b) {
  if (vec && in >= 4) {
    const float4 p = *reinterpret_cast<const float4*>(t.p + i);
    b.p[0] = p.x; b.p[1] = p.y; b.p[2] = p.z; b.p[3] = p.w;
    if (t.flags & AW_GRAD_BF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t.g) + i);
      b.g[0] = bf16lo(u.x); b.g[1] = bf16hi(u.x); b.g[2] = bf16lo(u.y); b.g[3] = bf16hi(u.y);
    } else {
      const float4 g = *reinterpret_cast<const float4*>(static_cast<const float*>(t.g) + i);
      b.g[0] = g.x; b.g[1] = g.y; b.g[2] = g.z; b.g[3] = g.w;
    }
    if constexpr (EIGHT) {
      b.cm = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i);
      b.cv = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i);
    } else {
      const float4 m = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + i);
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + i);
      b.m[0] = m.x; b.m[1] = m.y; b.m[2] = m.z; b.m[3] = m.w;
      b.v[0] = v.x; b.v[1] = v.y; b.v[2] = v.z; b.v[3] = v.w;
    }
  } else {
    b.cm = b.cv = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b.p[j] = b.g[j] = b.m[j] = b.v[j] = 0.f;
      if (j >= in) continue;
      b.p[j] = t.p[i + j];
      b.g[j] = t.flags & AW_GRAD_BF16 ? load1<ACT_BF16>(t.g, size_t(i + j)) : load1<ACT_F32>(t.g, size_t(i + j));
      if constexpr (EIGHT) {
        b.cm |= uint32_t(static_cast<const uint8_t*>(t.m)[i + j]) << (8 * j);
        b.cv |= uint32_t(static_cast<const uint8_t*>(t.v)[i + j]) << (8 * j);
      } else {
        b.m[j] = static_cast<const float*>(t.m)[i + j];
        b.v[j] = static_cast<const float*>(t.v)[i + j];
      }
    }
  }
}

template <bool EIGHT>
__device__ __forceinline__ void aw_store(const AwTensor& t, int64_t i, int in, bool vec, const AwBlock& b) {
  if (vec && in >= 4) {
    *reinterpret_cast<float4*>(t.p + i) = make_float4(b.p[0], b.p[1], b.p[2], b.p[3]);
    if (t.copy) *reinterpret_cast<uint2*>(t.copy + i) = make_uint2(pack_bf16x2(b.p[0], b.p[1]), pack_bf16x2(b.p[2], b.p[3]));
    if constexpr (EIGHT) {
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i) = b.cm;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i) = b.cv;
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(t.m) + i) = make_float4(b.m[0], b.m[1], b.m[2], b.m[3]);
      *reinterpret_cast<float4*>(static_cast<float*>(t.v) + i) = make_float4(b.v[0], b.v[1], b.v[2], b.v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= in) continue;
      t.p[i + j] = b.p[j];
      if (t.copy) t.copy[i + j] = uint16_t(pack_bf16x2(b.p[j], b.p[j]));
      if constexpr (EIGHT) {
        static_cast<uint8_t*>(t.m)[i + j] = uint8_t(b.cm >> (8 * j));
        static_cast<uint8_t*>(t.v)[i + j] = uint8_t(b.cv >> (8 * j));
      } else {
        static_cast<float*>(t.m)[i + j] = b.m[j];
        static_cast<float*>(t.v)[i + j] = b.v[j];
      }
    }
  }
}

// A run of one tensor's values from `base` on.
template <bool EIGHT>
__device__ __forceinline__ void aw_run(const AwTensor& t, int64_t base, int run, const AwScalars& s) {
  const bool vec = t.flags & AW_ALIGNED;
  const int64_t end = min(t.n, base + run);
  float gs = 1.f, lr = 0.f, by1 = s.by1, root2 = s.root2;
  int64_t step = s.step;
  bool ready = false;
  float stay = 0.f, to = 0.f;
  uint32_t key = 0;
  for (int64_t at = base; at < end; at += 1024) {
    const int64_t i = at + 4 * int(threadIdx.x);
    const int in = int(min(end - i, int64_t(4)));   // this thread's values, 0 or less past the end
    AwBlock b;
    int fm = 0, fv = 0;
    const int64_t block = (at >> 8) + (threadIdx.x >> 6);
    if constexpr (EIGHT) {
      if (256 * block < t.n) {
        fm = t.me[block];
        fv = t.ve[block];
      }
    }
    aw_load<EIGHT>(t, i, in, vec, b);
    if (!ready) {   // behind the first loads, which it does not wait for
      ready = true;
      if (s.grad_scale) gs = *s.grad_scale;
      lr = (s.lr_device ? *s.lr_device : s.lr) * t.lr_scale;
      if (s.step_device) {
        step = *s.step_device;
        by1 = float(-1.0 / expm1(double(step) * s.log1));
        root2 = float(1.0 / sqrt(-expm1(double(step) * s.log2)));
      }
      stay = 1.f - lr * t.decay;
      to = lr * by1;
      if constexpr (EIGHT) key = aw_mix(uint32_t(step) * 0x9E3779B1u + aw_mix(t.index * 0xBB67AE85u + s.seed));
    }
    if constexpr (EIGHT) {
      const int lm = aw_by(fm, AW_M_TOP), lv = aw_by(fv, AW_V_TOP);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b.m[j] = aw_m(b.cm >> (8 * j) & 255u, lm);
        b.v[j] = aw_v(b.cv >> (8 * j) & 255u, lv);
      }
    }
    uint32_t top = 0;   // exponent fields of the largest m' (low half) and v'
    float root[4], least = 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float g = b.g[j] * gs;
      b.m[j] = fmaf(s.beta1, b.m[j], s.rest1 * g);
      b.v[j] = fmaf(s.beta2, b.v[j], s.rest2 * (g * g));
      // one unit in the last place of the hardware's root and reciprocal is far below
      // what p' is rounded by
      root[j] = __builtin_amdgcn_sqrtf(b.v[j]);
      least = fminf(least, b.v[j]);
    }
    if (least < 0x1p-126f) {   // the hardware's root takes subnormal numbers as 0
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (b.v[j] < 0x1p-126f) root[j] = __builtin_amdgcn_sqrtf(b.v[j] * 0x1p64f) * 0x1p-32f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float den = fmaf(root[j], root2, s.eps);
      b.p[j] = fmaf(-to * b.m[j], __builtin_amdgcn_rcpf(den), b.p[j] * stay);
      if constexpr (EIGHT) {
        const u16x2_t f = {(unsigned short)(aw_exp_field(b.m[j])), (unsigned short)(aw_exp_field(b.v[j]))};
        top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, top), f));
      }
    }
    if constexpr (EIGHT) {
      top = aw_wave_max2(top);
      const int nm = max(int(top & 0xFFFFu), 1), nv = max(int(top >> 16), 1);
      const int lm = aw_by(nm, AW_M_TOP), lv = aw_by(nv, AW_V_TOP);
      b.cm = b.cv = 0;
      const uint32_t h0 = uint32_t(i) * 0x9E3779B1u + uint32_t(i >> 32) * 0xBB67AE85u + key;   // i is a multiple of 4
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t h = aw_mix(h0 + j * 0x9E3779B1u);
        const uint32_t um = __float_as_uint(b.m[j]), uv = __float_as_uint(b.v[j]), am = um & 0x7FFFFFFFu;
        uint32_t c = aw_code(__uint_as_float(am), lm, h & 0xFFFFu), d = max(aw_code(b.v[j], lv, h >> 16), min(uv, 1u));
        c = am >= 0x7F800000u ? AW_M_NAN : c;
        d = uv >= 0x7F800000u ? AW_V_NAN : d;
        b.cm |= (c | (um >> 24 & 128u)) << (8 * j);
        b.cv |= d << (8 * j);
      }
      if (max(nm, nv) == 254) {   // what a largest value would be rounded up to is 2^128: its own code instead
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (nm == 254 && (b.cm >> (8 * j) & 127u) == 8 * AW_M_TOP + 16) b.cm -= 1u << (8 * j);
          if (nv == 254 && (b.cv >> (8 * j) & 255u) == 8 * AW_V_TOP + 16) b.cv -= 1u << (8 * j);
        }
      }
      if ((threadIdx.x & 63) == 0 && 256 * block < t.n) {
        t.me[block] = uint8_t(nm);
        t.ve[block] = uint8_t(nv);
      }
    }
    aw_store<EIGHT>(t, i, in, vec, b);
  }
}

// Which tensor workgroup `bid` is in: each lane compares one tensor's first workgroup.
__device__ __forceinline__ int aw_find(const AwLaunch& a, uint32_t bid) {
  const int lane = threadIdx.x & 63;
  const bool past = lane < a.count && a.start[lane < AW_TENSORS ? lane : 0] <= bid;
  return __builtin_amdgcn_readfirstlane(__builtin_popcountll(__ballot(past)) - 1);
}

__global__ __launch_bounds__(256) void aw_step_kernel(AwLaunch a) {
  const int k = aw_find(a, blockIdx.x);
  const AwTensor t = a.t[k];
  const int64_t base = int64_t(blockIdx.x - a.start[k]) * a.run;
  if (t.flags & AW_EIGHT) aw_run<true>(t, base, a.run, a.s);
  else aw_run<false>(t, base, a.run, a.s);
}

__global__ void aw_count_kernel(int64_t* step) { *step += 1; }

// The values of codes: p and copy hold where m's and v's go.
template <bool BF>
__device__ __forceinline__ void aw_put(void* out, int64_t i, int in, bool vec, const float (&x)[4]) {
  if (vec && in >= 4) {
    if constexpr (BF) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    else *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= in) continue;
      if constexpr (BF) static_cast<uint16_t*>(out)[i + j] = uint16_t(pack_bf16x2(x[j], x[j]));
      else static_cast<float*>(out)[i + j] = x[j];
    }
  }
}

template <bool BF>
__global__ __launch_bounds__(256) void aw_values_kernel(AwLaunch a) {
  const int k = aw_find(a, blockIdx.x);
  const AwTensor t = a.t[k];
  const int64_t base = int64_t(blockIdx.x - a.start[k]) * a.run, end = min(t.n, base + a.run);
  const bool vec = t.flags & AW_ALIGNED;
  for (int64_t at = base; at < end; at += 1024) {
    const int64_t i = at + 4 * int(threadIdx.x), block = i >> 8;
    const int in = int(min(end - i, int64_t(4)));
    if (in <= 0) continue;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      void* out = which ? static_cast<void*>(t.copy) : static_cast<void*>(t.p);
      if (!out) continue;
      const uint8_t* codes = static_cast<const uint8_t*>(which ? t.v : t.m) + i;
      const int by = aw_by((which ? t.ve : t.me)[block], which ? AW_V_TOP : AW_M_TOP);
      uint32_t u = 0;
      if (vec && in >= 4) {
        u = *reinterpret_cast<const uint32_t*>(codes);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < in) u |= uint32_t(codes[j]) << (8 * j);
      }
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = u >> (8 * j) & 255u;
        x[j] = which ? aw_v(c, by) : aw_m(c, by);
      }
      aw_put<BF>(out, i, in, vec, x);
    }
  }
}

namespace {


// launch(description, workgroups) for the tensors that have work, AW_TENSORS at a time
template <typename F>
hipError_t aw_launches(const AwTensor* tensors, int count, const AwScalars& s, int run, F&& launch) {
  AwLaunch a;
  a.s = s;
  a.run = run;
  a.count = 0;
  uint32_t blocks = 0;
  auto go = [&]() {
    if (a.count == 0) return hipSuccess;
    for (int j = a.count; j < AW_TENSORS; ++j) {
      a.t[j] = a.t[0];
      a.start[j] = 0;
    }
    launch(a, blocks);
    a.count = 0;
    blocks = 0;
    return hipGetLastError();
  };
  constexpr int64_t kMost = (int64_t(1) << 24) - 1;   // workgroups of a launch: its threads fit 32 bits
  for (int k = 0; k < count; ++k) {
    const int64_t need = (tensors[k].n + a.run - 1) / a.run;
    if (need == 0) continue;
    if (a.count == AW_TENSORS || blocks + need > kMost) {
      const hipError_t e = go();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = tensors[k];
    a.start[a.count++] = blocks;
    blocks += uint32_t(need);
  }
  return go();
}

}  // namespace

hipError_t launch_adamw(const AwTensor* tensors, int count, const AwScalars& s, int64_t* count_up, hipStream_t stream) {
  if (count_up) {
    hipLaunchKernelGGL(aw_count_kernel, dim3(1), dim3(1), 0, stream, count_up);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // a workgroup's values: steps of 100 M values in us 521, 526, 534, 542 for runs of 1024,
  // 2048, 4096, 8192 (fp32 moments), of 7 M in 120 tensors 42, 45, 48, 64 (codes)
  return aw_launches(tensors, count, s, 1024, [&](const AwLaunch& a, uint32_t blocks) {
    hipLaunchKernelGGL(aw_step_kernel, dim3(blocks), dim3(256), 0, stream, a);
  });
}

hipError_t launch_adamw_values(const AwTensor* tensors, int count, bool bf16, hipStream_t stream) {
  // 188, 157, 143, 141 us: nothing but short reads and stores in each
  return aw_launches(tensors, count, AwScalars{}, 4096, [&](const AwLaunch& a, uint32_t blocks) {
    if (bf16) hipLaunchKernelGGL((aw_values_kernel<true>), dim3(blocks), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((aw_values_kernel<false>), dim3(blocks), dim3(256), 0, stream, a);
  });
}

}  // namespace bmoe
