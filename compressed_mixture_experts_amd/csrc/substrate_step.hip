// Step of a latent substrate and its ternary codes (include/bmoe_update.h):
//     W' = fl32((1 - decay) W - step O),  scale = mean |W'|,
//     code = sign(W') where 2 |W'| > scale.
// The codes need the mean over all of W', so there are two passes, both bound
// by memory: the first reads W and O, writes W' and one fp64 partial sum of
// |W'| per workgroup; the second adds the partial sums (every workgroup the
// same ones in the same order), reads W' again and writes 2 bits per weight.
// fp64 keeps the codes independent of how the sum was split: a weight's code
// could only differ if an fp32 number lay within about 1e-13 of the threshold
// relative to it.
//
// Few weights are one workgroup's, in one launch: it holds W' in registers between
// its sum and its codes, so nothing is read twice.
#include "step_ops.hpp"

namespace bmoe {

constexpr int SS_BLOCKS = 1024;  // most workgroups of the first pass
// Most weights of the single workgroup, 16 per thread: about where the GPU takes as
// long for the two launches (us there, one and two: 16 x 64 3.3 and 3.9, 64 x 256 5.2
// and 4.9, 96 x 256 7.2 and 5.0), while a call costs the host 9.3 and 13.4.
constexpr size_t SS_ONE = size_t(1) << 14;

__device__ __forceinline__ double ss_wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The sum over a workgroup of NT, valid in every thread.
template <int NT>
__device__ __forceinline__ double ss_block_sum(double v, double* red) {
  v = ss_wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v += red[w];
  return v;
}

// Four weights after the step: two products and a difference in fp64, one rounding
// to fp32.
__device__ __forceinline__ float4 ss_step(float4 w, uint2 o, double keep, double step) {
#pragma clang fp contract(off)
  w.x = float(keep * double(w.x) - step * double(bf16lo(o.x)));
  w.y = float(keep * double(w.y) - step * double(bf16hi(o.x)));
  w.z = float(keep * double(w.z) - step * double(bf16lo(o.y)));
  w.w = float(keep * double(w.w) - step * double(bf16hi(o.y)));
  return w;
}

__device__ __forceinline__ double ss_abs(float4 w) {
  return (fabs(double(w.x)) + fabs(double(w.y))) + (fabs(double(w.z)) + fabs(double(w.w)));
}

// The word of the 16 columns that four lanes hold between them, in each of the four.
__device__ __forceinline__ uint32_t ss_word(float4 v, double mean) {
  const float e[4] = {v.x, v.y, v.z, v.w};
  uint32_t code = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // column c = 4 (lane % 4) + j: bit 16 (c % 2) + c / 2, the sign 8 above;
    // false for a NaN weight and for a NaN or infinite mean
    if (2.0 * fabs(double(e[j])) > mean) code |= (e[j] < 0.f ? 0x101u : 0x1u) << (16 * (j & 1) + (j >> 1));
  }
  code <<= 2 * (threadIdx.x & 3);
  code |= __shfl_xor(code, 1);
  code |= __shfl_xor(code, 2);
  return code;
}

// All of it by one workgroup.
template <bool UPD>
__global__ __launch_bounds__(1024) void sub_one_kernel(SubStepArgs a) {
  constexpr int NV = int(SS_ONE / 4 / 1024);  // groups of four weights per thread
  __shared__ double red[16];
  const uint32_t quads = uint32_t(a.n / 4), t = threadIdx.x;
  float4 w[NV];
  uint2 o[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t q = t + 1024 * k;
    w[k] = q < quads ? reinterpret_cast<const float4*>(a.w)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
    if (UPD && q < quads) o[k] = reinterpret_cast<const uint2*>(a.o)[q];
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t q = t + 1024 * k;
    if (UPD && q < quads) {
      w[k] = ss_step(w[k], o[k], a.keep, a.step);
      reinterpret_cast<float4*>(a.w_out)[q] = w[k];
    }
    s += ss_abs(w[k]);
  }
  const double mean = ss_block_sum<1024>(s, red) / double(a.n);
  if (t == 0 && a.scale) *a.scale = float(mean);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const uint32_t q = t + 1024 * k, word = ss_word(w[k], mean);
    if ((t & 3) == 0 && q < quads) a.packed[q / 4] = word;
  }
}

template <bool UPD>
__global__ __launch_bounds__(256) void sub_update_kernel(SubStepArgs a) {
  __shared__ double red[4];
  const size_t quads = a.n / 4;
  double s = 0.0;
  for (size_t q = size_t(blockIdx.x) * 256 + threadIdx.x; q < quads; q += size_t(gridDim.x) * 256) {
    float4 w = reinterpret_cast<const float4*>(a.w)[q];
    if constexpr (UPD) {
      w = ss_step(w, reinterpret_cast<const uint2*>(a.o)[q], a.keep, a.step);
      reinterpret_cast<float4*>(a.w_out)[q] = w;
    }
    s += ss_abs(w);
  }
  s = ss_block_sum<256>(s, red);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void sub_codes_kernel(SubStepArgs a, const float* w, int blocks) {
  __shared__ double red[4];
  // a wave takes 1024 weights at a time, four loads of 1 KiB; four lanes hold the
  // 16 columns of a word between them, and lane l keeps the word of load l % 4
  const int lane = threadIdx.x & 63;
  const size_t words = a.n / 16, step = size_t(gridDim.x) * 256;
  size_t w0 = size_t(blockIdx.x) * 256 + (threadIdx.x & ~63u);
  float4 v[4];
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const size_t quad = 4 * w0 + 64 * k + lane;
      v[k] = quad < 4 * words ? reinterpret_cast<const float4*>(w)[quad] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load();  // on their way while the partial sums are added
  double s = 0.0;
  for (int p = threadIdx.x; p < blocks; p += 256) s += a.part[p];
  const double mean = ss_block_sum<256>(s, red) / double(a.n);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.scale) *a.scale = float(mean);
  while (w0 < words) {
    uint32_t keep = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t code = ss_word(v[k], mean);
      if ((lane & 3) == k) keep = code;
    }
    const size_t word = w0 + 16 * (lane & 3) + (lane >> 2);
    if (word < words) a.packed[word] = keep;
    w0 += step;
    load();
  }
}

static int ss_blocks(size_t n) {
  const size_t b = (n / 4 + 255) / 256;
  return int(b < SS_BLOCKS ? b : SS_BLOCKS);
}

size_t sub_step_workspace(size_t n) { return n <= SS_ONE ? 0 : size_t(ss_blocks(n)) * 8; }

hipError_t launch_sub_step(const SubStepArgs& a, hipStream_t s) {
  if (a.n <= SS_ONE) {
    if (a.o) hipLaunchKernelGGL(sub_one_kernel<true>, dim3(1), dim3(1024), 0, s, a);
    else hipLaunchKernelGGL(sub_one_kernel<false>, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  const int blocks = ss_blocks(a.n);
  if (a.o) hipLaunchKernelGGL(sub_update_kernel<true>, dim3(unsigned(blocks)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(sub_update_kernel<false>, dim3(unsigned(blocks)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t cb = (a.n / 16 + 255) / 256;
  hipLaunchKernelGGL(sub_codes_kernel, dim3(unsigned(cb < 2048 ? cb : 2048)), dim3(256), 0, s, a, a.o ? a.w_out : a.w,
                     blocks);
  return hipGetLastError();
}

}  // namespace bmoe
