// Norms around a block (include/bmoe_block.h): the norm behind it, gate, residual and
// the norm in front of the next block, forward and backward.
//
// Bound by HBM: four rows read or written in the forward (b, r, s, y), six in the backward
// (dy, s, b, d_sum, db, dr), some 20 operations an element.  As in layer_norm.hip a row is
// held in registers between its loads and its stores and a workgroup loops over rows, which
// keeps the columns' weights and sums in registers.  Here that is five weights or four and
// four sums a column, so a thread has one group of 8 columns up to width 8192 (two beyond)
// and rows of more than 512 are shared by several waves.
#include "row_ops.hpp"
#include "step_ops.hpp"

namespace bmoe {

// The row's 1 / root mean square, x as it is: normed values are x rstd on return, x
// times a power of two where its squares leave fp32 or vanish in it.
template <int TPR, int NV, int E>
__device__ __forceinline__ LnStats bn_root(float (&x)[NV][E], int width, float eps, LnRed<TPR>& red, int& turn) {
  const float inv = 1.0f / float(width);
  float unit = 1.f, var = 0.f;
  auto squares = [&]() {
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) q[0] = fmaf(x[v][j], x[v][j], q[0]);
    ln_row_sum<TPR>(q, red, turn);
    var = q[0] * inv;
  };
  squares();
  const bool large = !(var < __builtin_inff()), small = var + eps < 0x1p-100f;
  if (large || small) {
    unit = large ? 0x1p-80f : 0x1p96f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) x[v][j] *= unit;
    squares();
  }
  return {0.f, 0.f, 1.0f / sqrtf(var + eps * unit * unit), unit};
}

// A weight's values for the thread's columns (`otherwise` without one): in registers over a
// workgroup's rows, or with 1024 threads, whose registers a row and its sums fill, read
// again where they are used.
template <int CUT, int TPR, int NV>
struct BnWeight {
  static constexpr bool KEEP = TPR < 1024;
  const float* p;
  int width, t;
  float otherwise, kept[KEEP ? NV : 1][8];
  __device__ __forceinline__ void read(int v, float (&w)[8]) const {
    const int at = 8 * (t + TPR * v);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = otherwise;
    if (p && at < width) ln_load<ACT_F32, CUT>(p, size_t(at), width - at, w);
  }
  __device__ __forceinline__ BnWeight(const void* q, float o, int wd, int th) : p(static_cast<const float*>(q)), width(wd), t(th), otherwise(o) {
    if constexpr (KEEP) {
#pragma unroll
      for (int v = 0; v < NV; ++v) read(v, kept[v]);
    }
  }
  __device__ __forceinline__ void get(int v, float (&w)[8]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = kept[v][j];
    } else {
      read(v, w);
    }
  }
};

// Threads of a workgroup: whole rows, and 256 at least of those that need no barrier.
constexpr int bn_threads(int tpr) { return tpr == 64 ? 256 : tpr; }
// Waves per SIMD that the registers leave room for.
constexpr int BN_FWD_WAVES = 4, BN_BWD_WAVES = 2;

template <int ACT, int CUT, int TPR, int NV>
__global__ __launch_bounds__(bn_threads(TPR), BN_FWD_WAVES) void bn_fwd_kernel(BnFwdArgs a) {
  constexpr int E = 8, RPW = bn_threads(TPR) / TPR;
  __shared__ LnRed<TPR> red;
  int turn = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, width = a.width;
  using Weight = BnWeight<CUT, TPR, NV>;
  const Weight wgp(a.gamma_post, 1.f, width, t), wbp(a.beta_post, 0.f, width, t),
      wgc(a.gate_kind == BN_GATE_CHANNEL ? a.gate : nullptr, 1.f, width, t), wga(a.gamma, 1.f, width, t), wbe(a.beta, 0.f, width, t);
  for (int row = blockIdx.x * RPW + sub; row < a.rows; row += gridDim.x * RPW) {
    const size_t at = size_t(row) * width;
    float x[NV][E], r[NV][E], gr[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[v][j] = r[v][j] = 0.f;
        gr[v][j] = 1.f;
      }
      if (in > 0) {
        ln_load<ACT, CUT>(a.b, at + size_t(g) * E, in, x[v]);
        if (a.r) ln_load<ACT, CUT>(a.r, at + size_t(g) * E, in, r[v]);
        if (a.gate_kind == BN_GATE_ROWS) ln_load<ACT, CUT>(a.gate, at + size_t(g) * E, in, gr[v]);
      }
    }
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.post) {
      const LnStats n = a.layer ? ln_centre<CUT, TPR>(x, width, t, a.eps, red, turn) : bn_root<TPR>(x, width, a.eps, red, turn);
      st.x = n.mean;
      st.y = n.rstd * n.unit;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float gp[E], bp[E];
        wgp.get(v, gp);
        wbp.get(v, bp);
#pragma unroll
        for (int j = 0; j < E; ++j) x[v][j] = fmaf((x[v][j] - n.off) * n.rstd, gp[j], bp[j]);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
      float gc[E];
      wgc.get(v, gc);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float z = a.scale * gc[j] * gr[v][j] * x[v][j];
        // 0 past the row, also where the row's norm is no number
        x[v][j] = (CUT == LN_ANY ? j < in : in > 0) ? (a.r ? fmaf(a.alpha, r[v][j], z) : z) : 0.f;
      }
      ln_round<ACT, E>(x[v]);
      if (in > 0) ln_store<ACT, CUT>(a.s, at + size_t(g) * E, in, x[v]);
    }
    const LnStats n = a.layer ? ln_centre<CUT, TPR>(x, width, t, a.eps, red, turn) : bn_root<TPR>(x, width, a.eps, red, turn);
    st.z = n.mean;
    st.w = n.rstd * n.unit;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
      float y[E], ga[E], be[E];
      wga.get(v, ga);
      wbe.get(v, be);
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = fmaf((x[v][j] - n.off) * n.rstd, ga[j], be[j]);
      if (in > 0) ln_store<ACT, CUT>(a.y, at + size_t(g) * E, in, y);
    }
    if (t == 0 && a.stats) a.stats[row] = st;
  }
}

// Backward.  Every workgroup keeps its columns' sums over its rows,
//     sum dy shat,  sum dy,  sum w bhat,  sum w   (bhat = b without the norm behind the block),
// w = ds or, with a gate of rows, scale gate ds, and writes them as one partial row; the
// gradients of all weights are multiples of their totals (bn_colsum_kernel).
template <int ACT, int DACT, int CUT, int TPR, int NV>
__global__ __launch_bounds__(bn_threads(TPR), TPR == 1024 ? 4 : BN_BWD_WAVES) void bn_bwd_kernel(BnBwdArgs a) {
  constexpr int E = 8, RPW = bn_threads(TPR) / TPR;
  __shared__ LnRed<TPR> red;
  __shared__ float cols[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * E : 1];
  int turn = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, width = a.width;
  const float inv = 1.0f / float(width);
  float sums[4][NV][E] = {};
  using Weight = BnWeight<CUT, TPR, NV>;
  const Weight wgp(a.gamma_post, 1.f, width, t), wbp(a.beta_post, 0.f, width, t),
      wgc(a.gate_kind == BN_GATE_CHANNEL ? a.gate : nullptr, 1.f, width, t), wga(a.gamma, 1.f, width, t);
  for (int row = blockIdx.x * RPW + sub; row < a.rows; row += gridDim.x * RPW) {
    const size_t at = size_t(row) * width;
    float x[NV][E], d[NV][E], b[NV][E], e[NV][E], gr[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[v][j] = d[v][j] = b[v][j] = e[v][j] = 0.f;
        gr[v][j] = 1.f;
      }
      if (in > 0) {
        const size_t i = at + size_t(g) * E;
        ln_load<ACT, CUT>(a.s, i, in, x[v]);
        ln_load<DACT, CUT>(a.dy, i, in, d[v]);
        ln_load<ACT, CUT>(a.b, i, in, b[v]);
        if (a.d_sum) ln_load<ACT, CUT>(a.d_sum, i, in, e[v]);
        if (a.gate_kind == BN_GATE_ROWS) ln_load<ACT, CUT>(a.gate, i, in, gr[v]);
      }
    }
    const float4 st = a.stats[row];
    float c[2] = {0.f, 0.f};  // sums of v and v shat, v = gamma dy
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int in = width - E * (t + TPR * v);
      float ga[E];
      wga.get(v, ga);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        // past the row dy is 0 and shat is made 0, so that an infinite 1 / deviation
        // reaches no other column
        x[v][j] = (CUT == LN_ANY ? j < in : in > 0) ? (x[v][j] - st.z) * st.w : 0.f;
        sums[0][v][j] = fmaf(d[v][j], x[v][j], sums[0][v][j]);
        sums[1][v][j] += d[v][j];
        d[v][j] *= ga[j];
        c[0] += d[v][j];
        c[1] = fmaf(d[v][j], x[v][j], c[1]);
      }
    }
    ln_row_sum<TPR>(c, red, turn);
    const float c0 = a.layer ? c[0] * inv : 0.f, c1 = c[1] * inv;
    float q[2] = {0.f, 0.f};  // the same of v = gamma_post dz and bhat
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
      const size_t i = at + size_t(g) * E;
      float o[E], dg[E], gp[E], bp[E], gc[E];
      wgp.get(v, gp);
      wbp.get(v, bp);
      wgc.get(v, gc);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const bool on = CUT == LN_ANY ? j < in : in > 0;
        const float ds = on ? fmaf(st.w, d[v][j] - c0 - x[v][j] * c1, e[v][j]) : 0.f;
        o[j] = a.alpha * ds;
        b[v][j] = a.post ? (on ? (b[v][j] - st.x) * st.y : 0.f) : b[v][j];
        const float dz = a.scale * ds;
        dg[j] = dz * fmaf(b[v][j], gp[j], bp[j]);
        const float dw = dz * gr[v][j];   // a gate of rows' part of it
        const float w = a.gate_kind == BN_GATE_ROWS ? dw : ds;
        sums[2][v][j] = fmaf(w, b[v][j], sums[2][v][j]);
        sums[3][v][j] += w;
        d[v][j] = dw * gc[j] * gp[j];
        q[0] += d[v][j];
        q[1] = fmaf(d[v][j], b[v][j], q[1]);
      }
      if (in > 0) {
        if (a.dr) ln_store<ACT, CUT>(a.dr, i, in, o);
        if (a.d_gate) ln_store<ACT, CUT>(a.d_gate, i, in, dg);
      }
    }
    float q0 = 0.f, q1 = 0.f, by = 1.f;
    if (a.post) {
      ln_row_sum<TPR>(q, red, turn);
      q0 = a.layer ? q[0] * inv : 0.f;
      q1 = q[1] * inv;
      by = st.y;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int g = t + TPR * v, in = width - E * g;
      float o[E];
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = by * (d[v][j] - q0 - b[v][j] * q1);
      if (in > 0) ln_store<ACT, CUT>(a.db, at + size_t(g) * E, in, o);
    }
  }
  if (!a.part) return;
  float* out = a.part + size_t(blockIdx.x) * 4 * width;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!a.layer && (k & 1)) continue;   // of no use to the other kind
    if constexpr (RPW == 1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = E * (t + TPR * v);
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (c + j < width) out[size_t(k) * width + c + j] = sums[k][v][j];
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < E; ++j) cols[sub][(t + TPR * v) * E + j] = sums[k][v][j];
      __syncthreads();
      for (int c = threadIdx.x; c < width; c += bn_threads(TPR)) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < RPW; ++w) s += cols[w][c];
        out[size_t(k) * width + c] = s;
      }
    }
  }
}

// The weights' gradients from P partial rows: 16 columns per workgroup, 16 groups of
// lanes that take the rows p, p + 16, ... each, their sums added in order.
__global__ __launch_bounds__(256) void bn_colsum_kernel(BnBwdArgs a, int P) {
  __shared__ float sm[4][16][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, c = blockIdx.x * 16 + col, width = a.width;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < width) {
#pragma unroll 4
    for (int p = grp; p < P; p += 16)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (a.layer || !(k & 1)) s[k] += a.part[(size_t(p) * 4 + k) * width + c];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sm[k][grp][col] = s[k];
  __syncthreads();
  if (grp != 0 || c >= width) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s[k] = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s[k] += sm[k][w][col];
  }
  const float gp = a.gamma_post ? a.gamma_post[c] : 1.f, bp = a.beta_post ? a.beta_post[c] : 0.f;
  const bool channel = a.gate_kind == BN_GATE_CHANNEL;
  const float by = a.gate_kind == BN_GATE_ROWS ? 1.f : a.scale * (channel ? static_cast<const float*>(a.gate)[c] : 1.f);
  if (a.d_gamma) a.d_gamma[c] = s[0];
  if (a.d_beta) a.d_beta[c] = s[1];
  if (a.d_gamma_post) a.d_gamma_post[c] = by * s[2];
  if (a.d_beta_post) a.d_beta_post[c] = by * s[3];
  if (a.d_gate_channel) a.d_gate_channel[c] = a.scale * (a.layer ? fmaf(gp, s[2], bp * s[3]) : gp * s[2]);
}

namespace {

bool bn_aligned(const void* p, size_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

constexpr int BN_CUS = 256;  // of a whole MI355X

// Threads of a row of `groups` groups of 8.
int bn_tpr(int groups) {
  int t = 64;
  while (t < groups && t < 1024) t *= 2;
  return t;
}

// Workgroups of the backward: what runs at a time.  Its rows of 4097 to 8192 go to 512
// threads, whose registers hold two groups with their sums, where 1024 would spill.
int bn_bwd_blocks(int rows, int width) {
  const int tpr = width > 8192 ? 1024 : bn_tpr((width + 7) / 8) < 512 ? bn_tpr((width + 7) / 8) : 512;
  const int threads = bn_threads(tpr), rpw = threads / tpr;
  const int need = (rows + rpw - 1) / rpw, most = tpr == 1024 ? BN_CUS : BN_CUS * (BN_BWD_WAVES * 256 / threads);
  return need < most ? need : most;
}

#define BN_SHAPES(GO, WIDE)                                            \
  const int tpr = bn_tpr((a.width + 7) / 8);                           \
  if (whole) {                                                         \
    if (a.width > 8192) return GO(LN_WHOLE, 1024, 2);                  \
    if (tpr == 1024) return WIDE(LN_WHOLE);                            \
    if (tpr == 512) return GO(LN_WHOLE, 512, 1);                       \
    if (tpr == 256) return GO(LN_WHOLE, 256, 1);                       \
    return tpr == 128 ? GO(LN_WHOLE, 128, 1) : GO(LN_WHOLE, 64, 1);    \
  }                                                                    \
  if (a.width > 8192) return GO(LN_ANY, 1024, 2);                      \
  if (tpr == 1024) return WIDE(LN_ANY);                                \
  if (tpr == 512) return GO(LN_ANY, 512, 1);                           \
  if (tpr == 256) return GO(LN_ANY, 256, 1);                           \
  return tpr == 128 ? GO(LN_ANY, 128, 1) : GO(LN_ANY, 64, 1);

template <int ACT, int CUT, int TPR, int NV>
hipError_t bn_fwd_go(const BnFwdArgs& a, hipStream_t s) {
  constexpr int RPW = bn_threads(TPR) / TPR;
  constexpr int most = BN_CUS * (BN_FWD_WAVES * 256 / bn_threads(TPR));
  const int blocks = (a.rows + RPW - 1) / RPW;
  hipLaunchKernelGGL((bn_fwd_kernel<ACT, CUT, TPR, NV>), dim3(unsigned(blocks < most ? blocks : most)),
                     dim3(bn_threads(TPR)), 0, s, a);
  return hipGetLastError();
}

template <int ACT>
hipError_t bn_fwd_act(const BnFwdArgs& a, bool whole, hipStream_t s) {
#define BN_GO(C, T, V) bn_fwd_go<ACT, C, T, V>(a, s)
#define BN_WIDE(C) BN_GO(C, 1024, 1)
  BN_SHAPES(BN_GO, BN_WIDE)
#undef BN_WIDE
#undef BN_GO
}

template <int ACT, int DACT, int CUT, int TPR, int NV>
hipError_t bn_bwd_go(const BnBwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((bn_bwd_kernel<ACT, DACT, CUT, TPR, NV>), dim3(unsigned(bn_bwd_blocks(a.rows, a.width))),
                     dim3(bn_threads(TPR)), 0, s, a);
  return hipGetLastError();
}

template <int ACT, int DACT>
hipError_t bn_bwd_act(const BnBwdArgs& a, bool whole, hipStream_t s) {
#define BN_GO(C, T, V) bn_bwd_go<ACT, DACT, C, T, V>(a, s)
#define BN_WIDE(C) BN_GO(C, 512, 2)
  BN_SHAPES(BN_GO, BN_WIDE)
#undef BN_WIDE
#undef BN_GO
}

}  // namespace

size_t bn_bwd_workspace(int rows, int width) { return size_t(bn_bwd_blocks(rows, width)) * 4 * width * 4; }

hipError_t launch_block_norm_fwd(const BnFwdArgs& a, int act, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const bool whole = a.width % 8 == 0 && bn_aligned(a.b, 16) && bn_aligned(a.r, 16) && bn_aligned(a.s, 16) && bn_aligned(a.y, 16) &&
                     bn_aligned(a.gate, 16) && bn_aligned(a.gamma_post, 16) && bn_aligned(a.beta_post, 16) &&
                     bn_aligned(a.gamma, 16) && bn_aligned(a.beta, 16);
  return act == ACT_BF16 ? bn_fwd_act<ACT_BF16>(a, whole, s) : bn_fwd_act<ACT_F32>(a, whole, s);
}

hipError_t launch_block_norm_bwd(const BnBwdArgs& a, int act, int dact, hipStream_t s) {
  const bool whole = a.width % 8 == 0 && bn_aligned(a.b, 16) && bn_aligned(a.s, 16) && bn_aligned(a.dy, 16) &&
                     bn_aligned(a.d_sum, 16) && bn_aligned(a.db, 16) && bn_aligned(a.dr, 16) && bn_aligned(a.d_gate, 16) &&
                     bn_aligned(a.gate, 16) && bn_aligned(a.gamma_post, 16) && bn_aligned(a.beta_post, 16) && bn_aligned(a.gamma, 16);
  if (a.rows > 0) {
    const hipError_t e = act == ACT_BF16 ? (dact == ACT_BF16 ? bn_bwd_act<ACT_BF16, ACT_BF16>(a, whole, s)
                                                             : bn_bwd_act<ACT_BF16, ACT_F32>(a, whole, s))
                                         : bn_bwd_act<ACT_F32, ACT_F32>(a, whole, s);
    if (e != hipSuccess) return e;
  }
  if (!a.d_gamma && !a.d_beta && !a.d_gamma_post && !a.d_beta_post && !a.d_gate_channel) return hipSuccess;
  hipLaunchKernelGGL(bn_colsum_kernel, dim3(unsigned((a.width + 15) / 16)), dim3(256), 0, s, a, a.rows > 0 ? bn_bwd_blocks(a.rows, a.width) : 0);
  return hipGetLastError();
}

}  // namespace bmoe
