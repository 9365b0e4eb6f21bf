// Norms around a block (include/bmoe_block.h): the norm behind it, gate, residual and
// the norm in front of the next block, forward and backward.
//
// Bound by HBM: four rows read or written in the forward (b, r, s, y), six in the backward
// (dy, s, b, d_sum, db, dr), some 20 operations an element.  As in layer_norm.hip a row is
// held in registers between its loads and its stores and a workgroup loops over rows, which
// keeps the columns' weights and sums in registers.  Here that is five weights or four and
// four sums a column, so a thread has one group of 8 columns up to width 8192 (two beyond, in
// the backward from 4097 on), and rows of more than 512 are shared by several waves, those
// of up to 256 share a wave.
//
// Every load is a whole group of 8 without a condition: where the width is no multiple
// of 8 a row's last group is its last 8 columns, of which the group before has some
// already (what is read of those is dropped), and threads past the row read its last group
// and drop all of it.  A condition around a load makes the wave wait for it at its end.
#include "row_ops.hpp"
#include "step_ops.hpp"

#include <algorithm>

namespace bmoe {

// Rows of whole groups at 16-byte alignment, any of 8 columns and more, of fewer.
enum BnCut { BN_WHOLE, BN_OVER, BN_NARROW };

// A thread's groups: the first column of group v, and which of its 8 elements are this
// thread's to count (on) and whether any are (any).
template <int CUT, int TPR>
struct BnCols {
  int width, t;
  __device__ __forceinline__ int first(int v) const { return CUT == BN_NARROW ? 0 : min(8 * (t + TPR * v), width - 8); }
  __device__ __forceinline__ bool any(int v) const { return 8 * (t + TPR * v) < width; }
  __device__ __forceinline__ bool on(int v, int j) const {
    if constexpr (CUT == BN_WHOLE) return any(v);
    else if constexpr (CUT == BN_OVER) return j >= 8 * (t + TPR * v) - (width - 8) || 8 * (t + TPR * v) <= width - 8;
    else return t == 0 && j < width;
  }
  template <int ACT>
  __device__ __forceinline__ void load(const void* p, size_t row, int v, float (&x)[8]) const {
    if constexpr (CUT == BN_NARROW) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = load1<ACT>(p, row + min(j, width - 1));
    } else {
      ln_load<ACT, CUT == BN_WHOLE ? LN_WHOLE : LN_ANY>(p, row + first(v), 8, x);
    }
  }
  // STREAM: past L2 where the alignment allows it (ln_store)
  template <int ACT, bool STREAM = true>
  __device__ __forceinline__ void store(void* p, size_t row, int v, const float (&x)[8]) const {
    if constexpr (CUT == BN_WHOLE && STREAM) {
      if (any(v)) ln_store<ACT, LN_WHOLE>(p, row + first(v), 8, x);
    } else {
      if (CUT != BN_NARROW && on(v, 0)) {
        ln_store<ACT, LN_ANY>(p, row + first(v), 8, x);
      } else if (any(v)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (on(v, j)) ln_store<ACT, LN_SINGLE>(p, row + first(v) + j, 1, x + j);
      }
    }
  }
};

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

// Waves per SIMD that the registers leave room for.
constexpr int BN_FWD_WAVES = 4, BN_BWD_WAVES = 3;

// A weight's values for the thread's columns (`otherwise` without one): in registers over
// a workgroup's rows (KEEP) or, where a row and its sums fill those, read in every row.
template <int CUT, int TPR, int NV, bool KEEP>
struct BnWeight {
  const float* p;
  BnCols<CUT, TPR> cols;
  float otherwise, kept[KEEP ? NV : 1][8];
  __device__ __forceinline__ void read(int v, float (&w)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = otherwise;
    if (p) cols.template load<ACT_F32>(p, 0, v, w);
  }
  __device__ __forceinline__ BnWeight(const void* q, float o, BnCols<CUT, TPR> c) : p(static_cast<const float*>(q)), cols(c), otherwise(o) {
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

// Threads of a workgroup: whole rows.  In the forward a row that takes barriers has the
// workgroup to itself, so that what its size asks for (LnStats) is everybody's (8192 x 1024
// fp32 26.3 us, with two rows to a workgroup 27.8).  The backward's partial rows are as many
// as its workgroups, so those of narrow rows are as large as the registers allow.
constexpr int bn_fwd_threads(int tpr) { return tpr > 64 ? tpr : 256; }
constexpr int bn_fwd_waves(int tpr) { return tpr > 256 ? 4 : BN_FWD_WAVES; }
// (Rows that share barriers wait for each other: with three of 2048 to a workgroup 32768 x
// 2048 takes 191 us in place of 180, 1024 x 2048 22 in place of 25.)
constexpr int bn_bwd_threads(int tpr) { return tpr <= 128 ? 256 * BN_BWD_WAVES : tpr; }

template <int ACT, int CUT, int TPR, int NV>
__global__ __launch_bounds__(bn_fwd_threads(TPR), bn_fwd_waves(TPR)) void bn_fwd_kernel(BnFwdArgs a) {
  constexpr int E = 8, RPW = bn_fwd_threads(TPR) / TPR;
  __shared__ LnRed<TPR> red;
  int turn = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, width = a.width;
  const BnCols<CUT, TPR> cols{width, t};
  constexpr bool KEEP = NV == 1;
  using Weight = BnWeight<CUT, TPR, NV, KEEP>;
  const Weight wga(a.gamma, 1.f, cols), wbe(a.beta, 0.f, cols);
  // scale gate z as xhat p + q (gamma_post and beta_post are 1 and 0 without the norm)
  auto fold = [&](int v, float (&p)[E], float (&q)[E]) {
    float gc[E];
    using Once = BnWeight<CUT, TPR, NV, false>;
    Once(a.gamma_post, 1.f, cols).get(v, p);
    Once(a.beta_post, 0.f, cols).get(v, q);
    Once(a.gate_kind == BN_GATE_CHANNEL ? a.gate : nullptr, 1.f, cols).get(v, gc);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      p[j] *= a.scale * gc[j];
      q[j] *= a.scale * gc[j];
    }
  };
  float wp[KEEP ? NV : 1][E], wq[KEEP ? NV : 1][E];
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < NV; ++v) fold(v, wp[v], wq[v]);
  }
  auto on = [&](int v, int j) { return cols.on(v, j); };
  // past the last row that one again, not stored
  for (int base = blockIdx.x * RPW; base < a.rows; base += gridDim.x * RPW) {
    const int row = min(base + sub, a.rows - 1);
    const bool live = base + sub < a.rows;
    const size_t at = size_t(row) * width;
    float x[NV][E], r[NV][E], gr[NV][E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        r[v][j] = 0.f;
        gr[v][j] = 1.f;
      }
      cols.template load<ACT>(a.b, at, v, x[v]);
      if (a.r) cols.template load<ACT>(a.r, at, v, r[v]);
      if (a.gate_kind == BN_GATE_ROWS) cols.template load<ACT>(a.gate, at, v, gr[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < E; ++j) x[v][j] = on(v, j) ? x[v][j] : 0.f;
    auto normed = [&]() {
      return a.layer ? ln_centre<TPR>(x, width, a.eps, red, turn, on) : bn_root<TPR>(x, width, a.eps, red, turn);
    };
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.post) {
      const LnStats n = normed();
      st.x = n.mean;
      st.y = n.rstd * n.unit;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < E; ++j) x[v][j] = (x[v][j] - n.off) * n.rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int l = KEEP ? v : 0;
      if constexpr (!KEEP) fold(v, wp[0], wq[0]);
      float o[E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float z = gr[v][j] * fmaf(x[v][j], wp[l][j], wq[l][j]);
        o[j] = a.r ? fmaf(a.alpha, r[v][j], z) : z;
      }
      ln_round<ACT, E>(o);
      if (live) cols.template store<ACT>(a.s, at, v, o);
#pragma unroll
      for (int j = 0; j < E; ++j) x[v][j] = on(v, j) ? o[j] : 0.f;   // also where the row's norm is no number
    }
    const LnStats n = normed();
    st.z = n.mean;
    st.w = n.rstd * n.unit;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float y[E], ga[E], be[E];
      wga.get(v, ga);
      wbe.get(v, be);
#pragma unroll
      for (int j = 0; j < E; ++j) y[j] = fmaf((x[v][j] - n.off) * n.rstd, ga[j], be[j]);
      if (live) cols.template store<ACT>(a.y, at, v, y);
    }
    if (live && t == 0 && a.stats) a.stats[row] = st;
  }
}

// Backward.  Every workgroup keeps its columns' sums over its rows,
//     sum dy shat,  sum dy,  sum w bhat,  sum w   (bhat = b without the norm behind the block),
// w = ds or, with a gate of rows, scale gate ds, and writes them as one partial row; the
// gradients of all weights are multiples of their totals (bn_colsum_kernel).
//
// Rows beyond 8192 leave no registers for all of these: the first two sums are in LDS, in
// places of the thread's own (2048 x 16384 bf16 514 us with them spilled).
constexpr int bn_bwd_waves(int tpr) { return tpr == 1024 ? 4 : tpr == 512 ? 2 : BN_BWD_WAVES; }
template <int ACT, int DACT, int CUT, int TPR, int NV>
__global__ __launch_bounds__(bn_bwd_threads(TPR), bn_bwd_waves(TPR)) void bn_bwd_kernel(BnBwdArgs a) {
  constexpr int E = 8, NT = bn_bwd_threads(TPR), RPW = NT / TPR;
  constexpr bool FAR = TPR == 1024, LATE = NV > 1;   // LATE: b, d_sum and gate read where they are used
  extern __shared__ __attribute__((aligned(16))) float far[];   // FAR: [2][NV * E][NT]
  __shared__ LnRed<TPR> red[TPR > 64 ? RPW : 1];
  __shared__ float staged[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * E : 1];
  int turn = 0;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, width = a.width;
  LnRed<TPR>& mine = red[TPR > 64 ? sub : 0];
  const BnCols<CUT, TPR> cols{width, t};
  const float inv = 1.0f / float(width);
  float sums[4][NV][E] = {};
  if constexpr (FAR) {
#pragma unroll
    for (int k = 0; k < 2 * NV * E; ++k) far[k * NT + threadIdx.x] = 0.f;
  }
  using Weight = BnWeight<CUT, TPR, NV, (TPR < 1024)>;
  const Weight wgp(a.gamma_post, 1.f, cols), wbp(a.beta_post, 0.f, cols),
      wgc(a.gate_kind == BN_GATE_CHANNEL ? a.gate : nullptr, 1.f, cols), wga(a.gamma, 1.f, cols);
  // all rows of a workgroup at a time, since they share its barriers; past the last row
  // that one again, not stored
  for (int base = blockIdx.x * RPW; base < a.rows; base += gridDim.x * RPW) {
    const int row = min(base + sub, a.rows - 1);
    const bool live = base + sub < a.rows;
    const size_t at = size_t(row) * width;
    float x[NV][E], d[NV][E], b[NV][E], e[LATE ? 1 : NV][E], gr[LATE ? 1 : NV][E];
    auto rest = [&](int v, float (&ev)[E], float (&gv)[E]) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        ev[j] = 0.f;
        gv[j] = 1.f;
      }
      if (a.d_sum) cols.template load<ACT>(a.d_sum, at, v, ev);
      if (a.gate_kind == BN_GATE_ROWS) cols.template load<ACT>(a.gate, at, v, gv);
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      cols.template load<ACT>(a.s, at, v, x[v]);
      cols.template load<DACT>(a.dy, at, v, d[v]);
      if constexpr (!LATE) {
        cols.template load<ACT>(a.b, at, v, b[v]);
        rest(v, e[v], gr[v]);
      }
    }
    const float4 st = a.stats[row];
    // what counts: this thread's columns, not those of a row that is there twice
    auto on = [&](int v, int j) { return live && cols.on(v, j); };
    float c[2] = {0.f, 0.f};  // sums of v and v shat, v = gamma dy
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float ga[E];
      wga.get(v, ga);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        // 0 in what does not count, so that nothing of it reaches a sum
        x[v][j] = on(v, j) ? (x[v][j] - st.z) * st.w : 0.f;
        d[v][j] = on(v, j) ? d[v][j] : 0.f;
        if constexpr (FAR) {
          float* f = far + (v * E + j) * NT + threadIdx.x;
          f[0] = fmaf(d[v][j], x[v][j], f[0]);
          f[NV * E * NT] += d[v][j];
        } else {
          sums[0][v][j] = fmaf(d[v][j], x[v][j], sums[0][v][j]);
          sums[1][v][j] += d[v][j];
        }
        d[v][j] *= ga[j];
        c[0] += d[v][j];
        c[1] = fmaf(d[v][j], x[v][j], c[1]);
      }
    }
    ln_row_sum<TPR>(c, mine, turn);
    const float c0 = a.layer ? c[0] * inv : 0.f, c1 = c[1] * inv;
    float q[2] = {0.f, 0.f};  // the same of v = gamma_post dz and bhat
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float o[E], dg[E], gp[E], bp[E], gc[E];
      wgp.get(v, gp);
      wbp.get(v, bp);
      wgc.get(v, gc);
      const int l = LATE ? 0 : v;
      if constexpr (LATE) {
        cols.template load<ACT>(a.b, at, v, b[v]);
        rest(v, e[0], gr[0]);
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float ds = on(v, j) ? fmaf(st.w, d[v][j] - c0 - x[v][j] * c1, e[l][j]) : 0.f;
        o[j] = a.alpha * ds;
        b[v][j] = on(v, j) ? (a.post ? (b[v][j] - st.x) * st.y : b[v][j]) : 0.f;
        const float dz = a.scale * ds;
        dg[j] = dz * fmaf(b[v][j], gp[j], bp[j]);
        const float dw = dz * gr[l][j];   // a gate of rows' part of it
        const float w = a.gate_kind == BN_GATE_ROWS ? dw : ds;
        sums[2][v][j] = fmaf(w, b[v][j], sums[2][v][j]);
        sums[3][v][j] += w;
        d[v][j] = dw * gc[j] * gp[j];
        q[0] += d[v][j];
        q[1] = fmaf(d[v][j], b[v][j], q[1]);
      }
      if (live && a.dr) cols.template store<ACT>(a.dr, at, v, o);
      if (live && a.d_gate) cols.template store<ACT>(a.d_gate, at, v, dg);
    }
    float q0 = 0.f, q1 = 0.f, by = 1.f;
    if (a.post) {
      ln_row_sum<TPR>(q, mine, turn);
      q0 = a.layer ? q[0] * inv : 0.f;
      q1 = q[1] * inv;
      by = st.y;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float o[E];
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = by * (d[v][j] - q0 - b[v][j] * q1);
      if (live) cols.template store<ACT>(a.db, at, v, o);
    }
  }
  if (!a.part) return;
  float* out = a.part + size_t(blockIdx.x) * 4 * width;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!a.layer && (k & 1)) continue;   // of no use to the other kind
    auto sum = [&](int v, int j) { return FAR && k < 2 ? far[(k * NV * E + v * E + j) * NT + threadIdx.x] : sums[k][v][j]; };
    if constexpr (RPW == 1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float w[E];
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = sum(v, j);
        cols.template store<ACT_F32, false>(out, size_t(k) * width, v, w);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (cols.on(v, j)) staged[sub][cols.first(v) + j] = sum(v, j);
      __syncthreads();
      for (int c = threadIdx.x; c < width; c += NT) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < RPW; ++w) s += staged[w][c];
        out[size_t(k) * width + c] = s;
      }
    }
  }
}

// The weights' gradients from P partial rows: 16 columns of two sums per workgroup (of s in
// the first half of the grid, of b in the other), 64 groups of lanes that take the rows p,
// p + 64, ... each, their sums added in order.
__global__ __launch_bounds__(1024) void bn_colsum_kernel(BnBwdArgs a, int P, int half) {
  __shared__ float sm[2][64][17];
  const bool post = int(blockIdx.x) >= half;
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4, c = (blockIdx.x - (post ? half : 0)) * 16 + col, width = a.width;
  float s[2] = {0.f, 0.f};
  const float* p = a.part + min(c, width - 1) + (post ? 2 * size_t(width) : 0);
#pragma unroll 8
  for (int r = grp; r < P; r += 64) {
    s[0] += p[size_t(r) * 4 * width];
    if (a.layer) s[1] += p[(size_t(r) * 4 + 1) * width];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) sm[k][grp][col] = s[k];
  __syncthreads();
  if (threadIdx.x < 256) {   // eight sums of eight groups for both, then those
    const int k = threadIdx.x >> 7, g = threadIdx.x >> 4 & 7;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sm[k][8 * g + w][col];
    sm[k][8 * g][col] = v;
  }
  __syncthreads();
  if (grp != 0 || c >= width) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    s[k] = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s[k] += sm[k][8 * w][col];
  }
  if (!post) {
    if (a.d_gamma) a.d_gamma[c] = s[0];
    if (a.d_beta) a.d_beta[c] = s[1];
    return;
  }
  const float gp = a.gamma_post ? a.gamma_post[c] : 1.f, bp = a.beta_post ? a.beta_post[c] : 0.f;
  const bool channel = a.gate_kind == BN_GATE_CHANNEL;
  const float by = a.gate_kind == BN_GATE_ROWS ? 1.f : a.scale * (channel ? static_cast<const float*>(a.gate)[c] : 1.f);
  if (a.d_gamma_post) a.d_gamma_post[c] = by * s[0];
  if (a.d_beta_post) a.d_beta_post[c] = by * s[1];
  if (a.d_gate_channel) a.d_gate_channel[c] = a.scale * (a.layer ? fmaf(gp, s[0], bp * s[1]) : gp * s[0]);
}

namespace {

bool bn_aligned(const void* p, size_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

constexpr int BN_CUS = 256;  // of a whole MI355X

// Threads of a row: a group of 8 columns each, 16 threads at least, 1024 at most.
int bn_tpr(int width) {
  int t = 16;
  while (8 * t < width && t < 1024) t *= 2;
  return t;
}

// Workgroups of the backward: what runs at a time, the rows spread evenly.  Its rows of
// 4097 to 8192 go to 512 threads, whose registers hold two groups with their sums, where
// 1024 would spill.  A workgroup of one row at a time takes up to 4 even where more
// workgroups would run: a partial row is as long as its row in fp32, four times (us by rows of
// a workgroup 1, 2, 3, 4: 500 x 2048 bf16 23.0, 17.0, 15.3, 15.2, 128 x 2048 11.0, 10.1, 10.9, 11.9,
// 200 x 4096 20.7, 15.5, 15.4, 15.7; with several rows at a time 300 x 1024 fp32 11.5, 13.5, 15.5,
// 18.5).
int bn_bwd_blocks(int rows, int width) {
  if (rows == 0) return 0;
  const int tpr = width > 8192 ? 1024 : bn_tpr(width) < 512 ? bn_tpr(width) : 512;
  const int threads = bn_bwd_threads(tpr), rpw = threads / tpr;
  const int need = (rows + rpw - 1) / rpw, most = BN_CUS * (bn_bwd_waves(tpr) * 256 / threads);
  int times = (need + most - 1) / most;
  if (rpw == 1) times = std::max(times, std::min(4, (need + 127) / 128));
  return (need + times - 1) / times;
}

#define BN_SHAPES(GO, WIDE)                                            \
  const int tpr = bn_tpr(a.width);                                     \
  if (a.width < 8) return GO(BN_NARROW, 16, 1);                        \
  if (whole) {                                                         \
    if (a.width > 8192) return GO(BN_WHOLE, 1024, 2);                  \
    if (tpr == 1024) return WIDE(BN_WHOLE);                            \
    if (tpr == 512) return GO(BN_WHOLE, 512, 1);                       \
    if (tpr == 256) return GO(BN_WHOLE, 256, 1);                       \
    if (tpr == 128) return GO(BN_WHOLE, 128, 1);                       \
    if (tpr == 64) return GO(BN_WHOLE, 64, 1);                         \
    return tpr == 32 ? GO(BN_WHOLE, 32, 1) : GO(BN_WHOLE, 16, 1);      \
  }                                                                    \
  if (a.width > 8192) return GO(BN_OVER, 1024, 2);                      \
  if (tpr == 1024) return WIDE(BN_OVER);                                \
  if (tpr == 512) return GO(BN_OVER, 512, 1);                           \
  if (tpr == 256) return GO(BN_OVER, 256, 1);                           \
  if (tpr == 128) return GO(BN_OVER, 128, 1);                          \
  if (tpr == 64) return GO(BN_OVER, 64, 1);                            \
  return tpr == 32 ? GO(BN_OVER, 32, 1) : GO(BN_OVER, 16, 1);

template <int ACT, int CUT, int TPR, int NV>
hipError_t bn_fwd_go(const BnFwdArgs& a, hipStream_t s) {
  constexpr int RPW = bn_fwd_threads(TPR) / TPR;
  constexpr int most = BN_CUS * (bn_fwd_waves(TPR) * 256 / bn_fwd_threads(TPR));
  const int blocks = (a.rows + RPW - 1) / RPW;
  hipLaunchKernelGGL((bn_fwd_kernel<ACT, CUT, TPR, NV>), dim3(unsigned(blocks < most ? blocks : most)),
                     dim3(bn_fwd_threads(TPR)), 0, s, a);
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
  constexpr size_t lds = TPR == 1024 ? size_t(2) * NV * 8 * TPR * 4 : 0;
  const auto kernel = bn_bwd_kernel<ACT, DACT, CUT, TPR, NV>;
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(unsigned(bn_bwd_blocks(a.rows, a.width))), dim3(bn_bwd_threads(TPR)), lds, s, a);
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
  const int half = (a.width + 15) / 16;
  const bool post = a.d_gamma_post || a.d_beta_post || a.d_gate_channel;
  hipLaunchKernelGGL(bn_colsum_kernel, dim3(unsigned(half * (post ? 2 : 1))), dim3(1024), 0, s, a,
                     a.rows > 0 ? bn_bwd_blocks(a.rows, a.width) : 0, half);
  return hipGetLastError();
}

}  // namespace bmoe
