// Orthogonalised update of a latent substrate (include/bmoe_update.h):
// momentum, Frobenius normalisation and five steps of the quintic
//     X <- a X + (b A + c A A) X = P X,   A = X X^T,  P = a I + b A + c A A
// taken on the smaller side S of the matrix (L the larger one).
//
// All products run on MFMA in fp16 with fp32 sums.  fp16 keeps 11 bits where
// bf16 keeps 8, and every factor's range is known: singular values stay below
// 1.21, so X is stored times 2^14, A, P and T times 2^13, Q times 2^11, far
// from both ends of fp16.
//
// Roundings.  A rounding of X adds noise in directions the gradient may not
// have, and a step multiplies what is small by a = 3.44: noise of X_0 grows
// 485-fold, that of X_2 41-fold.  A rounding of A, T, P or Q only bends P,
// which multiplies X from the left and adds no direction to its rows.  So X_0
// and X_2, where it matters most, are kept as hi + lo (two fp16 terms, 22
// bits) in the products P X, and the first two steps are taken together,
//     A_1 = P_0 A_0 P_0 = P_0 T,   Q = P_1 P_0,   X_2 = Q X_0,
// (everything in A is a polynomial of A_0: the factors commute and stay
// symmetric), which saves X_1's rounding and its two products with L.  With
// X in one fp16 term throughout, a gradient of rank S / 8 came out 2e-2 off,
// with this 3e-3; full-rank ones 1e-3.
//
// Symmetric results (A, T A, P, Q) compute only the tiles on and above the
// diagonal and write each also mirrored.
//
// Layouts: every product is D[m][n] = sum_k A[m][k] B[n][k], both operands
// with k contiguous.  A = X X^T reads X as XS [S][L]; X' = P X, taken as
// X'^T = X^T P (P symmetric), reads X as XL [L][S].  A product's epilogue
// writes its tile both ways.  S and L are padded to multiples of 128 with
// zeros, which stay zero.
#include "common.hpp"

namespace bmoe {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(1))) void ns_glob_t;
typedef __attribute__((address_space(3))) void ns_lds_t;

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr int NS_SUMS = 512;        // partial sums of squares
constexpr int NS_T = 128;           // output tile
constexpr int NS_K = 64;            // contraction step
constexpr int NS_TILE = NS_T * NS_K;
constexpr int NS_ST = NS_T + 4;     // row stride of the staged output tile (halves)
constexpr int NS_LDS = 2 * 2 * NS_TILE * 2;

// ------------------------------------------------------------------ momentum
template <bool BF>
__device__ __forceinline__ float ns_grad(const void* g, size_t i) {
  return load1<BF ? ACT_BF16 : ACT_F32>(g, i);
}

// U's element from the gradient and the momentum M' (as stored).
__device__ __forceinline__ float ns_u(float g, float m1, float mu, int nesterov) {
  return nesterov ? fmaf(mu, m1, g) : m1;
}

// M' = mu M + G and the sum of U^2 (fp64 partial sums, one per workgroup).
template <bool BF, bool V4>
__global__ __launch_bounds__(256) void ns_momentum_kernel(OrthoArgs a, double* part) {
  __shared__ double red[4];
  constexpr int W = V4 ? 4 : 1;
  const size_t n = size_t(a.rows) * a.cols / W;
  double s = 0.0;
  for (size_t q = size_t(blockIdx.x) * 256 + threadIdx.x; q < n; q += size_t(gridDim.x) * 256) {
    float g[W], m[W];
    if constexpr (V4) {
      if constexpr (BF) {
        const uint2 u = reinterpret_cast<const uint2*>(a.grad)[q];
        g[0] = bf16lo(u.x); g[1] = bf16hi(u.x); g[2] = bf16lo(u.y); g[3] = bf16hi(u.y);
      } else {
        const float4 u = reinterpret_cast<const float4*>(a.grad)[q];
        g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
      }
      if (a.m) {
        const float4 u = reinterpret_cast<const float4*>(a.m)[q];
        m[0] = u.x; m[1] = u.y; m[2] = u.z; m[3] = u.w;
      }
    } else {
      g[0] = ns_grad<BF>(a.grad, q);
      if (a.m) m[0] = a.m[q];
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float u = g[j];
      if (a.m) {
        m[j] = fmaf(a.mu, m[j], g[j]);
        u = ns_u(g[j], m[j], a.mu, a.nesterov);
      }
      s = fma(double(u), double(u), s);
    }
    if (a.m) {
      if constexpr (V4) reinterpret_cast<float4*>(a.m_out)[q] = make_float4(m[0], m[1], m[2], m[3]);
      else a.m_out[q] = m[0];
    }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
}

// X_0 = U / ||U||_F times 2^14 as fp16 hi (+ lo): 64 x 64 tiles of the padded
// matrix, written in the caller's orientation from registers and transposed
// through LDS.
struct NsCast {
  const double* part;       // NS_SUMS-bounded partial sums of U^2
  int32_t parts;
  _Float16* xs;             // [Sp][Lp]
  _Float16* xh;             // [Lp][Sp]
  _Float16* xl;             // [Lp][Sp]
  int32_t Sp, Lp;
};

template <bool BF>
__global__ __launch_bounds__(256) void ns_cast_kernel(OrthoArgs a, NsCast c) {
  __shared__ double red[4];
  __shared__ _Float16 th[64][68], tl[64][68];
  const int tid = threadIdx.x;
  double s = 0.0;
  for (int p = tid; p < c.parts; p += 256) s += c.part[p];
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  const double norm = sqrt(((red[0] + red[1]) + red[2]) + red[3]);
  // NaN for a norm that is NaN or infinite, so that all of the result is NaN
  const double scale = norm > 0.0 ? (norm < __builtin_inf() ? 16384.0 / norm : __builtin_nan("")) : (norm == 0.0 ? 0.0 : norm);
  const bool tall = a.rows > a.cols;
  const int cp = tall ? c.Sp : c.Lp;  // padded columns
  const int tc = cp / 64;
  const int r0 = int(blockIdx.x / tc) * 64, c0 = int(blockIdx.x % tc) * 64;
  const int lc = 4 * (tid & 15);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = 16 * i + (tid >> 4), r = r0 + lr;
    f16x4_t hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = c0 + lc + j;
      float v = 0.f;
      if (r < a.rows && col < a.cols) {
        const size_t at = size_t(r) * a.cols + col;
        const float g = ns_grad<BF>(a.grad, at);
        v = float(double(a.m ? ns_u(g, a.m_out[at], a.mu, a.nesterov) : g) * scale);
      }
      hi[j] = _Float16(v);
      lo[j] = _Float16(v - float(hi[j]));
    }
    *reinterpret_cast<f16x4_t*>(&th[lr][lc]) = hi;
    *reinterpret_cast<f16x4_t*>(&tl[lr][lc]) = lo;
    const size_t at = size_t(r) * cp + c0 + lc;
    if (tall) {
      *reinterpret_cast<f16x4_t*>(c.xh + at) = hi;
      *reinterpret_cast<f16x4_t*>(c.xl + at) = lo;
    } else {
      *reinterpret_cast<f16x4_t*>(c.xs + at) = hi;
    }
  }
  __syncthreads();
  const int rp = tall ? c.Lp : c.Sp;  // padded rows
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tcx = 16 * i + (tid >> 4);  // column of the tile, row of the transposed one
    f16x4_t hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = th[lc + j][tcx];
      lo[j] = tl[lc + j][tcx];
    }
    const size_t at = size_t(c0 + tcx) * rp + r0 + lc;
    if (tall) {
      *reinterpret_cast<f16x4_t*>(c.xs + at) = hi;
    } else {
      *reinterpret_cast<f16x4_t*>(c.xh + at) = hi;
      *reinterpret_cast<f16x4_t*>(c.xl + at) = lo;
    }
  }
}

// ------------------------------------------------------------------ products
enum NsMode { NS_SYM = 0, NS_PROD = 1, NS_LAST = 2 };

struct NsGemm {
  const _Float16* a;        // [M][K]
  const _Float16* a2;       // second term of the left operand, or null
  const _Float16* b;        // [N][K]
  int32_t M, N, K;          // multiples of NS_T, NS_T and NS_K
  float alpha;              // D = alpha sum (+ beta C + diag on the diagonal)
  // NS_SYM: d [N][N]; c [N][N] or null
  const _Float16* c;
  float beta, diag;
  _Float16* d;              // NS_SYM; NS_PROD: D's hi [M][N]
  _Float16* lo;             // NS_PROD: D's lo [M][N], or null
  _Float16* dt;             // NS_PROD: D's hi transposed [N][M]
  // NS_LAST: bf16, D cut to rows x cols and transposed back when wide
  uint16_t* out;
  int32_t rows, cols;       // of out
};

// One workgroup of four waves per 128 x 128 tile of D, each wave 64 x 64 (4 x 4
// MFMA blocks of 16 x 16 x 32).  Both operand tiles of a 64-deep step come
// straight into LDS (16 bytes per lane), the next step's while this one's
// products run, two buffers.  Chunk ch (16 bytes) of row r sits at ch ^ (r % 8)
// of its row.
template <int MODE>
__global__ __launch_bounds__(256, 2) void ns_gemm_kernel(NsGemm p) {
  extern __shared__ __attribute__((aligned(16))) _Float16 sm[];  // [2][A tile | B tile]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int wm = wave & 1, wn = wave >> 1;
  int tm, tn;
  {
    int t = xcd_remap(blockIdx.x, gridDim.x);
    const int nt = p.N / NS_T;
    if constexpr (MODE == NS_SYM) {
      tm = 0;
      while (t >= nt - tm) {
        t -= nt - tm;
        ++tm;
      }
      tn = tm + t;
    } else {
      tm = t / nt;
      tn = t % nt;
    }
  }
  const int m0 = tm * NS_T, n0 = tn * NS_T;
  const int K = p.K, nk1 = K / NS_K, nk = p.a2 ? 2 * nk1 : nk1;
  // loads of a step: 32 of 8 rows each, 8 per wave; waves 0 and 1 A, 2 and 3 B
  const int lrow = 64 * (wave & 1) + (lane >> 3), lch = 8 * ((lane & 7) ^ (lane >> 3));
  const bool isb = wave >= 2;
  const size_t lbase = size_t((isb ? n0 : m0) + lrow) * K + lch;
  auto load = [&](int kt, int buf) {
    const bool second = kt >= nk1;
    const _Float16* src = (isb ? p.b : second ? p.a2 : p.a) + lbase + (second ? kt - nk1 : kt) * NS_K;
    _Float16* dst = sm + buf * 2 * NS_TILE + (isb ? NS_TILE : 0) + 64 * (wave & 1) * NS_K;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      __builtin_amdgcn_global_load_lds((ns_glob_t*)(src + size_t(8 * j) * K), (ns_lds_t*)(dst + 8 * j * NS_K), 16, 0, 0);
  };
  f32x4_t acc[4][4];  // [n block][m block]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  load(0, 0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < nk) load(kt + 1, buf ^ 1);
    const _Float16* A = sm + buf * 2 * NS_TILE + (64 * wm + l16) * NS_K;
    const _Float16* B = sm + buf * 2 * NS_TILE + NS_TILE + (64 * wn + l16) * NS_K;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int ch = 8 * ((4 * s + g) ^ (l16 & 7));
      f16x8_t fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fa[i] = *reinterpret_cast<const f16x8_t*>(A + 16 * i * NS_K + ch);
        fb[i] = *reinterpret_cast<const f16x8_t*>(B + 16 * i * NS_K + ch);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[i], fa[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();  // waits for this wave's loads, then for every wave
  }
  // acc[i][j][r] = D[m0 + 64 wm + 16 j + l16][n0 + 64 wn + 16 i + 4 g + r]
  _Float16* st = sm;  // [NS_T][NS_ST]
  const int rows_m = 64 * wm + l16, cols_n = 64 * wn + 4 * g;
  auto staged = [&](auto&& f) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f16x4_t*>(st + (rows_m + 16 * j) * NS_ST + cols_n + 16 * i) = f(i, j);
    __syncthreads();
  };
  // the staged tile to dst (row stride ld) as it is
  auto direct = [&](_Float16* dst, size_t ld) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = 16 * q + (tid >> 4), c = 8 * (tid & 15);
      const uint2 u = *reinterpret_cast<const uint2*>(st + r * NS_ST + c);
      const uint2 v = *reinterpret_cast<const uint2*>(st + r * NS_ST + c + 4);
      *reinterpret_cast<uint4*>(dst + size_t(r) * ld + c) = make_uint4(u.x, u.y, v.x, v.y);
    }
  };
  // column c of the staged tile, rows r .. r + 7
  auto column8 = [&](int c, int r) {
    f16x8_t v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = st[(r + e) * NS_ST + c];
    return v;
  };
  auto transposed = [&](_Float16* dst, size_t ld) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = 32 * (q >> 1) + (tid >> 3), r = 8 * (tid & 7) + 64 * (q & 1);
      *reinterpret_cast<f16x8_t*>(dst + size_t(c) * ld + r) = column8(c, r);
    }
  };
  if constexpr (MODE == NS_SYM) {
    staged([&](int i, int j) {
      const int m = m0 + rows_m + 16 * j, n = n0 + cols_n + 16 * i;
      f16x4_t cv = {0, 0, 0, 0}, o;
      if (p.c) cv = *reinterpret_cast<const f16x4_t*>(p.c + size_t(m) * p.N + n);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = fmaf(p.alpha, acc[i][j][r], p.beta * float(cv[r]));
        if (m == n + r) v += p.diag;
        o[r] = _Float16(v);
      }
      return o;
    });
    direct(p.d + size_t(m0) * p.N + n0, p.N);
    if (tm != tn) transposed(p.d + size_t(n0) * p.N + m0, p.N);
  } else if constexpr (MODE == NS_PROD) {
    staged([&](int i, int j) {
      f16x4_t o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = _Float16(p.alpha * acc[i][j][r]);
      return o;
    });
    direct(p.d + size_t(m0) * p.N + n0, p.N);
    transposed(p.dt + size_t(n0) * p.M + m0, p.M);
    if (p.lo) {
      __syncthreads();
      staged([&](int i, int j) {
        f16x4_t o;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = p.alpha * acc[i][j][r];
          o[r] = _Float16(v - float(_Float16(v)));
        }
        return o;
      });
      direct(p.lo + size_t(m0) * p.N + n0, p.N);
    }
  } else {
    staged([&](int i, int j) {
      uint2 o;
      o.x = pack_bf16x2(p.alpha * acc[i][j][0], p.alpha * acc[i][j][1]);
      o.y = pack_bf16x2(p.alpha * acc[i][j][2], p.alpha * acc[i][j][3]);
      return __builtin_bit_cast(f16x4_t, o);
    });
    const bool tall = p.rows > p.cols;
    const size_t ld = p.cols;
    const bool vec = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      int r, c;  // of out
      f16x8_t v;
      if (tall) {
        const int lr = 16 * q + (tid >> 4), lc = 8 * (tid & 15);
        r = m0 + lr;
        c = n0 + lc;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = st[lr * NS_ST + lc + e];
      } else {
        const int lc = 32 * (q >> 1) + (tid >> 3), lr = 8 * (tid & 7) + 64 * (q & 1);
        r = n0 + lc;
        c = m0 + lr;
        v = column8(lc, lr);
      }
      if (r >= p.rows || c >= p.cols) continue;
      uint16_t* dst = p.out + size_t(r) * ld + c;
      const uint4 u = __builtin_bit_cast(uint4, v);
      if (vec) {
        *reinterpret_cast<uint4*>(dst) = u;
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.cols) dst[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

// ------------------------------------------------------------------ host
namespace {

struct NsPlan {
  size_t part, xs, xh[2], xl[2], A, T, P, Q, total;
  int S, L, Sp, Lp;
};

NsPlan ns_plan(int rows, int cols) {
  NsPlan q{};
  q.S = rows < cols ? rows : cols;
  q.L = rows < cols ? cols : rows;
  q.Sp = (q.S + NS_T - 1) / NS_T * NS_T;
  q.Lp = (q.L + NS_T - 1) / NS_T * NS_T;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t x = size_t(q.Sp) * q.Lp * 2, s = size_t(q.Sp) * q.Sp * 2;
  q.part = take(NS_SUMS * 8);
  q.xs = take(x);
  for (int k = 0; k < 2; ++k) {
    q.xh[k] = take(x);
    q.xl[k] = take(x);
  }
  q.A = take(s);
  q.T = take(s);
  q.P = take(s);
  q.Q = take(s);
  q.total = o;
  return q;
}

template <int MODE>
hipError_t ns_go(const NsGemm& p, hipStream_t s) {
  const int nt = p.N / NS_T;
  const int tiles = MODE == NS_SYM ? nt * (nt + 1) / 2 : (p.M / NS_T) * nt;
  hipLaunchKernelGGL(ns_gemm_kernel<MODE>, dim3(unsigned(tiles)), dim3(256), NS_LDS, s, p);
  return hipGetLastError();
}

}  // namespace

size_t ortho_workspace(int rows, int cols) { return ns_plan(rows, cols).total; }

hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t s) {
  const NsPlan q = ns_plan(a.rows, a.cols);
  char* ws = static_cast<char*>(a.ws);
  auto at = [&](size_t off) { return reinterpret_cast<_Float16*>(ws + off); };
  double* part = reinterpret_cast<double*>(ws + q.part);
  const size_t n = size_t(a.rows) * a.cols;
  auto al = [](const void* p, size_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; };
  const bool v4 = n % 4 == 0 && al(a.grad, a.grad_bf16 ? 8 : 16) && al(a.m, 16) && al(a.m_out, 16);
  const size_t work = (v4 ? n / 4 : n);
  const size_t nb = (work + 255) / 256;
  const int blocks = int(nb < NS_SUMS ? nb : NS_SUMS);
#define NS_MOM(BF, V) hipLaunchKernelGGL((ns_momentum_kernel<BF, V>), dim3(unsigned(blocks)), dim3(256), 0, s, a, part)
  if (a.grad_bf16) {
    if (v4) NS_MOM(true, true);
    else NS_MOM(true, false);
  } else {
    if (v4) NS_MOM(false, true);
    else NS_MOM(false, false);
  }
#undef NS_MOM
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const NsCast c{part, blocks, at(q.xs), at(q.xh[0]), at(q.xl[0]), q.Sp, q.Lp};
  const unsigned tiles = unsigned((q.Sp / 64) * (q.Lp / 64));
  if (a.grad_bf16) hipLaunchKernelGGL(ns_cast_kernel<true>, dim3(tiles), dim3(256), 0, s, a, c);
  else hipLaunchKernelGGL(ns_cast_kernel<false>, dim3(tiles), dim3(256), 0, s, a, c);
  e = hipGetLastError();
  if (e != hipSuccess) return e;

  constexpr float up13 = 8192.f, dn13 = 1.f / 8192.f;
  _Float16 *A = at(q.A), *T = at(q.T), *P = at(q.P), *Q = at(q.Q);
  NsGemm sym{};
  sym.M = sym.N = q.Sp;
  // A (2^13) = XS XS^T, factors 2^14 each
  auto gram = [&]() {
    NsGemm g = sym;
    g.a = g.b = at(q.xs);
    g.K = q.Lp;
    g.alpha = 1.f / 32768.f;
    g.d = A;
    return ns_go<NS_SYM>(g, s);
  };
  // d (2^13) = a I + b A + c A A of the matrix in src (2^13)
  auto poly = [&](const _Float16* src, _Float16* d) {
    NsGemm g = sym;
    g.a = g.b = g.c = src;
    g.K = q.Sp;
    g.alpha = NS_C * dn13;
    g.beta = NS_B;
    g.diag = NS_A * up13;
    g.d = d;
    return ns_go<NS_SYM>(g, s);
  };
  // d = x y of commuting symmetric matrices, times alpha
  auto mul = [&](const _Float16* x, const _Float16* y, float alpha, _Float16* d) {
    NsGemm g = sym;
    g.a = x;
    g.b = y;
    g.K = q.Sp;
    g.alpha = alpha;
    g.d = d;
    return ns_go<NS_SYM>(g, s);
  };
  // X (from buffer k, hi + lo when two) times f (2^logf) into the other buffer
  NsGemm prod{};
  prod.M = q.Lp;
  prod.N = prod.K = q.Sp;
  auto step = [&](int k, bool two, const _Float16* f, float alpha, bool keep_lo) {
    NsGemm g = prod;
    g.a = at(q.xh[k]);
    g.a2 = two ? at(q.xl[k]) : nullptr;
    g.b = f;
    g.alpha = alpha;
    g.d = at(q.xh[k ^ 1]);
    g.lo = keep_lo ? at(q.xl[k ^ 1]) : nullptr;
    g.dt = at(q.xs);
    return ns_go<NS_PROD>(g, s);
  };
#define NS_DO(call)                     \
  do {                                  \
    e = (call);                         \
    if (e != hipSuccess) return e;      \
  } while (0)
  // steps 0 and 1: P_0, T = P_0 A_0, A_1 = P_0 T, P_1, Q = P_1 P_0 (2^11), X_2 = Q X_0
  NS_DO(gram());
  NS_DO(poly(A, P));
  NS_DO(mul(P, A, dn13, T));
  NS_DO(mul(P, T, dn13, A));
  NS_DO(poly(A, T));
  NS_DO(mul(T, P, 1.f / 32768.f, Q));
  NS_DO(step(0, true, Q, 1.f / 2048.f, true));
  // step 2
  NS_DO(gram());
  NS_DO(poly(A, P));
  NS_DO(step(1, true, P, dn13, false));
  // step 3
  NS_DO(gram());
  NS_DO(poly(A, P));
  NS_DO(step(0, false, P, dn13, false));
  // step 4: X_5 (unscaled) in bf16
  NS_DO(gram());
  NS_DO(poly(A, P));
  NsGemm g = prod;
  g.a = at(q.xh[1]);
  g.b = P;
  g.alpha = dn13 / 16384.f;
  g.out = a.out;
  g.rows = a.rows;
  g.cols = a.cols;
  NS_DO(ns_go<NS_LAST>(g, s));
#undef NS_DO
  return hipSuccess;
}

}  // namespace bmoe
