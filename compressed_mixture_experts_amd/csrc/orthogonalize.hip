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
// which multiplies X from the left and adds no direction to its rows.  So up to
// X_2, where it matters most, X is kept as hi + lo in the products P X: hi fp16 and
// lo e4m3 (16 bits together, noise below X_3's own), whose products with P's e4m3
// copy run at twice fp16's rate.  With X in one fp16 term throughout, a gradient
// of rank S / 8 came out 2e-2 off, with this 3e-3; full-rank ones 1e-3.  lo in fp16
// brought rank one from 6.5e-3 to 5e-3 (lo's exponent from the data: 6e-3) and nothing
// else, and costs more (755 and 731 us at 2048 x 8192, 428 and 412 at 1300 x 6000).
//
// Long matrices take the first two steps together,
//     A_1 = P_0 A_0 P_0 = P_0 T,   Q = P_1 P_0,   X_2 = Q X_0
// (everything in A is a polynomial of A_0: the factors commute and stay
// symmetric), which saves X_1's rounding and its two products with L.
//
// A, P, T and Q round most where they are largest, on the diagonal, and there all
// alike when X's rows are equally long: 48 x 16384 normal entries came out 5e-3
// off.  So each keeps the ratio of its true diagonal to the stored one (fp32) and
// what it is multiplied into is multiplied by that ratio's row or column as well:
// exact for the diagonal's part, within fp16's rounding for the others' (now
// 1.7e-3, bf16's own).
//
// Symmetric results (A, T, P, Q) compute only the tiles on and above the
// diagonal and write each also mirrored.
//
// Layouts: every product is D[m][n] = sum_k A[m][k] B[n][k], both operands
// with k contiguous.  A = X X^T reads X as XS [S][L]; X' = P X, taken as
// X'^T = X^T P (P symmetric), reads X as XL [L][S].  A product's epilogue
// writes its tile both ways.  S and L are padded to multiples of 64 with zeros,
// which stay zero.
#include "step_ops.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace bmoe {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(1))) void ns_glob_t;
typedef __attribute__((address_space(3))) void ns_lds_t;
typedef const __attribute__((address_space(4))) int32_t ns_const_int_t;

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr int NS_SUMS = 512;        // partial sums of squares
constexpr int NS_K = 64;            // contraction step
constexpr int NS_SPLIT = 16;        // most workgroups that share a tile
constexpr int NS_SHARED = 512;      // most workgroups of a product that shares tiles

// The second terms of four v = hi + lo: (v - hi) f, f = 2^e, as four e4m3 bytes, off by
// 2^-4 of lo or by half of e4m3's last subnormal place, 2^-10 / f.  X's entries stay
// below 2^15, hi is off by at most 8 and e = NS_LO saturates nothing.  X_0, whose
// roundings grow most, takes e from its largest entry: in [2^m, 2^(m+1)) hi is off by
// at most 2^(m-11), 256 of e4m3's 448 at e = 19 - m.  m is 0 at least (||X_0|| is 2^14,
// of at most 2^28 entries) and 14 at most.  Without that, large matrices' small entries
// had their second terms among the subnormals: rank one came out 8.2e-3 off at 8192 x
// 8192 and 1.3e-2 at 16384 x 16384 (now 6.2e-3 and 7.0e-3; at 2048 x 8192 6.6e-3, now
// 6.0e-3).
constexpr int NS_LO = 5, NS_LO_MAX = 19;
__device__ __forceinline__ uint32_t ns_lo4(f32x4_t v, f16x4_t hi, float f) {
  int u = __builtin_amdgcn_cvt_pk_fp8_f32((v[0] - float(hi[0])) * f, (v[1] - float(hi[1])) * f, 0, false);
  u = __builtin_amdgcn_cvt_pk_fp8_f32((v[2] - float(hi[2])) * f, (v[3] - float(hi[3])) * f, u, true);
  return uint32_t(u);
}
// Eight fp16 values times f as e4m3 bytes.
__device__ __forceinline__ uint2 ns_fp8x8(uint4 h, float f) {
  const f16x8_t v = __builtin_bit_cast(f16x8_t, h);
  uint32_t u[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(float(v[4 * k]) * f, float(v[4 * k + 1]) * f, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(float(v[4 * k + 2]) * f, float(v[4 * k + 3]) * f, w, true);
    u[k] = uint32_t(w);
  }
  return make_uint2(u[0], u[1]);
}

// ------------------------------------------------------------------ momentum
// U's element from the gradient and the momentum M' (as stored).
__device__ __forceinline__ float ns_u(float g, float m1, float mu, int nesterov) {
  return nesterov ? fmaf(mu, m1, g) : m1;
}

// W consecutive elements from i on (W = 4: 16-byte, or for bf16 8-byte, loads).
template <bool BF, int W>
__device__ __forceinline__ void ns_load_grad(const void* g, size_t i, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = load1<BF ? ACT_BF16 : ACT_F32>(g, i);
  } else if constexpr (BF) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + i);
    v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
  } else {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}

// M' = mu M + G, the sum of U^2 (fp64 partial sums, one per workgroup) and the
// largest |U| (NS_SUMS floats behind the sums).
template <bool BF, int W>
__global__ __launch_bounds__(256) void ns_momentum_kernel(const void* grad, const float* mom, float* m_out, double* part,
                                                           size_t n, float mu, int nesterov) {
  __shared__ double red[4];
  __shared__ float top[4];
  double s = 0.0;
  float mx = 0.f;
  for (size_t i = (size_t(blockIdx.x) * 256 + threadIdx.x) * W; i < n; i += size_t(gridDim.x) * 256 * W) {
    float g[W], m[W];
    ns_load_grad<BF, W>(grad, i, g);
    if (mom) ns_load_grad<false, W>(mom, i, m);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float u = g[j];
      if (mom) {
        m[j] = fmaf(mu, m[j], g[j]);
        u = ns_u(g[j], m[j], mu, nesterov);
      }
      s = fma(double(u), double(u), s);
      mx = fmaxf(mx, fabsf(u));
    }
    if (mom) {
      if constexpr (W == 4) *reinterpret_cast<float4*>(m_out + i) = make_float4(m[0], m[1], m[2], m[3]);
      else m_out[i] = m[0];
    }
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    s += __shfl_xor(s, k);
    mx = fmaxf(mx, __shfl_xor(mx, k));
  }
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = s;
    top[threadIdx.x >> 6] = mx;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    part[blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
    reinterpret_cast<float*>(part + NS_SUMS)[blockIdx.x] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  }
}

// X_0 = U / ||U||_F times 2^14 as fp16 hi (+ lo): 64 x 64 tiles of the padded
// matrix, written in the caller's orientation from registers and transposed
// through LDS.
struct NsCast {
  _Float16* xs;             // [Sp][Lp]
  _Float16* xh;             // [Lp][Sp]
  uint8_t* xl;              // [Lp] rows of 2 Sp bytes, Sp of them second terms
  uint8_t* zero[3];         // rows of 2 Sp bytes to clear from Sp up to a multiple of 128: Lp of
                            // xl and of the other X's second terms, Sp of the factor's e4m3 copy
  int32_t* ticket;          // [NS_SHARED / 2], cleared
  int32_t* lo_exp;          // the exponents of the second terms of X_0 and of later X, written
};

template <bool BF, int W>
__global__ __launch_bounds__(256) void ns_cast_kernel(const void* grad, const float* mom, const double* part, int parts,
                                                       int rows, int cols, int Sp, int Lp, float mu, int nesterov, NsCast c) {
  __shared__ double red[4];
  __shared__ float top[4];
  __shared__ _Float16 th[64][68];
  __shared__ uint32_t tl[64][17];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) c.ticket[tid] = 0;
  static_assert(NS_SHARED / 2 == 256, "one ticket per thread");
  const bool tall = rows > cols;
  const int cp = tall ? Sp : Lp;  // padded columns
  const int tc = cp / 64;
  const int r0 = int(blockIdx.x / tc) * 64, c0 = int(blockIdx.x % tc) * 64;
  const int lc = 4 * (tid & 15);
  // four rows of four elements per thread, on their way while the norm is added up
  float g[4][4], m[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 16 * i + (tid >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) g[i][j] = m[i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j += W) {
      const size_t at = size_t(r) * cols + c0 + lc + j;
      if (r < rows && c0 + lc + j < cols) {
        float v[W];
        ns_load_grad<BF, W>(grad, at, v);
#pragma unroll
        for (int e = 0; e < W; ++e) g[i][j + e] = v[e];
        if (mom) {
          ns_load_grad<false, W>(mom, at, v);
#pragma unroll
          for (int e = 0; e < W; ++e) m[i][j + e] = v[e];
        }
      }
    }
  }
  double s = 0.0;
  float mx = 0.f;
  for (int p = tid; p < parts; p += 256) {
    s += part[p];
    mx = fmaxf(mx, reinterpret_cast<const float*>(part + NS_SUMS)[p]);
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    s += __shfl_xor(s, k);
    mx = fmaxf(mx, __shfl_xor(mx, k));
  }
  if ((tid & 63) == 0) {
    red[tid >> 6] = s;
    top[tid >> 6] = mx;
  }
  __syncthreads();
  const double norm = sqrt(((red[0] + red[1]) + red[2]) + red[3]);
  // NaN for a norm that is NaN or infinite, so that all of the result is NaN
  const double scale = norm > 0.0 ? (norm < __builtin_inf() ? 16384.0 / norm : __builtin_nan("")) : (norm == 0.0 ? 0.0 : norm);
  mx = float(double(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))) * scale);
  const int lo_exp = min(max(NS_LO_MAX + 127 - int(__float_as_uint(mx) >> 23 & 255u), NS_LO), NS_LO_MAX);
  const float lo_by = __uint_as_float(uint32_t(127 + lo_exp) << 23);
  if (blockIdx.x == 0 && tid < 2) c.lo_exp[tid] = tid == 0 ? lo_exp : NS_LO;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = 16 * i + (tid >> 4);
    f32x4_t v;
    f16x4_t hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = float(double(mom ? ns_u(g[i][j], m[i][j], mu, nesterov) : g[i][j]) * scale);
      hi[j] = _Float16(v[j]);
    }
    const uint32_t lo = ns_lo4(v, hi, lo_by);
    *reinterpret_cast<f16x4_t*>(&th[lr][lc]) = hi;
    tl[lr][tid & 15] = lo;
    const size_t at = size_t(r0 + lr) * cp + c0 + lc;
    if (tall) {
      *reinterpret_cast<f16x4_t*>(c.xh + at) = hi;
      *reinterpret_cast<uint32_t*>(c.xl + 2 * at - (c0 + lc)) = lo;
    } else {
      *reinterpret_cast<f16x4_t*>(c.xs + at) = hi;
    }
  }
  __syncthreads();
  const int rp = tall ? Lp : Sp;  // padded rows
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tcx = 16 * i + (tid >> 4);  // column of the tile, row of the transposed one
    f16x4_t hi;
    uint32_t lo = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = th[lc + j][tcx];
      lo |= (tl[lc + j][tcx >> 2] >> (8 * (tcx & 3)) & 0xFFu) << (8 * j);
    }
    const size_t at = size_t(c0 + tcx) * rp + r0 + lc;
    if (tall) {
      *reinterpret_cast<f16x4_t*>(c.xs + at) = hi;
    } else {
      *reinterpret_cast<f16x4_t*>(c.xh + at) = hi;
      *reinterpret_cast<uint32_t*>(c.xl + 2 * at - (r0 + lc)) = lo;
    }
  }
  const int l0 = tall ? r0 : c0, s0 = tall ? c0 : r0;
  if (Sp % 128 != 0 && s0 + 64 == Sp) {
    const int l = l0 + (tid >> 2);
    const size_t at = size_t(l) * 2 * Sp + Sp + 16 * (tid & 3);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < 2 || l < Sp) *reinterpret_cast<uint4*>(c.zero[k] + at) = make_uint4(0, 0, 0, 0);
  }
}

// ------------------------------------------------------------------ products
enum NsMode { NS_SYM = 0, NS_PROD = 1, NS_LAST = 2 };

struct NsGemm {
  const _Float16* a;        // [M][K]
  const _Float16* b;        // [N][K]
  const uint8_t* a8;        // NS_PROD: [M] rows of 2 K bytes, K of them the second term of a and 0
                            // up to a multiple of 128 (the offsets of a then hold here too); or null
  const uint8_t* b8;        // [N] such rows, b as e4m3
  int32_t exp8;             // sum of a b scales 2^(exp8 - e) times that of a8 b8, e the
  const int32_t* lo_exp;    // exponent of a8's second terms (NS_PROD)
  int32_t M, N, K;          // multiples of NS_K
  int32_t grid, tiles;      // workgroups; NS_SYM: tiles, else tiles of a row of tiles
  uint32_t by_tiles;        // floor(2^32 / tiles) + 1 (0 for 1): t / tiles = t by_tiles / 2^32
  float alpha;              // D = alpha sum (+ beta C + diag on the diagonal)
  const float* ra;          // [N] true over stored diagonal of a (NS_SYM; and of c) and
  const float* rb;          // of b, or null
  float* rd;                // NS_SYM: the same of d, written
  // NS_SYM: d [N][N]; c [N][N] or null
  int32_t band;             // tile rows of a band of tiles: 2^band
  int32_t split, per;       // workgroups that share a tile's depth, steps of each
  float* part;              // [tiles][split][tile] their sums when split > 1
  int32_t* ticket;          // [tiles] zero before and after the product
  const _Float16* c;
  float beta, diag;
  _Float16* d;              // NS_SYM; NS_PROD: D's hi [M][N]
  uint8_t* d8;              // NS_SYM: D times f8 as e4m3 (a later product's b8), or null
  float f8;
  uint8_t* lo;              // NS_PROD: D's second term (a later product's a8), or null
  _Float16* dt;             // NS_PROD: D's hi transposed [N][M]
  // NS_LAST: bf16, D cut to rows x cols and transposed back when wide
  uint16_t* out;
  int32_t rows, cols;       // of out
};

// One workgroup per TM x TN tile of D, KG groups of NW = WM x WN waves of one TM /
// WM x TN / WN part each (MFMA blocks of 16 x 16 x 32).  Both operand tiles of a 64-deep step
// come straight into LDS (16 bytes per lane), NBUF steps in a ring, so that
// NBUF - 1 steps are on their way while one is used.  Chunk ch (16 bytes) of row
// r sits at ch ^ (r % 8) of its row.
//
// A step is two 32-deep halves with a set of fragments in registers each: the
// reads of the next half are issued among the products of the current one, and
// the barrier that frees a ring place stands between the halves, where every
// wave has products of its own to do on both sides.
//
// With KG = 2 a step is 128 deep and a second group of as many waves takes its
// second half, in sums of its own that the first group's end up added to: two
// waves per SIMD where a tile leaves registers for four waves only, at the same
// LDS traffic (tiles of 96, X X^T of 2048 x 8192: 54 -> 50 us; tiles of 32 and 64
// gain nothing).
template <int MODE, int TM, int TN, int WM, int WN, int KG, int NBUF, bool EARLY>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void ns_gemm_kernel(
    const _Float16* left, const _Float16* right, int M, int N, int K, int grid, int tiles, uint32_t by_tiles, int log_band,
    int split, int per, NsGemm p) {
  constexpr int NW = WM * WN, NT = 64 * NW * KG;
  static_assert(KG == 1 || (KG == 2 && MODE == NS_SYM), "the second term's steps are one group's");
  constexpr int PM = TM / WM, PN = TN / WN, IM = PM / 16, IN = PN / 16;
  constexpr int STAGE = (TM + TN) * NS_K;        // halves of a ring place
  constexpr int LPW = (TM + TN) / 8 / NW;        // loads per wave and step
  constexpr int ST = TN + 4;                     // row stride of the staged tile (halves)
  static_assert((TM + TN) / 8 % NW == 0 && PM % 16 == 0 && PN % 16 == 0, "whole loads and blocks per wave");
  extern __shared__ __attribute__((aligned(16))) _Float16 sm[];  // [NBUF][KG][TM rows of A | TN rows of B][64]
  const int tid = threadIdx.x, lane = tid & 63, any = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = KG > 1 ? any / NW : 0, wave = KG > 1 ? any % NW : any;
  const int l16 = lane & 15, g = lane >> 4;  // row of a block, 16-byte chunk of its depth
  const int wm = wave % WM, wn = wave / WM;
  int tm, tn, tile = 0, share = 0;
  {
    // no division here: what happens before the first loads is on every product's
    // path (with two of them and arguments read where they are used 82.4 in place of
    // 78.9 us a call at 512 x 512, 219.8 of 212 at 1024 x 4096)
    int t = xcd_remap(blockIdx.x, grid);
    // t / tiles: right below 2^32 / tiles (at most 512 tiles to a row, at most
    // NS_SHARED workgroups that share tiles)
    auto quotient = [&]() { return by_tiles ? int(__umulhi(uint32_t(t), by_tiles)) : t; };
    if constexpr (MODE == NS_SYM) {
      // an XCD's workgroups take the same share of many tiles: its L2 then holds few
      // columns of the operand (118 -> 114 us a call at 256 x 8192, 357 -> 350 at
      // 1024 x 8192 against all shares of few tiles)
      if (split > 1) {
        share = quotient();
        t -= share * tiles;
      }
      tile = t;
      // tiles on and above the diagonal, by bands of 2^log_band tile rows, column by
      // column within a band: the tiles an XCD runs at a time form a block that
      // needs few row blocks of the operand in its L2
      static_assert(MODE != NS_SYM || TM == TN, "mirrored tiles are square");
      const int nt = (N + TN - 1) / TN, h = 1 << log_band;
      int r0 = 0;
      for (;; r0 += h) {
        const int hh = min(h, nt - r0), band = hh * (nt - r0) - hh * (hh - 1) / 2;
        if (t < band) break;
        t -= band;
      }
      // columns of 1, 2, .. h - 1 tiles, then of h
      int c = 0;
      const int few = h * (h - 1) / 2;
      if (t >= few) {
        t -= few;
        c = h - 1 + (t >> log_band);
        t &= h - 1;
      } else {
        while (t > c) t -= ++c;
      }
      tn = r0 + c;
      tm = r0 + t;
    } else {
      tm = quotient();
      tn = t - tm * tiles;
    }
  }
  const int m0 = tm * TM, n0 = tn * TN;
  const int nk1 = K / NS_K;
  // this workgroup's steps: k0 .. k0 + nk - 1
  int k0 = 0, nk = nk1;
  if constexpr (MODE == NS_SYM) {
    k0 = share * per;
    nk = min(per, nk1 - k0);
  }
  const int nkh = KG > 1 ? nk / KG : nk;  // whole steps in fp16, then those of the second term: 128 deep
  const bool two = MODE == NS_PROD && p.a8;
  if (two) nk += (nk1 + 1) / 2;
  // a load fills 8 rows of 64; a wave's loads are all of A or all of B.  Byte
  // offsets of this lane's pieces in it; 8-row groups past the matrix (M and N
  // are multiples of 8) read its last one and are not stored
  static_assert(TM / 8 % LPW == 0, "no wave loads both operands");
  const bool isb = wave * LPW >= TM / 8;
  // where the fragments take all registers (tiles of 256) the first row's part, the
  // same for the whole wave, stays in scalar ones (706 -> 699 us a call at 2048 x
  // 8192); elsewhere the additions at every load cost more (197 -> 199 at 1024 x 4096)
  constexpr bool SCALAR = TM == 256;
  const uint32_t lane_off = 2u * (__umul24(lane >> 3, K) + 8u * ((lane & 7) ^ (lane >> 3)));
  uint32_t off[LPW];
#pragma unroll
  for (int j = 0; j < LPW; ++j) {
    const int q = wave * LPW + j;
    off[j] = 2u * uint32_t(isb ? min(n0 + 8 * q - TM, N - 8) : min(m0 + 8 * q, M - 8)) * uint32_t(K);
    if (!SCALAR) off[j] += lane_off;
  }
  const char* base = reinterpret_cast<const char*>(isb ? right : left);
  const char* base8 = reinterpret_cast<const char*>(isb ? p.b8 : p.a8);
  // pieces j0 .. j1 - 1 of this wave's loads of step kt (past the last one: the last
  // one again, never read) into ring place `buf`; the first step of all waits for no
  // argument but the preloaded ones
  auto load = [&](int kt, int buf, int j0 = 0, int j1 = 64, bool head = false) {
    kt = min(KG > 1 ? kt * KG + kg : kt, nk - 1);
    const bool second = MODE == NS_PROD && !head && kt >= nkh;
    const char* src = second ? base8 : base;
    src += size_t(second ? kt - nkh : k0 + kt) * (2 * NS_K);
    _Float16* dst = sm + (buf * KG + kg) * STAGE + wave * LPW * 8 * NS_K;
#pragma unroll
    for (int j = 0; j < LPW; ++j)
      if (j >= j0 && j < j1)
        __builtin_amdgcn_global_load_lds((ns_glob_t*)(src + off[j] + (SCALAR ? lane_off : 0u)), (ns_lds_t*)(dst + 8 * j * NS_K), 16, 0, 0);
  };
  // the ratios of this lane's rows and columns (1 past the matrix), read behind
  // the first steps' loads: ahead of them or in the epilogue their latency shows
  float ram[IM], rbm[IM];
  f32x4_t ran[IN], rbn[IN];
  auto ratios = [&](const float* r, float (&rm)[IM], f32x4_t (&rn)[IN]) {
#pragma unroll
    for (int j = 0; j < IM; ++j) {
      const int m = m0 + PM * wm + 16 * j + l16;
      rm[j] = MODE == NS_SYM && r && m < M ? r[m] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      const int n = n0 + PN * wn + 16 * i + 4 * g;
      rn[i] = f32x4_t{1.f, 1.f, 1.f, 1.f};
      if (r && n < N) rn[i] = *reinterpret_cast<const f32x4_t*>(r + n);
    }
  };
  f32x4_t acc[IN][IM];
#pragma unroll
  for (int i = 0; i < IN; ++i)
#pragma unroll
    for (int j = 0; j < IM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  f16x8_t fa[2][IM], fb[2][IN];
  auto read = [&](int buf, int h, f16x8_t (&a)[IM], f16x8_t (&b)[IN]) {
    const int ch = 8 * ((4 * h + g) ^ (l16 & 7));
    const _Float16* A = sm + (buf * KG + kg) * STAGE + (PM * wm + l16) * NS_K + ch;
    const _Float16* B = sm + (buf * KG + kg) * STAGE + (TM + PN * wn + l16) * NS_K + ch;
#pragma unroll
    for (int j = 0; j < IM; ++j) a[j] = *reinterpret_cast<const f16x8_t*>(A + 16 * j * NS_K);
#pragma unroll
    for (int i = 0; i < IN; ++i) b[i] = *reinterpret_cast<const f16x8_t*>(B + 16 * i * NS_K);
  };
  auto mul = [&](const f16x8_t (&a)[IM], const f16x8_t (&b)[IN]) {
#pragma unroll
    for (int i = 0; i < IN; ++i)
#pragma unroll
      for (int j = 0; j < IM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[i], a[j], acc[i][j], 0, 0, 0);
  };
  // order of a region with NL loads: a read behind each of the first products, the
  // loads evenly among the others; nothing crosses the region's end
  auto spread = [&](auto loads) {
    constexpr int NL = decltype(loads)::value, REST = IM * IN - IM - IN;
    constexpr int GAP = NL > 0 && REST / std::max(NL, 1) > 0 ? REST / std::max(NL, 1) : 1;
#pragma unroll
    for (int m = 0; m < IM + IN; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
#pragma unroll
    for (int m = 0; m < NL; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, GAP, 0);
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, IM * IN, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // this wave's reads are done and its loads of all but the newest `left` steps
  // have arrived; then the same of every wave
  auto arrive = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NBUF - 2) * LPW) : "memory");
  };
#pragma unroll
  for (int b = 0; b < NBUF - 1; ++b) load(b, b, 0, 64, b == 0);
  // a scalar read while they arrive (behind arrive() a vector one, which waits for all
  // loads before it: 0.4 us)
  int scale8 = 0;
  if constexpr (MODE == NS_PROD) scale8 = 127 + p.exp8 - *reinterpret_cast<ns_const_int_t*>(reinterpret_cast<uintptr_t>(p.lo_exp));
  arrive();
  load(NBUF - 1, NBUF - 1);
  if constexpr (MODE == NS_SYM) ratios(p.ra, ram, ran);
  ratios(p.rb, rbm, rbn);
  if constexpr (MODE == NS_SYM)
    asm volatile("" ::"s"(p.d), "s"(p.c), "s"(p.d8), "s"(p.f8), "s"(p.rd), "s"(p.alpha), "s"(p.beta), "s"(p.diag));
  read(0, 0, fa[0], fb[0]);
  int buf = 0;
  for (int kt = 0; kt < nkh; ++kt) {
    const int next = buf + 1 == NBUF ? 0 : buf + 1;
    read(buf, 1, fa[1], fb[1]);
    mul(fa[0], fb[0]);
    spread(std::integral_constant<int, 0>{});
    arrive();
    // the loads among the products behind the reads: a burst of them before the
    // reads holds its wave up (tile 256: 131 -> 123 us for X = Q X_0 at 2048 x
    // 8192 with an fp16 second term); with few products to a step (EARLY) they go
    // first, to arrive sooner
    if constexpr (EARLY) load(kt + NBUF, buf);
    read(next, 0, fa[0], fb[0]);
    if constexpr (!EARLY) load(kt + NBUF, buf);
    mul(fa[1], fb[1]);
    spread(std::integral_constant<int, LPW>{});
    buf = next;
  }
  if (KG > 1 && nkh * KG + kg < nk) {  // an odd depth's last piece is the first group's
    read(buf, 1, fa[1], fb[1]);
    mul(fa[0], fb[0]);
    mul(fa[1], fb[1]);
  }
  if constexpr (MODE == NS_PROD) {
    // the second term's steps: 128 bytes of a row are 128 deep, and lane group g takes
    // the chunks g and 4 + g of both operands.  The fragments are as large as both
    // halves' above, so there is one set: the lower blocks' rows are read among the
    // upper ones' products and the other way round, each column block's as soon as
    // its last product is issued.
    if (two) {
      constexpr int H = IM / 2, R = IM - H;
      i32x8_t ea[IM], eb[IN];
      auto read8 = [&](int buf, int row) {
        const _Float16* q = sm + buf * STAGE + (row + l16) * NS_K;
        const int ch = 8 * (g ^ (l16 & 7));
        const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(q + ch), hi = *reinterpret_cast<const i32x4_t*>(q + (ch ^ 32));
        return i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      };
      auto mul8 = [&](int i, int j) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(eb[i], ea[j], acc[i][j], 0, 0, 0, scale8, 0, 127);
      };
#pragma unroll
      for (int i = 0; i < IN; ++i) eb[i] = read8(buf, TM + PN * wn + 16 * i);
#pragma unroll
      for (int j = 0; j < H; ++j) ea[j] = read8(buf, PM * wm + 16 * j);
      for (int kt = nkh; kt < nk; ++kt) {
        const int next = buf + 1 == NBUF ? 0 : buf + 1;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
#pragma unroll
          for (int j = H + i * R / IN; j < H + (i + 1) * R / IN; ++j) ea[j] = read8(buf, PM * wm + 16 * j);
#pragma unroll
          for (int j = 0; j < H; ++j) mul8(i, j);
          __builtin_amdgcn_sched_barrier(0);
        }
        arrive();
        if constexpr (EARLY) load(kt + NBUF, buf);
#pragma unroll
        for (int i = 0; i < IN; ++i) {
#pragma unroll
          for (int j = H; j < IM; ++j) mul8(i, j);
          eb[i] = read8(next, TM + PN * wn + 16 * i);
#pragma unroll
          for (int j = i * H / IN; j < (i + 1) * H / IN; ++j) ea[j] = read8(next, PM * wm + 16 * j);
          if constexpr (!EARLY) load(kt + NBUF, buf, i * LPW / IN, (i + 1) * LPW / IN);
          __builtin_amdgcn_sched_barrier(0);
        }
        buf = next;
      }
    }
  }
  // loads past the last step may still be writing to the ring
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const bool first = KG == 1 || kg == 0;  // whose sums are the tile's
  if constexpr (KG > 1) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(sm) + wave * 64 + lane;
    if (!first) {
#pragma unroll
      for (int i = 0; i < IN; ++i)
#pragma unroll
        for (int j = 0; j < IM; ++j) q[(i * IM + j) * 64 * NW] = acc[i][j];
    }
    __syncthreads();
    if (first) {
#pragma unroll
      for (int i = 0; i < IN; ++i)
#pragma unroll
        for (int j = 0; j < IM; ++j) acc[i][j] += q[(i * IM + j) * 64 * NW];
    }
    __syncthreads();
  }

  if constexpr (MODE == NS_SYM) {
    if (split > 1) {
      // the sums go to memory; the workgroup that comes last to a tile adds all of
      // them in the order of the depth and goes on alone.  Nobody waits.  The
      // XCDs' L2s do not see each other's writes, so the sums are stored past them
      // and read past them (agent scope); a fence that writes the whole L2 back
      // instead cost 54 us a product.
      constexpr int PAIRS = IM * IN * 2, NS = 64 * NW;  // pairs of sums, threads that hold them
      typedef float f32x2_t __attribute__((ext_vector_type(2)));
      unsigned long long* own =
          reinterpret_cast<unsigned long long*>(p.part) + (size_t(tile) * split + share) * PAIRS * NS + tid;
      if (first) {
#pragma unroll
        for (int i = 0; i < IN; ++i)
#pragma unroll
          for (int j = 0; j < IM; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const f32x2_t v = {acc[i][j][2 * h], acc[i][j][2 * h + 1]};
              __hip_atomic_store(own + ((i * IM + j) * 2 + h) * NS, __builtin_bit_cast(unsigned long long, v),
                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // they are there before the ticket says so
      __syncthreads();
      int* last = reinterpret_cast<int*>(sm);
      if (tid == 0) {
        *last = __hip_atomic_fetch_add(p.ticket + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == split - 1;
        if (*last) p.ticket[tile] = 0;
      }
      __syncthreads();
      if (!*last) return;
      const unsigned long long* all =
          reinterpret_cast<const unsigned long long*>(p.part) + size_t(tile) * split * PAIRS * NS + tid;
      constexpr int G = 32 / PAIRS > 0 ? 32 / PAIRS : 1;  // shares read at a time
      for (int q0 = 0; first && q0 < split; q0 += G) {
        unsigned long long v[G][PAIRS];
#pragma unroll
        for (int q = 0; q < G; ++q)
          if (q0 + q < split)
#pragma unroll
            for (int k = 0; k < PAIRS; ++k)
              v[q][k] = __hip_atomic_load(all + (size_t(q0 + q) * PAIRS + k) * NS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int q = 0; q < G; ++q)
          if (q0 + q < split)
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) {
              const f32x2_t w = __builtin_bit_cast(f32x2_t, v[q][k]);
              f32x4_t& a = acc[k / 2 / IM][k / 2 % IM];
              a[2 * (k % 2)] = q0 + q == 0 ? w.x : a[2 * (k % 2)] + w.x;
              a[2 * (k % 2) + 1] = q0 + q == 0 ? w.y : a[2 * (k % 2) + 1] + w.y;
            }
      }
      __syncthreads();  // *last is read before the tile is staged over it
    }
  }

  // acc[i][j][r] = D[m0 + PM wm + 16 j + l16][n0 + PN wn + 16 i + 4 g + r]
  _Float16* st = sm;  // [TM][ST]
  // f(four sums of consecutive columns, row, first column, blocks) to the staged tile
  auto staged = [&](auto&& f) {
    if (first) {
#pragma unroll
      for (int j = 0; j < IM; ++j)
#pragma unroll
        for (int i = 0; i < IN; ++i) {
          const int m = PM * wm + 16 * j + l16, n = PN * wn + 16 * i + 4 * g;
          *reinterpret_cast<f16x4_t*>(st + m * ST + n) = f(acc[i][j], m, n, i, j);
        }
    }
    __syncthreads();
  };
  auto row8 = [&](int r, int c) {
    const uint2 u = *reinterpret_cast<const uint2*>(st + r * ST + c);
    const uint2 v = *reinterpret_cast<const uint2*>(st + r * ST + c + 4);
    return make_uint4(u.x, u.y, v.x, v.y);
  };
  // column c of the staged tile, rows r .. r + 7
  auto column8 = [&](int c, int r) {
    f16x8_t v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = st[(r + e) * ST + c];
    return __builtin_bit_cast(uint4, v);
  };
  // f(row, first column) for every 16-byte piece of the tile inside M x N, and
  // f(column, first row) for those of the transposed tile, RL of them (up to
  // 192 contiguous bytes) per group of lanes
  constexpr int PIECES = TM * TN / 8, RL = TM % 64 == 0 ? 8 : TM / 8;
  auto pieces = [&](auto&& f) {
#pragma unroll 4
    for (int q = 0; q < (PIECES + NT - 1) / NT; ++q) {
      const int k = tid + NT * q;
      if (PIECES % NT != 0 && k >= PIECES) break;
      const int r = k / (TN / 8), c = 8 * (k % (TN / 8));
      if (m0 + r < M && n0 + c < N) f(r, c);
    }
  };
  auto tpieces = [&](auto&& f) {
#pragma unroll 4
    for (int q = 0; q < (PIECES + NT - 1) / NT; ++q) {
      const int k = tid + NT * q;
      if (PIECES % NT != 0 && k >= PIECES) break;
      const int c = k / RL % TN, r = 8 * (k % RL + RL * (k / RL / TN));
      if (m0 + r < M && n0 + c < N) f(c, r);
    }
  };
  auto direct = [&](_Float16* dst, size_t ld) {
    pieces([&](int r, int c) { *reinterpret_cast<uint4*>(dst + size_t(r) * ld + c) = row8(r, c); });
  };
  auto transposed = [&](_Float16* dst, size_t ld) {
    tpieces([&](int c, int r) { *reinterpret_cast<uint4*>(dst + size_t(c) * ld + r) = column8(c, r); });
  };
  if constexpr (MODE == NS_SYM) {
    float dv[IM], ds[IM];  // this lane's elements of the diagonal, true and stored
#pragma unroll
    for (int j = 0; j < IM; ++j) dv[j] = ds[j] = 1.f;
    staged([&](f32x4_t a, int m, int n, int i, int j) {
      m += m0;
      n += n0;
      f16x4_t cv = {0, 0, 0, 0}, o;
      if (p.c && m < M && n < N) cv = *reinterpret_cast<const f16x4_t*>(p.c + size_t(m) * N + n);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sa = 0.5f * (ram[j] + ran[i][r]), sb = 0.5f * (rbm[j] + rbn[i][r]);
        float v = sa * fmaf(p.alpha * sb, a[r], p.beta * float(cv[r]));
        const bool on = m == n + r;
        v += on ? p.diag : 0.f;
        o[r] = _Float16(v);
        dv[j] = on ? v : dv[j];
        ds[j] = on ? float(o[r]) : ds[j];
      }
      return o;
    });
    // eight values to d, and to its e4m3 copy
    auto put = [&](int row, int col, uint4 u) {
      *reinterpret_cast<uint4*>(p.d + size_t(row) * N + col) = u;
      if (p.d8) *reinterpret_cast<uint2*>(p.d8 + 2 * size_t(row) * N + col) = ns_fp8x8(u, p.f8);
    };
    pieces([&](int r, int c) { put(m0 + r, n0 + c, row8(r, c)); });
    if (tm != tn) tpieces([&](int c, int r) { put(n0 + c, m0 + r, column8(c, r)); });
    // the ratios, 1 where the stored value is subnormal and its rounding coarse; at
    // the end, where no barrier waits for the stores
    if (tm == tn && first) {
#pragma unroll
      for (int j = 0; j < IM; ++j) {
        const int ml = PM * wm + 16 * j + l16, nl = ml - PN * wn;  // its column in this wave's part
        if (nl >= 0 && nl < PN && (nl >> 2 & 3) == g && m0 + ml < M)
          p.rd[m0 + ml] = fabsf(ds[j]) >= 6.1035156e-5f ? dv[j] / ds[j] : 1.f;
      }
    }
  } else if constexpr (MODE == NS_PROD) {
    staged([&](f32x4_t a, int, int, int i, int) {
      a *= p.alpha * rbn[i];
      f16x4_t o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = _Float16(a[r]);
      return o;
    });
    direct(p.d + size_t(m0) * N + n0, N);
    transposed(p.dt + size_t(n0) * M + m0, M);
    if (p.lo) {
      constexpr int SW = TN / 4 + 1;  // row stride of the staged bytes (words)
      uint32_t* s8 = reinterpret_cast<uint32_t*>(sm);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < IM; ++j)
#pragma unroll
        for (int i = 0; i < IN; ++i) {
          const f32x4_t v = acc[i][j] * (p.alpha * rbn[i]);
          f16x4_t hi;
#pragma unroll
          for (int r = 0; r < 4; ++r) hi[r] = _Float16(v[r]);
          s8[(PM * wm + 16 * j + l16) * SW + (PN * wn + 16 * i) / 4 + g] = ns_lo4(v, hi, float(1 << NS_LO));
        }
      __syncthreads();
      pieces([&](int r, int c) {
        const uint32_t* q = s8 + r * SW + c / 4;
        *reinterpret_cast<uint2*>(p.lo + 2 * size_t(m0 + r) * N + n0 + c) = make_uint2(q[0], q[1]);
      });
    }
  } else {
    staged([&](f32x4_t a, int, int, int i, int) {
      a *= p.alpha * rbn[i];
      uint2 o;
      o.x = pack_bf16x2(a[0], a[1]);
      o.y = pack_bf16x2(a[2], a[3]);
      return __builtin_bit_cast(f16x4_t, o);
    });
    const bool vec = p.cols % 8 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    // eight columns of out from row r, column c on
    auto put = [&](int r, int c, uint4 u) {
      if (r >= p.rows || c >= p.cols) return;
      uint16_t* dst = p.out + size_t(r) * p.cols + c;
      if (vec) {
        *reinterpret_cast<uint4*>(dst) = u;
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.cols) dst[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
      }
    };
    if (p.rows > p.cols) pieces([&](int r, int c) { put(m0 + r, n0 + c, row8(r, c)); });
    else tpieces([&](int c, int r) { put(n0 + c, m0 + r, column8(c, r)); });
  }
}

// ------------------------------------------------------------------ host
namespace {

// Padded side: whole contraction steps.
int ns_pad(int n) { return (n + NS_K - 1) / NS_K * NS_K; }

// Tiles of side t in a product's result.
template <int MODE>
int ns_tiles(const NsGemm& p, int t) {
  const int nm = (p.M + t - 1) / t, nn = (p.N + t - 1) / t;
  return MODE == NS_SYM ? nn * (nn + 1) / 2 : nm * nn;
}

// A tile side: microseconds of a step of 64 by a lone workgroup of a CU (latency
// and the CU's own limits), and by each of two that share one (0: one fills it).
struct NsSide {
  int side;
  double one, two;
};

struct NsTile {
  int side, split;
};

// Time of a product in tiles of a side, `split` workgroups to a tile, in
// microseconds.  A step takes what the CU does, or all workgroups together: 256 t
// bytes each from L2 into LDS and 128 t^2 operations at 1.15 PFLOP/s.  Symmetric
// products get 23 TB/s from L2 (19 where the operand is beyond the L2s, 16 where
// shares read different parts of the depth), two workgroups of a CU take longer where
// the operand is beyond the L2s and where some CUs get a third, and adding a tile's
// shares up takes 1.4 us and more with its area and their number.  General ones get
// 20 TB/s in small tiles and 14 in large ones, whole rounds of workgroups, and the
// epilogue of a large tile counts.  The constants are fitted to whole calls with
// every side and split forced: X X^T of 23 sizes from 192 x 8192 to 1800 x 8192, the
// products of side 320 to 2560, those with X of 35 sizes from 64 x 2000 to 2048 x 8192.
template <int MODE>
double ns_time(const NsGemm& p, NsSide s, int split) {
  const int t = s.side, nk = p.K / NS_K, steps = p.a8 ? nk + (nk + 1) / 2 : nk, n = ns_tiles<MODE>(p, t) * split;
  const int cus = NS_SHARED / 2;
  double cu = s.one, rate, once = 0.0;
  if (s.two == 0) cu = s.one * ((n + cus - 1) / cus);
  if constexpr (MODE == NS_SYM) {
    const bool far = 2.0 * p.N * p.K >= 8 << 20;
    if (s.two > 0 && n > cus) cu = s.two * (far ? 1.28 : 1.0) * (n > 2 * cus ? 1.25 : 1.0);
    rate = split > 1 ? 16e6 : far ? 19e6 : 23e6;
    if (split > 1) once = 1.4 + (t > 64 ? 1.9 * t * t / 4096 : t > 32 ? 1.0 : 0.42) * (0.8 + 0.4 * split);
  } else {
    if (s.two > 0 && n > cus) cu = s.two * ((n + 2 * cus - 1) / (2 * cus));
    rate = t > 64 ? 14e6 : 20e6;
    once = t > 128 ? 3.4 : t > 64 ? 1.4 : t > 32 ? 0.5 : 0.0;
  }
  const double step = std::max({cu, double(n) * t * 256 / rate, double(n) * t * t * 128 / 1.15e9});
  return (steps + split - 1) / split * step + once;
}

template <int MODE>
NsTile ns_pick(const NsGemm& p) {
  NsTile best{0, 1};
  double least = 0;
  auto look = [&](NsSide s) {
    // as many workgroups as run at a time: two per CU up to tiles of 64
    const int most = (s.two > 0 ? NS_SHARED : NS_SHARED / 2) / std::max(1, ns_tiles<MODE>(p, s.side)), steps = p.K / NS_K;
    for (int split = 1; split == 1 || (MODE == NS_SYM && split <= std::min(most, NS_SPLIT)); ++split) {
      // whole shares only
      if (split > 1 && (split - 1) * ((steps + split - 1) / split) >= steps) continue;
      const double time = ns_time<MODE>(p, s, split);
      if (!best.side || time < least) {
        best = NsTile{s.side, split};
        least = time;
      }
    }
  };
  look({32, 0.14, 0.17});
  look({64, 0.205, 0.29});
  if (MODE == NS_SYM) look({96, 0.32, 0});
  look({128, 0.41, 0});
  if (MODE != NS_SYM) look({256, 1.2, 0});
  return best;
}

struct NsPlan {
  size_t part, xs, xh[2], xl[2], m[4], r[4], m8, shares, ticket, lo_exp, total;
  int S, L, Sp, Lp;
  NsTile gram, square;      // tiles of X X^T and of the products of side S
};

NsPlan ns_plan(int rows, int cols) {
  NsPlan q{};
  q.S = rows < cols ? rows : cols;
  q.L = rows < cols ? cols : rows;
  q.Sp = ns_pad(q.S);
  q.Lp = ns_pad(q.L);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t x = size_t(q.Sp) * q.Lp * 2, s = size_t(q.Sp) * q.Sp * 2;
  q.part = take(NS_SUMS * 8 + NS_SUMS * 4);
  q.xs = take(x);
  for (int k = 0; k < 2; ++k) {
    q.xh[k] = take(x);
    q.xl[k] = take(x);
  }
  for (int k = 0; k < 4; ++k) {
    q.m[k] = take(s);
    q.r[k] = take(size_t(q.Sp) * 4);
  }
  q.m8 = take(s);
  size_t shares = 0;
  auto pick = [&](int depth) {
    NsGemm g{};
    g.M = g.N = q.Sp;
    g.K = depth;
    const NsTile t = ns_pick<NS_SYM>(g);
    if (t.split > 1) shares = std::max(shares, size_t(ns_tiles<NS_SYM>(g, t.side)) * t.split * t.side * t.side * 4);
    return t;
  };
  q.gram = pick(q.Lp);
  q.square = pick(q.Sp);
  q.shares = take(shares);
  q.ticket = take(NS_SHARED / 2 * 4);
  q.lo_exp = take(8);
  q.total = o;
  return q;
}

template <int MODE, int T, int WM, int WN, int KG, int NBUF>
hipError_t ns_tile(NsGemm p, int split, hipStream_t s) {
  constexpr size_t ring = size_t(NBUF) * KG * 2 * T * NS_K * 2, stage = size_t(T) * (T + 4) * 2;
  constexpr size_t lds = ring > stage ? ring : stage;
  const auto kernel = ns_gemm_kernel<MODE, T, T, WM, WN, KG, NBUF, T <= 64>;
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  const int tiles = ns_tiles<MODE>(p, T);
  p.grid = tiles * split;
  p.tiles = MODE == NS_SYM ? tiles : (p.N + T - 1) / T;
  p.by_tiles = p.tiles > 1 ? uint32_t((uint64_t(1) << 32) / uint32_t(p.tiles)) + 1 : 0;
  p.split = split;
  p.per = (p.K / NS_K + split - 1) / split;
  // about as high as the block of tiles of one of the eight XCDs is wide
  p.band = std::max(0, int(std::lround(std::log2(tiles / 8.0) / 2)));
  hipLaunchKernelGGL(kernel, dim3(unsigned(tiles * split)), dim3(64 * WM * WN * KG), lds, s, p.a, p.b, p.M, p.N, p.K, p.grid, p.tiles,
                     p.by_tiles, p.band, p.split, p.per, p);
  return hipGetLastError();
}

template <int MODE>
hipError_t ns_go(const NsGemm& p, NsTile t, hipStream_t s) {
  if (t.side == 32) return ns_tile<MODE, 32, 2, 2, 1, 4>(p, t.split, s);
  if (t.side == 64) return ns_tile<MODE, 64, 2, 2, 1, 4>(p, t.split, s);
  if constexpr (MODE == NS_SYM) {
    if (t.side == 96) return ns_tile<MODE, 96, 2, 2, 2, 3>(p, t.split, s);
  } else {
    if (t.side == 256) return ns_tile<MODE, 256, 2, 4, 1, 2>(p, t.split, s);
  }
  return ns_tile<MODE, 128, 2, 4, 1, 3>(p, t.split, s);
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
  // four elements at a time where whole rows are aligned to it
  const bool v4 = a.cols % 4 == 0 && al(a.grad, a.grad_bf16 ? 8 : 16) && al(a.m, 16) && al(a.m_out, 16);
  const size_t nb = ((v4 ? n / 4 : n) + 255) / 256;
  const int blocks = int(nb < NS_SUMS ? nb : NS_SUMS);
  auto bytes = [&](size_t off) { return reinterpret_cast<uint8_t*>(ws + off); };
  int32_t* ticket = reinterpret_cast<int32_t*>(ws + q.ticket);
  int32_t* lo_exp = reinterpret_cast<int32_t*>(ws + q.lo_exp);
  const NsCast c{at(q.xs), at(q.xh[0]), bytes(q.xl[0]), {bytes(q.xl[0]), bytes(q.xl[1]), bytes(q.m8)}, ticket, lo_exp};
  const unsigned tiles = unsigned((q.Sp / 64) * (q.Lp / 64));
  hipError_t e = hipSuccess;
  auto head = [&](auto bf, auto w) {
    hipLaunchKernelGGL((ns_momentum_kernel<decltype(bf)::value, decltype(w)::value>), dim3(unsigned(blocks)), dim3(256), 0,
                       s, a.grad, a.m, a.m_out, part, n, a.mu, a.nesterov);
    e = hipGetLastError();
    if (e != hipSuccess) return;
    hipLaunchKernelGGL((ns_cast_kernel<decltype(bf)::value, decltype(w)::value>), dim3(tiles), dim3(256), 0, s, a.grad,
                       a.m ? a.m_out : nullptr, part, blocks, a.rows, a.cols, q.Sp, q.Lp, a.mu, a.nesterov, c);
    e = hipGetLastError();
  };
  using four = std::integral_constant<int, 4>;
  using single = std::integral_constant<int, 1>;
  if (a.grad_bf16) v4 ? head(std::true_type{}, four{}) : head(std::true_type{}, single{});
  else v4 ? head(std::false_type{}, four{}) : head(std::false_type{}, single{});
  if (e != hipSuccess) return e;

  constexpr float up13 = 8192.f, dn13 = 1.f / 8192.f;
  // a symmetric matrix and the ratios of its true diagonal to the stored one; with
  // an exponent it is the factor of a two-term X, whose second term takes it as
  // e4m3 times 2^-e8 (P at most 3.45 times 2^13 and Q at most 11.9 times 2^11: 221
  // and 381 of e4m3's 448)
  struct Sym {
    _Float16* m;
    float* r;
    int e8 = 0;
  };
  auto matrix = [&](int k, int e8 = 0) { return Sym{at(q.m[k]), reinterpret_cast<float*>(ws + q.r[k]), e8}; };
  const Sym A = matrix(0), T = matrix(1), P = matrix(2), P2 = matrix(2, 7), Q = matrix(3, 6);
  NsGemm sym{};
  sym.M = sym.N = q.Sp;
  sym.part = reinterpret_cast<float*>(ws + q.shares);
  sym.ticket = ticket;
  // A (2^13) = XS XS^T, factors 2^14 each
  auto gram = [&]() {
    NsGemm g = sym;
    g.a = g.b = at(q.xs);
    g.K = q.Lp;
    g.alpha = 1.f / 32768.f;
    g.d = A.m;
    g.rd = A.r;
    return ns_go<NS_SYM>(g, q.gram, s);
  };
  // d (2^13) = a I + b x + c x x (x 2^13)
  auto poly = [&](Sym x, Sym d) {
    NsGemm g = sym;
    g.a = g.b = g.c = x.m;
    g.ra = g.rb = x.r;
    g.K = q.Sp;
    g.alpha = NS_C * dn13;
    g.beta = NS_B;
    g.diag = NS_A * up13;
    g.d = d.m;
    g.rd = d.r;
    g.d8 = d.e8 ? bytes(q.m8) : nullptr;
    g.f8 = std::ldexp(1.f, -d.e8);
    return ns_go<NS_SYM>(g, q.square, s);
  };
  // d = x y of commuting symmetric matrices, times alpha
  auto mul = [&](Sym x, Sym y, float alpha, Sym d) {
    NsGemm g = sym;
    g.a = x.m;
    g.b = y.m;
    g.ra = x.r;
    g.rb = y.r;
    g.K = q.Sp;
    g.alpha = alpha;
    g.d = d.m;
    g.rd = d.r;
    g.d8 = d.e8 ? bytes(q.m8) : nullptr;
    g.f8 = std::ldexp(1.f, -d.e8);
    return ns_go<NS_SYM>(g, q.square, s);
  };
  // X (in buffer k; hi + lo where f has an e4m3 copy) times f into the other buffer
  NsGemm prod{};
  prod.M = q.Lp;
  prod.N = prod.K = q.Sp;
  prod.lo_exp = lo_exp;
  int k = 0;
  auto next = [&](Sym f, float alpha, bool keep_lo) {
    NsGemm g = prod;
    g.a = at(q.xh[k]);
    g.b = f.m;
    if (f.e8) {
      g.a8 = bytes(q.xl[k]);
      g.b8 = bytes(q.m8);
      g.exp8 = f.e8;
    }
    g.rb = f.r;
    g.alpha = alpha;
    k ^= 1;
    g.d = at(q.xh[k]);
    g.lo = keep_lo ? bytes(q.xl[k]) : nullptr;
    g.dt = at(q.xs);
    prod.lo_exp = lo_exp + 1;
    return ns_go<NS_PROD>(g, ns_pick<NS_PROD>(g), s);
  };
#define NS_DO(call)                     \
  do {                                  \
    e = (call);                         \
    if (e != hipSuccess) return e;      \
  } while (0)
  if (4 * q.L <= 5 * q.S) {
    // steps 0 and 1 one by one, from two terms: a product less than together (us a
    // call, one by one and together: 76 and 79 at 512 x 512, 133 and 137 at 1024 x
    // 1024, 348 and 352 at 2048 x 2048; both 152 at 1024 x 1280; 176 and 171 at 1024 x
    // 2048, 223 and 212 at 1024 x 4096)
    for (int i = 0; i < 2; ++i) {
      NS_DO(gram());
      NS_DO(poly(A, P2));
      NS_DO(next(P2, dn13, true));
    }
  } else {
    // together: P_0, T = P_0 A_0, A_1 = P_0 T, P_1, Q = P_1 P_0 (2^11), X_2 = Q X_0,
    // three products of side S for two with L
    NS_DO(gram());
    NS_DO(poly(A, P));
    NS_DO(mul(P, A, dn13, T));
    NS_DO(mul(P, T, dn13, A));
    NS_DO(poly(A, T));
    NS_DO(mul(T, P, 1.f / 32768.f, Q));
    NS_DO(next(Q, 1.f / 2048.f, true));
  }
  // step 2 from two terms, step 3 from one
  for (const Sym& f : {P2, P}) {
    NS_DO(gram());
    NS_DO(poly(A, f));
    NS_DO(next(f, dn13, false));
  }
  // step 4: X_5 (unscaled) in bf16
  NS_DO(gram());
  NS_DO(poly(A, P));
  NsGemm g = prod;
  g.a = at(q.xh[k]);
  g.b = P.m;
  g.rb = P.r;
  g.alpha = dn13 / 16384.f;
  g.out = a.out;
  g.rows = a.rows;
  g.cols = a.cols;
  NS_DO(ns_go<NS_LAST>(g, ns_pick<NS_LAST>(g), s));
#undef NS_DO
  return hipSuccess;
}

}  // namespace bmoe
