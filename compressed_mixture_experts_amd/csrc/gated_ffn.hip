// Dense gated feed-forward block (include/bmoe_ffn.h).
//
// Six matrix products over bf16 with fp32 sums, all by one kernel template:
//     forward   g | u = x Wg^T | x Wu^T -> h        y = h Wd^T
//     backward  dh = dy Wd -> dg | du               dx = [dg du] [Wg; Wu]
//               [dWg; dWu] = [dg du]^T x            dWd = dy^T h
// An operand has the contraction contiguous (x, h, dy and the weights of the forward) or
// its other side (the weights of the backward's first two, everything in the last two).
// Operand tiles of 64-deep or 32-deep steps come straight into LDS (16 bytes per lane) in a ring of
// steps, in the layout they have in memory; those of the second kind are turned on the
// way from LDS to registers (ds_read_b64_tr_b16), so no transposed copy of anything is
// written.
#include "butterfly_impl.hpp"
#include "row_ops.hpp"
#include "step_ops.hpp"

#include <algorithm>
#include <type_traits>

namespace bmoe {

typedef const __attribute__((address_space(1))) void gf_glob_t;
typedef __attribute__((address_space(3))) void gf_lds_t;
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t gf_lds4_t;

constexpr int GF_CUS = 256;       // of a whole MI355X
constexpr int GF_SPLIT = 16;      // most workgroups that share a tile's depth
constexpr int GF_FEW = 4;         // most tokens of the kernel that takes them one by one

// what the places of a step past a ragged depth are filled with
__device__ const uint4 gf_zeros = {0, 0, 0, 0};

enum GfEpilogue { GF_OUT, GF_PART, GF_GATE, GF_GRAD };
enum GfActivation { GF_SILU = 0, GF_GELU = 1 };

struct GfGemm {
  const uint16_t* a;        // [M][K], or [K][M] (AT)
  const uint16_t* b;        // [N][K], or [K][N] (BT); GF_GATE: [2 ff][K], N = 2 ff
  int32_t lda, ldb;         // elements of a row of each
  int32_t M, N, K;
  int32_t nm, nn, band;     // tile rows and columns, tile rows of a band
  int32_t split, per;       // workgroups that share a tile's depth, steps of each
  uint16_t* out;            // GF_OUT [M][N]; GF_GATE h [M][ff]; GF_GRAD [M][2 ff] dg | du
  const uint16_t* add16;    // GF_OUT: [M][N] or null
  const float* add32;       // the same
  float* part;              // GF_PART: [split][M][N]
  uint16_t* pa;             // GF_GATE: [M][2 ff], u act'(g) and act(g), or null; GF_GRAD: read
  uint8_t* fine;            // [M][ff] four more bits of both
  int32_t ff;
};

__device__ __forceinline__ float gf_sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)); }
// GELU is the layers' own up to the end of its tail's range, where that is 2.6e-8, and 0 or g
// beyond.
__device__ __forceinline__ float gf_gelu(float g) { return fabsf(g) > 5.75f ? (g > 0.f ? g : g * 0.f) : gelu_erf(g); }
template <int F>
__device__ __forceinline__ float gf_act(float g) {
  return F == GF_GELU ? gf_gelu(g) : g * gf_sigmoid(g);
}
// act(g) and its derivative
template <int F>
__device__ __forceinline__ float2 gf_act_slope(float g) {
  if constexpr (F == GF_GELU) {
    const float slope = 0.5f * (1.0f + erf_as(g * 0.70710678118654752f)) +
                        g * 0.39894228040143268f * __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);
    return make_float2(gf_gelu(g), slope);
  }
  const float s = gf_sigmoid(g);
  return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
}

// The two factors of dh that the backward takes, p = u act'(g) for dg and a = act(g) for du, are
// kept to 12 significant bits: as bf16, truncated, and a byte with the next four bits of
// both.  In bf16 alone their rounding would count in dx and dw_in as much as those of dg
// and du themselves (3.0e-3 off in all, with these 2.4e-3), in fp32 they would be three more
// bytes to write and read.
struct GfKept {
  uint32_t p, a;            // fp32 values with the four bits behind bf16's, rounded
};
__device__ __forceinline__ GfKept gf_keep(float p, float a) { return {__float_as_uint(p) + 0x800u, __float_as_uint(a) + 0x800u}; }
__device__ __forceinline__ uint32_t gf_fine(GfKept v) { return (v.p >> 12 & 15u) | (v.a >> 8 & 0xF0u); }
__device__ __forceinline__ float gf_kept_p(uint32_t bf16, uint32_t fine) { return __uint_as_float(bf16 << 16 | (fine & 15u) << 12); }
__device__ __forceinline__ float gf_kept_a(uint32_t bf16, uint32_t fine) { return __uint_as_float(bf16 << 16 | (fine & 0xF0u) << 8); }

// Where chunk 0 of depth k lies in rows of T values whose other side is contiguous: the 32
// lanes that LDS serves at a time read 32 bytes each of depths 0 .. 3 and 8 .. 11, which are
// in eight places of the banks this way.  (With 8 .. 11 where 0 .. 3 are, LDS is busy twice as
// long in dW_in of 16384 x 2048 x 8192, half of it with conflicts, and the product 1.8 % slower.)
template <int T>
__device__ __forceinline__ int gf_turned_swizzle(int k) {
  return (2 * (k & 3)) ^ ((T == 64 ? 2 : 8) * (k >> 3 & 1));
}

// One workgroup per TM x TN tile of D[m][n] = sum_k A[m][k] B[n][k], WM x WN waves of
// TM / WM x TN / WN each (MFMA blocks of 16 x 16 x 32), NBUF steps of depth BK in the ring.
//
// LDS, contraction contiguous: [rows][BK], 16-byte chunk c of row r at c ^ (r % 8), in steps
// of 32 at c ^ (r / 2 % 4); a lane reads its 8 values of depth as one 16-byte chunk.  Other
// side contiguous: [BK depths][rows], chunk c of depth k at c ^ gf_turned_swizzle(k); 16 lanes
// read 4 depths of 16 rows as 8 bytes each and get 4 depths of their row.
//
// A step's 32-deep halves have a set of fragments each in turn: the reads of the next half
// are issued among the products of the current one, and the barrier that frees a ring
// place stands in front of a step's last products.  The first step of a depth that is no
// multiple of BK is the short one: it is loaded ahead of the loop, so the loop has no case
// for it.
#if defined(__HIP_DEVICE_COMPILE__)   // the host's pass knows no buffer resources and would drop the kernels
template <bool AT, bool BT, int EPI, int F, int TM, int TN, int BK, int WM, int WN, int NBUF>
__device__ __forceinline__ void gf_gemm(const GfGemm p, int bid) {
  constexpr int NW = WM * WN, NT = 64 * NW;
  constexpr int PM = TM / WM, PN = TN / WN, IM = PM / 16, IN = PN / 16, H = BK / 32;
  constexpr int STAGE = (TM + TN) * BK;          // halves of a ring place: A's, then B's
  constexpr int LA = TM * BK / 512 / NW, LB = TN * BK / 512 / NW;   // loads per wave and step
  static_assert(TM * BK % (512 * NW) == 0 && TN * BK % (512 * NW) == 0, "whole loads per wave");
  static_assert(EPI != GF_GATE || IN % 2 == 0, "gate and up blocks in pairs");
  extern __shared__ __attribute__((aligned(16))) uint16_t sm[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int wm = wave % WM, wn = wave / WM;
  // an XCD's workgroups take the same share of a block of tiles: bands of tile rows,
  // column by column within a band
  int t = xcd_remap(bid, p.nm * p.nn * p.split);
  const int tiles = p.nm * p.nn, share = t / tiles;
  t -= share * tiles;
  const int r0 = t / (p.band * p.nn) * p.band;
  t -= r0 * p.nn;
  const int hh = min(p.band, p.nm - r0);
  const int tn = t / hh, tm = r0 + t - tn * hh;
  const int m0 = tm * TM, n0 = tn * TN;
  const int nk1 = (p.K + BK - 1) / BK, short_by = nk1 * BK - p.K;
  const int k0 = share * p.per, nk = min(p.per, nk1 - k0);

  // one operand's loads of this wave: byte offsets of this lane's pieces from the tile's
  // first element; rows and columns past the matrix read its last ones and are not stored
  auto place = [&](auto turned, auto side, const uint16_t* q, int ld, int first, int count, bool gate, auto& off, auto& deep, size_t& advance) {
    constexpr bool TURNED = decltype(turned)::value;
    constexpr int T = decltype(side)::value, L = T * BK / 512 / NW;
    advance = TURNED ? size_t(BK) * ld * 2 : BK * 2;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int w = wave * L + j;
      if constexpr (TURNED) {
        constexpr int RC = T / 8, RPL = 64 / RC;
        const int k = w * RPL + lane / RC, c = (lane % RC) ^ gf_turned_swizzle<T>(k);
        off[j] = 2u * (uint32_t(k) * uint32_t(ld) + uint32_t(min(first + 8 * c, count - 8) - first));
        deep[j] = k;
      } else {
        constexpr int RC = BK / 8, RPL = 64 / RC;
        const int r = lane / RC, row = w * RPL + r, c = (lane % RC) ^ (BK == 64 ? r & 7 : r >> 1 & 3);
        uint32_t at;
        if (gate) {   // blocks of 16 rows of Wg and Wu in turn
          const int half = min(first / 2 + 16 * (row >> 5) + (row & 15), p.ff - 1);
          at = uint32_t(half + (row & 16 ? p.ff : 0));
        } else {
          at = uint32_t(min(first + row, count - 1) - first);
        }
        off[j] = 2u * (at * uint32_t(ld) + 8u * c);
        deep[j] = 8 * c;
      }
    }
    return reinterpret_cast<const char*>(q + (TURNED ? size_t(first) : gate ? size_t(0) : size_t(first) * ld));
  };
  uint32_t aoff[LA], boff[LB];
  int adeep[LA], bdeep[LB];   // depth within a step of the lane's first value
  size_t astep, bstep;        // bytes of a step
  const char* abase = place(std::integral_constant<bool, AT>{}, std::integral_constant<int, TM>{}, p.a, p.lda, m0, p.M, false, aoff, adeep, astep);
  const char* bbase = place(std::integral_constant<bool, BT>{}, std::integral_constant<int, TN>{}, p.b, p.ldb, n0, p.N, EPI == GF_GATE, boff, bdeep, bstep);
  auto place_of = [&](int buf, bool b) { return sm + buf * STAGE + (b ? TM * BK + wave * LB * 512 : wave * LA * 512); };
  auto load = [&](int kt, int buf) {
    const int s = k0 + min(kt, nk - 1);   // past the last one: the last one again, never read
    // bytes that the first step is short by: the steps behind it start that much earlier.
    // The step's address is in scalar registers, the lane's offsets as they are: an address of
    // 64 bits per lane and load takes 16 registers and an addition each
    auto at = [&](const char* base, size_t step) {
      return const_cast<char*>(base + size_t(s) * step - (s > 0 ? step / BK * short_by : 0));
    };
    const auto ra = __builtin_amdgcn_make_buffer_rsrc(at(abase, astep), 0, -1, 0x00027000);
    const auto rb = __builtin_amdgcn_make_buffer_rsrc(at(bbase, bstep), 0, -1, 0x00027000);
#pragma unroll
    for (int j = 0; j < LA; ++j) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (gf_lds_t*)(place_of(buf, false) + 512 * j), 16, int(aoff[j]), 0, 0, 0);
#pragma unroll
    for (int j = 0; j < LB; ++j) __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (gf_lds_t*)(place_of(buf, true) + 512 * j), 16, int(boff[j]), 0, 0, 0);
  };
  // step 0 of the whole depth: zeros behind its last value
  auto load_short = [&]() {
    auto one = [&](const char* base, uint32_t off, int deep, uint16_t* dst) {
      const char* at = deep < BK - short_by ? base + off : reinterpret_cast<const char*>(&gf_zeros);
      __builtin_amdgcn_global_load_lds((gf_glob_t*)at, (gf_lds_t*)dst, 16, 0, 0);
    };
#pragma unroll
    for (int j = 0; j < LA; ++j) one(abase, aoff[j], adeep[j], place_of(0, false) + 512 * j);
#pragma unroll
    for (int j = 0; j < LB; ++j) one(bbase, boff[j], bdeep[j], place_of(0, true) + 512 * j);
  };

  f32x4_t acc[IN][IM];
#pragma unroll
  for (int i = 0; i < IN; ++i)
#pragma unroll
    for (int j = 0; j < IM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  bf16x8_t fa[2][IM], fb[2][IN];
  // one operand's fragments of half h: COUNT blocks of 16 rows from `row` on
  auto read_one = [&](auto turned, auto side, const uint16_t* tile, int row, int h, auto& f) {
    constexpr int T = decltype(side)::value, COUNT = sizeof(f) / sizeof(f[0]);
    if constexpr (decltype(turned)::value) {
      const int k = 8 * g + (l16 >> 2);   // further depths of this lane's have its place too
      const uint16_t* q = tile + k * T + 4 * (l16 & 3);
#pragma unroll
      for (int j = 0; j < COUNT; ++j) {
        const uint16_t* at = q + ((row + 16 * j) ^ (8 * gf_turned_swizzle<T>(k))) + 32 * h * T;
        const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((gf_lds4_t*)at);
        const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((gf_lds4_t*)(at + 4 * T));
        typedef short i16x8_t __attribute__((ext_vector_type(8)));
        f[j] = __builtin_bit_cast(bf16x8_t, i16x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
      }
    } else {
      const uint16_t* q = tile + (row + l16) * BK + 8 * ((4 * h + g) ^ (BK == 64 ? l16 & 7 : l16 >> 1 & 3));
#pragma unroll
      for (int j = 0; j < COUNT; ++j) f[j] = *reinterpret_cast<const bf16x8_t*>(q + 16 * j * BK);
    }
  };
  auto read = [&](int buf, int h, bf16x8_t (&a)[IM], bf16x8_t (&b)[IN]) {
    read_one(std::integral_constant<bool, AT>{}, std::integral_constant<int, TM>{}, sm + buf * STAGE, PM * wm, h, a);
    read_one(std::integral_constant<bool, BT>{}, std::integral_constant<int, TN>{}, sm + buf * STAGE + TM * BK, PN * wn, h, b);
  };
  auto mul = [&](const bf16x8_t (&a)[IM], const bf16x8_t (&b)[IN]) {
#pragma unroll
    for (int i = 0; i < IN; ++i)
#pragma unroll
      for (int j = 0; j < IM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], a[j], acc[i][j], 0, 0, 0);
  };
  // order of a region: the reads behind the first products, the loads among the others
  auto spread = [&](auto loads) {
    constexpr int NL = decltype(loads)::value, READS = (AT ? 2 : 1) * IM + (BT ? 2 : 1) * IN, MULS = IM * IN;
    constexpr int FIRST = READS < MULS / 2 ? READS : MULS / 2, PER = (READS + FIRST - 1) / FIRST;
    constexpr int REST = MULS - FIRST, GAP = NL > 0 && REST / std::max(NL, 1) > 0 ? REST / std::max(NL, 1) : 1;
#pragma unroll
    for (int m = 0; m < FIRST; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
    }
#pragma unroll
    for (int m = 0; m < NL; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, GAP, 0);
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MULS, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // this wave's reads are done and its loads of all but the newest steps have arrived;
  // then the same of every wave
  auto arrive = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NBUF - 2) * (LA + LB)) : "memory");
  };
  if (k0 == 0 && short_by) {
    load_short();
    if (nk == 1) {   // the loads past it read no more than it has
#pragma unroll
      for (int j = 0; j < LA; ++j) aoff[j] = adeep[j] < BK - short_by ? aoff[j] : 0;
#pragma unroll
      for (int j = 0; j < LB; ++j) boff[j] = bdeep[j] < BK - short_by ? boff[j] : 0;
    }
  } else {
    load(0, 0);
  }
#pragma unroll
  for (int b = 1; b < NBUF - 1; ++b) load(b, b);
  arrive();
  load(NBUF - 1, NBUF - 1);
  read(0, 0, fa[0], fb[0]);
  int buf = 0;
  // a step whose first half is in the fragments `set`
  auto step = [&](int kt, auto set) {
    constexpr int P = decltype(set)::value;
    const int next = buf + 1 == NBUF ? 0 : buf + 1;
    if constexpr (H == 2) {
      read(buf, 1, fa[1 - P], fb[1 - P]);
      mul(fa[P], fb[P]);
      spread(std::integral_constant<int, 0>{});
    }
    constexpr int Q = H == 2 ? 1 - P : P;
    arrive();
    read(next, 0, fa[1 - Q], fb[1 - Q]);
    load(kt + NBUF, buf);
    mul(fa[Q], fb[Q]);
    spread(std::integral_constant<int, LA + LB>{});
    buf = next;
  };
  using even = std::integral_constant<int, 0>;
  using odd = std::integral_constant<int, 1>;
  if constexpr (H == 2) {
    for (int kt = 0; kt < nk; ++kt) step(kt, even{});
  } else {
    int kt = 0;
    for (; kt + 1 < nk; kt += 2) {
      step(kt, even{});
      step(kt + 1, odd{});
    }
    if (kt < nk) step(kt, even{});
  }
  // loads past the last step may still be writing to the ring
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // acc[i][j][r] = D[m0 + PM wm + 16 j + l16][n0 + PN wn + 16 i + 4 g + r]
  if constexpr (EPI == GF_PART) {
    float* out = p.part + size_t(share) * p.M * p.N;
#pragma unroll
    for (int j = 0; j < IM; ++j) {
      const int m = m0 + PM * wm + 16 * j + l16;
#pragma unroll
      for (int i = 0; i < IN; ++i) {
        const int n = n0 + PN * wn + 16 * i + 4 * g;
        if (m < p.M && n < p.N) *reinterpret_cast<f32x4_t*>(out + size_t(m) * p.N + n) = acc[i][j];
      }
    }
    return;
  }
  uint16_t* st = sm;
  // bf16 values f(i, j) of this lane's blocks (i a multiple of BY, columns 16 / BY apart)
  // to a staged tile of W columns, and that in rows of 16 bytes to dst, W columns from c0 on
  // inside `cols`
  auto put = [&](auto by, uint16_t* dst, int ld, int c0, int cols, auto&& f) {
    constexpr int BY = decltype(by)::value, W = TN / BY, ST = W + 4;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < IM; ++j)
#pragma unroll
      for (int i = 0; i < IN; i += BY)
        *reinterpret_cast<uint2*>(st + (PM * wm + 16 * j + l16) * ST + (PN * wn + 16 * i) / BY + 4 * g) = f(i, j);
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < TM * W / 8 / NT; ++q) {
      const int k = tid + NT * q, r = k / (W / 8), c = 8 * (k % (W / 8));
      if (m0 + r >= p.M || c0 + c >= cols) continue;
      const uint2 lo = *reinterpret_cast<const uint2*>(st + r * ST + c), hi = *reinterpret_cast<const uint2*>(st + r * ST + c + 4);
      *reinterpret_cast<uint4*>(dst + size_t(m0 + r) * ld + c0 + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  };
  auto pack = [](f32x4_t v) { return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])); };
  auto four = [](const uint16_t* q) {
    const uint2 u = *reinterpret_cast<const uint2*>(q);
    return f32x4_t{bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y)};
  };
  using one = std::integral_constant<int, 1>;
  using two = std::integral_constant<int, 2>;
  if constexpr (EPI == GF_OUT) {
    if (p.add16 || p.add32) {
#pragma unroll
      for (int j = 0; j < IM; ++j) {
        const int m = m0 + PM * wm + 16 * j + l16;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
          const int n = n0 + PN * wn + 16 * i + 4 * g;
          if (m >= p.M || n >= p.N) continue;
          const size_t at = size_t(m) * p.N + n;
          if (p.add16) acc[i][j] += four(p.add16 + at);
          if (p.add32) acc[i][j] += *reinterpret_cast<const f32x4_t*>(p.add32 + at);
        }
      }
    }
    put(one{}, p.out, p.N, n0, p.N, [&](int i, int j) { return pack(acc[i][j]); });
  } else if constexpr (EPI == GF_GATE) {
    const int c0 = n0 / 2;
    if (!p.pa) {
      put(two{}, p.out, p.ff, c0, p.ff, [&](int i, int j) {
        f32x4_t h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = gf_act<F>(acc[i][j][r]) * acc[i + 1][j][r];
        return pack(h);
      });
      return;
    }
    // h, the kept factors and their further bits take the places of g and u: 7 of 8 words
#pragma unroll
    for (int j = 0; j < IM; ++j)
#pragma unroll
      for (int i = 0; i < IN; i += 2) {
        f32x4_t o;
        uint32_t kp[4], ka[4], fine = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float2 f = gf_act_slope<F>(acc[i][j][r]);
          const float u = acc[i + 1][j][r];
          o[r] = f.x * u;
          const GfKept k = gf_keep(u * f.y, f.x);
          kp[r] = k.p;
          ka[r] = k.a;
          fine |= gf_fine(k) << (8 * r);
        }
        auto upper = [](uint32_t x, uint32_t y) { return x >> 16 | (y & 0xFFFF0000u); };
        const uint2 h = pack(o);
        acc[i][j] = __builtin_bit_cast(f32x4_t, make_uint4(h.x, h.y, upper(kp[0], kp[1]), upper(kp[2], kp[3])));
        acc[i + 1][j] = __builtin_bit_cast(f32x4_t, make_uint4(upper(ka[0], ka[1]), upper(ka[2], ka[3]), fine, 0));
        asm volatile("" : "+v"(acc[i][j]), "+v"(acc[i + 1][j]));   // here, not where they are stored
      }
    auto words = [](f32x4_t v) { return __builtin_bit_cast(uint4, v); };
    // both factors beside each other, then h and the bytes
    constexpr int W = TN / 2, SF = TN + 4, SH = W + 4, SB = W / 4 + 1;   // halves, halves, words of a staged row
    uint32_t* bytes = reinterpret_cast<uint32_t*>(sm + TM * SH);
    auto each = [&](auto&& f) {   // f(row, column of this lane's first value, i, j)
#pragma unroll
      for (int j = 0; j < IM; ++j)
#pragma unroll
        for (int i = 0; i < IN; i += 2) f(PM * wm + 16 * j + l16, (PN * wn + 16 * i) / 2 + 4 * g, i, j);
    };
    auto eight = [&](int at) {
      const uint2 lo = *reinterpret_cast<const uint2*>(st + at), hi = *reinterpret_cast<const uint2*>(st + at + 4);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    };
    each([&](int r, int c, int i, int j) {
      *reinterpret_cast<uint2*>(st + r * SF + c) = make_uint2(words(acc[i][j]).z, words(acc[i][j]).w);
      *reinterpret_cast<uint2*>(st + r * SF + W + c) = make_uint2(words(acc[i + 1][j]).x, words(acc[i + 1][j]).y);
    });
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < TM * TN / 8 / NT; ++q) {
      const int k = tid + NT * q, r = k / (TN / 8), c = 8 * (k % (TN / 8)), h = c0 + c % W;
      if (m0 + r < p.M && h < p.ff) *reinterpret_cast<uint4*>(p.pa + size_t(m0 + r) * 2 * p.ff + (c < W ? 0 : p.ff) + h) = eight(r * SF + c);
    }
    __syncthreads();
    each([&](int r, int c, int i, int j) {
      *reinterpret_cast<uint2*>(st + r * SH + c) = make_uint2(words(acc[i][j]).x, words(acc[i][j]).y);
      bytes[r * SB + c / 4] = words(acc[i + 1][j]).z;
    });
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < TM * W / 8 / NT; ++q) {
      const int k = tid + NT * q, r = k / (W / 8), c = 8 * (k % (W / 8));
      if (m0 + r >= p.M || c0 + c >= p.ff) continue;
      const size_t at = size_t(m0 + r) * p.ff + c0 + c;
      *reinterpret_cast<uint4*>(p.out + at) = eight(r * SH + c);
      *reinterpret_cast<uint2*>(p.fine + at) = make_uint2(bytes[r * SB + c / 4], bytes[r * SB + c / 4 + 1]);
    }
  } else if constexpr (EPI == GF_GRAD) {
    // dh goes through LDS in fp32, PM rows at a time, so that its factors are read and dg and
    // du written in whole rows; the factors are on their way while it does
    constexpr int ST = TN + 4, PIECES = PM * TN / 8 / NT, PER = PIECES < 4 ? PIECES : 4;
    float* dh = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int part = 0; part < WM; ++part) {
      if (part > 0) __syncthreads();
      if (wm == part) {
#pragma unroll
        for (int j = 0; j < IM; ++j)
#pragma unroll
          for (int i = 0; i < IN; ++i) *reinterpret_cast<f32x4_t*>(dh + (16 * j + l16) * ST + PN * wn + 16 * i + 4 * g) = acc[i][j];
      }
#pragma unroll
      for (int q0 = 0; q0 < PIECES; q0 += PER) {
        uint4 pv[PER], av[PER];
        uint2 fv[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const int k = tid + NT * (q0 + q), r = k / (TN / 8), c = 8 * (k % (TN / 8));
          const size_t m = min(m0 + PM * part + r, p.M - 1);
          const int n = min(n0 + c, p.ff - 8);
          pv[q] = *reinterpret_cast<const uint4*>(p.pa + m * 2 * p.ff + n);
          av[q] = *reinterpret_cast<const uint4*>(p.pa + m * 2 * p.ff + p.ff + n);
          fv[q] = *reinterpret_cast<const uint2*>(p.fine + m * p.ff + n);
        }
        if (q0 == 0) __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const int k = tid + NT * (q0 + q), r = k / (TN / 8), c = 8 * (k % (TN / 8));
          const uint32_t pw[4] = {pv[q].x, pv[q].y, pv[q].z, pv[q].w}, aw[4] = {av[q].x, av[q].y, av[q].z, av[q].w}, fw[2] = {fv[q].x, fv[q].y};
          uint32_t dg[4], du[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 d = *reinterpret_cast<const float2*>(dh + r * ST + c + 2 * e);
            const uint32_t f = fw[e / 2] >> (16 * (e & 1));
            dg[e] = pack_bf16x2(d.x * gf_kept_p(pw[e], f), d.y * gf_kept_p(pw[e] >> 16, f >> 8));
            du[e] = pack_bf16x2(d.x * gf_kept_a(aw[e], f), d.y * gf_kept_a(aw[e] >> 16, f >> 8));
          }
          if (m0 + PM * part + r >= p.M || n0 + c >= p.ff) continue;
          uint16_t* out = p.out + size_t(m0 + PM * part + r) * 2 * p.ff + n0 + c;
          *reinterpret_cast<uint4*>(out) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
          *reinterpret_cast<uint4*>(out + p.ff) = make_uint4(du[0], du[1], du[2], du[3]);
        }
      }
    }
  }
}
#endif

template <bool AT, bool BT, int EPI, int F, int TM, int TN, int BK, int WM, int WN, int NBUF>
__global__ __launch_bounds__(64 * WM * WN, 2) void gf_gemm_kernel(GfGemm p) {
#if defined(__HIP_DEVICE_COMPILE__)
  gf_gemm<AT, BT, EPI, F, TM, TN, BK, WM, WN, NBUF>(p, blockIdx.x);
#endif
}

// dx, dW_in and dW_down, those of them that are wanted, in one launch: where one of them leaves CUs without work, the next
// one's workgroups take them (gf_group_pick).
struct GfGroup {
  GfGemm job[3];
  int32_t start[3];         // first workgroups, multiples of 8: a job's XCDs are the launch's
};
template <int EPI, int TM, int TN, int BK, int WM, int WN, int NBUF>
__global__ __launch_bounds__(64 * WM * WN, 2) void gf_group_kernel(GfGroup g) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int bid = blockIdx.x, k = bid < g.start[1] ? 0 : bid < g.start[2] ? 1 : 2;
  const GfGemm p = g.job[k];
  if (bid - g.start[k] >= p.nm * p.nn * p.split) return;
  if (k == 0) gf_gemm<false, true, EPI, 0, TM, TN, BK, WM, WN, NBUF>(p, bid);
  else gf_gemm<true, true, EPI, 0, TM, TN, BK, WM, WN, NBUF>(p, bid - g.start[k]);
#endif
}

// The shares' sums of up to three products, added in order, and what is added to them.
struct GfSum {
  const float* part;
  uint16_t* out;
  const uint16_t* add16;    // or null
  const float* add32;       // or null
  size_t n;
  int32_t split, blocks;
};
struct GfSums {
  GfSum of[3];
};
__global__ __launch_bounds__(256) void gf_reduce_kernel(GfSums g) {
  int b = blockIdx.x, w = 0;
  while (w < 2 && b >= g.of[w].blocks) b -= g.of[w++].blocks;
  const GfSum p = g.of[w];
  const size_t i = (size_t(b) * 256 + threadIdx.x) * 4;
  if (i >= p.n) return;
  f32x4_t s = *reinterpret_cast<const f32x4_t*>(p.part + i);
#pragma unroll 4
  for (int k = 1; k < p.split; ++k) s += *reinterpret_cast<const f32x4_t*>(p.part + k * p.n + i);
  if (p.add16) {
    const uint2 u = *reinterpret_cast<const uint2*>(p.add16 + i);
    s += f32x4_t{bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y)};
  }
  if (p.add32) s += *reinterpret_cast<const f32x4_t*>(p.add32 + i);
  *reinterpret_cast<uint2*>(p.out + i) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

// Few tokens: bound by the weights' bytes, each of which is read once, a row's 1024 at a
// time by a wave (16 bytes per lane), and multiplied in fp32 without the matrix cores: with
// TOK tokens 8 + 8 TOK operations on 8 weights, 6 us of the 20 that 100 MB take at TOK = 4.
// (One token, d 2048, ff 8192: 22.5 us, 4.5 TB/s with both launches; as operands of MFMA,
// 64 bytes of 16 rows at a time, 30, in tiles of 64 28.  8 tokens: 39, in tiles 28.)
// A wave takes four rows (GATE: two of Wg and of Wu each), DEEP steps of 512 of their depth
// on their way at a time: of a short depth more would be loaded for nothing (four steps:
// one token 23.8 us, at d 1024, ff 4096 11.6 instead of 9.7, four tokens 13.0 instead of
// 11.6).  `parts` waves of a workgroup share the depth of the same rows.
// h stays fp32 between the launches: no matrix core asks for it in bf16, and it comes out of
// the L2 (four tokens 27.0 us, in bf16 25.5).
struct GfFew {
  const uint16_t* x;        // [M][K], GATE
  float* h;                 // GATE: [M][R], written; otherwise [M][K], read
  const uint16_t* w;        // [R][K], GATE: [2 R][K]
  const uint16_t* add;      // [M][R] or null
  uint16_t* out;            // [M][R], GATE: or null
  uint16_t* pa;             // GATE: [M][2 R] or null
  uint8_t* fine;            // GATE: [M][R] when pa is set
  int32_t M, R, K, parts;
};
constexpr int GF_FEW_WAVES = 8;
template <bool GATE, int F, int TOK>
__global__ __launch_bounds__(64 * GF_FEW_WAVES) void gf_few_kernel(GfFew p) {
  constexpr int ROWS = GATE ? 2 : 4, DEEP = TOK > (GATE ? 2 : 1) ? 1 : 2;
  __shared__ float red[GF_FEW_WAVES][4][TOK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = GF_FEW_WAVES / p.parts, part = wave % p.parts;
  const int row0 = (blockIdx.x * groups + wave / p.parts) * ROWS;
  const int steps = (p.K + 511) / 512, per = (steps + p.parts - 1) / p.parts, s0 = part * per, s1 = min(s0 + per, steps);
  const uint16_t* w[4];
  constexpr int XV = GATE ? 1 : 2;   // of 16 bytes for 8 values of x or h
  const uint4* x[TOK];
#pragma unroll
  for (int r = 0; r < 4; ++r) w[r] = p.w + size_t(min(row0 + r % ROWS, p.R - 1) + r / ROWS * p.R) * p.K;
#pragma unroll
  for (int m = 0; m < TOK; ++m) x[m] = reinterpret_cast<const uint4*>(GATE ? static_cast<const void*>(p.x) : p.h) + size_t(min(m, p.M - 1)) * p.K / 8 * XV;
  float acc[4][TOK] = {};
  for (int s = s0; s < s1; s += DEEP) {
    uint4 wv[DEEP][4], xv[DEEP][TOK][XV];
#pragma unroll
    for (int u = 0; u < DEEP; ++u) {
      const int at = min(512 * (s + u) + 8 * lane, p.K - 8);   // past the end the last one, which counts as zeros
#pragma unroll
      for (int r = 0; r < 4; ++r) wv[u][r] = *reinterpret_cast<const uint4*>(w[r] + at);
#pragma unroll
      for (int m = 0; m < TOK; ++m)
#pragma unroll
        for (int v = 0; v < XV; ++v) xv[u][m][v] = x[m][at / 8 * XV + v];
    }
#pragma unroll
    for (int u = 0; u < DEEP; ++u) {
      const bool in = s + u < s1 && 512 * (s + u) + 8 * lane < p.K;
      float xf[TOK][8];
#pragma unroll
      for (int m = 0; m < TOK; ++m) {
#pragma unroll
        for (int v = 0; v < XV; ++v) {
          const uint32_t q[4] = {xv[u][m][v].x, xv[u][m][v].y, xv[u][m][v].z, xv[u][m][v].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (GATE) {
              xf[m][2 * e] = in ? bf16lo(q[e]) : 0.f;
              xf[m][2 * e + 1] = in ? bf16hi(q[e]) : 0.f;
            } else {
              xf[m][4 * v + e] = in ? __uint_as_float(q[e]) : 0.f;
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t q[4] = {wv[u][r].x, wv[u][r].y, wv[u][r].z, wv[u][r].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = in ? bf16lo(q[e]) : 0.f, hi = in ? bf16hi(q[e]) : 0.f;
#pragma unroll
          for (int m = 0; m < TOK; ++m) {
            acc[r][m] = fmaf(lo, xf[m][2 * e], acc[r][m]);
            acc[r][m] = fmaf(hi, xf[m][2 * e + 1], acc[r][m]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      const float v = ln_wave_sum<64>(acc[r][m]);
      if (lane == 0) red[wave][r][m] = v;
    }
  __syncthreads();
  // one value of the result each
  const int e = threadIdx.x, m = e % TOK, r = e / TOK % ROWS, group = e / (TOK * ROWS);
  const int row = (blockIdx.x * groups + group) * ROWS + r;
  if (group >= groups || m >= p.M || row >= p.R) return;
  float v = 0.f, u = 0.f;
  for (int k = group * p.parts; k < (group + 1) * p.parts; ++k) {
    v += red[k][r][m];
    if (GATE) u += red[k][(ROWS + r) & 3][m];
  }
  const size_t at = size_t(m) * p.R + row;
  if constexpr (GATE) {
    if (p.pa) {
      const float2 f = gf_act_slope<F>(v);
      const GfKept k = gf_keep(u * f.y, f.x);
      p.pa[at + size_t(m) * p.R] = uint16_t(k.p >> 16);
      p.pa[at + size_t(m + 1) * p.R] = uint16_t(k.a >> 16);
      p.fine[at] = uint8_t(gf_fine(k));
    }
    v = gf_act<F>(v) * u;
    p.h[at] = v;
    if (!p.out) return;
  } else if (p.add) {
    v += load1<ACT_BF16>(p.add, at);
  }
  p.out[at] = uint16_t(pack_bf16x2(v, v));
}

__global__ __launch_bounds__(256) void gf_zero_kernel(uint16_t* out, size_t n) {
  for (size_t i = (size_t(blockIdx.x) * 256 + threadIdx.x) * 8; i < n; i += size_t(gridDim.x) * 2048)
    *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ host
namespace {

// Tiles a product may have.  GF_128 has eight waves of 64 x 32 and a CU of its own, GF_128_2
// four of 64 x 64 and shares the CU with a second workgroup.
enum GfTiling { GF_64, GF_128, GF_128_2, GF_256 };
struct GfTile {
  GfTiling tiling;
  int split;
  double time;
};
constexpr int gf_tile_side(GfTiling t) { return t == GF_64 ? 64 : t == GF_256 ? 256 : 128; }

// A product's tiles and the workgroups that share a tile's depth, by a time estimate in
// microseconds: rounds of workgroups over the CUs, a step of 64 by the lone workgroup of
// a CU or by each of two, a tile's beginning and end; shares are written and read again in
// fp32 by a launch behind.  Operands turned in LDS take longer, their reads being half as
// wide.  The constants are fitted to 31 products of 0.6 to 1100 GFLOP, each with every
// tile and split forced (M x N x K, us: 16384 x 2048 x 8192 as x W^T, 256 405, 128_2 467, 128 516,
// 64 777; 2736 x 512 x 4001 as dy^T x, 128_2 in 5 shares 27.7, 64 40.8; 4096 x 1024 x 4096 128 32.8,
// 128_2 in 2 shares 41.1, 64 46.2; 256 x 2048 x 8192 64 in 2 shares 17.7, 128 in 8 18.3); a
// pick is within a tenth of the best of them.
struct GfOption {
  GfTiling tiling;
  int per_cu;
  double lone[2], shared[2], once;   // steps: plain, turned
};
constexpr GfOption gf_options[] = {{GF_64, 2, {0.2, 0.38}, {0.42, 0.53}, 3.0},
                                   {GF_128, 1, {0.48, 0.73}, {0, 0}, 2.0},
                                   {GF_128_2, 2, {0.66, 0.8}, {0.91, 1.0}, 3.0},
                                   {GF_256, 1, {1.58, 1.71}, {0, 0}, 4.0}};
GfTile gf_pick(int M, int N, int K, bool turned, bool may_split) {
  GfTile best{GF_64, 1, 0};
  const int steps = (K + 63) / 64;
  for (const GfOption& o : gf_options) {
    const int side = gf_tile_side(o.tiling);
    const int64_t tiles = int64_t((M + side - 1) / side) * ((N + side - 1) / side);
    for (int split = 1; split <= (may_split ? GF_SPLIT : 1); ++split) {
      const int per = (steps + split - 1) / split;
      // no share without a step, and then none of twice as many steps of 32 either, nor of one less
      if (split > 1 && ((split - 1) * per >= steps || per < 4)) break;
      const int64_t n = tiles * split;
      const double step = o.per_cu == 1 || n <= GF_CUS ? o.lone[turned] : o.shared[turned];
      double time = double((n + GF_CUS * o.per_cu - 1) / (GF_CUS * o.per_cu)) * (per * step + o.once);
      if (split > 1) time += 3.0 + double(M) * N * split / 1e6;
      if (best.time == 0 || time < best.time) best = GfTile{o.tiling, split, time};
    }
  }
  return best;
}

// g, u -> h, and dh -> dg, du: never in shares, whose sums the epilogue would lack.
GfTiling gf_gate_tiling(int tokens, int d, int ff) { return gf_pick(tokens, 2 * ff, d, false, false).tiling; }
GfTiling gf_grad_tiling(int tokens, int d, int ff) { return gf_pick(tokens, ff, d, true, false).tiling; }

size_t gf_round(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t gf_part_bytes(int M, int N, int split) { return gf_round(size_t(split) * M * N * 4); }
size_t gf_pick_bytes(int M, int N, int K, bool turned) {
  const int split = gf_pick(M, N, K, turned, true).split;
  return split > 1 ? gf_part_bytes(M, N, split) : 0;
}

// A product's tiles and steps; its workgroups.
int gf_plan(GfGemm& p, int side, int step) {
  p.nm = (p.M + side - 1) / side;
  p.nn = (p.N + side - 1) / side;
  p.per = ((p.K + step - 1) / step + p.split - 1) / p.split;
  p.band = std::min(p.nm, 8);
  return p.nm * p.nn * p.split;
}

template <bool AT, bool BT, int EPI, int F, int T, int BK, int WM, int WN, int NBUF>
hipError_t gf_go(GfGemm p, hipStream_t s) {
  // the ring; staged tiles of bf16, or of fp32 in WM parts
  constexpr size_t ring = size_t(NBUF) * 2 * T * BK * 2;
  constexpr size_t stage = EPI == GF_GRAD ? size_t(T / WM) * (T + 4) * 4 : size_t(T) * (T + 4) * 2;
  constexpr size_t lds = ring > stage ? ring : stage;
  const auto kernel = gf_gemm_kernel<AT, BT, EPI, F, T, T, BK, WM, WN, NBUF>;
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(unsigned(gf_plan(p, T, BK))), dim3(64 * WM * WN), lds, s, p);
  return hipGetLastError();
}

// F: of GF_GATE alone (what GF_GRAD needs of the activation is in the state).
template <bool AT, bool BT, int EPI, int F = GF_SILU>
hipError_t gf_tiled(const GfGemm& p, GfTiling t, hipStream_t s) {
  if (t == GF_64) return gf_go<AT, BT, EPI, F, 64, 64, 2, 2, 4>(p, s);
  if (t == GF_128) return gf_go<AT, BT, EPI, F, 128, 64, 2, 4, 3>(p, s);
  if (t == GF_128_2) return gf_go<AT, BT, EPI, F, 128, 64, 2, 2, 2>(p, s);
  // Steps of 32 in a ring of four load three quarters of the ring ahead where steps of 64 in
  // the same LDS load half; with a turned operand that is the faster (dx of 16384 x 2048 x 8192
  // 955 us against 1006, dg | du 675 against 698, dW_in and dW_down 715 against 735 on average),
  // with none the doubled barriers cost as much (h 1109 against 1097, y 487 both).
  if constexpr (BT) return gf_go<AT, BT, EPI, F, 256, 32, 2, 4, 4>(p, s);
  else return gf_go<AT, BT, EPI, F, 256, 64, 2, 4, 2>(p, s);
}

// The second launch of products written as partial sums.
hipError_t gf_reduce(const GfGemm* p, int count, hipStream_t s) {
  GfSums g{};
  unsigned blocks = 0;
  for (int k = 0; k < count; ++k) {
    if (p[k].M == 0) continue;
    const size_t n = size_t(p[k].M) * p[k].N;
    g.of[k] = GfSum{p[k].part, p[k].out, p[k].add16, p[k].add32, n, p[k].split, int32_t((n / 4 + 255) / 256)};
    blocks += unsigned(g.of[k].blocks);
  }
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(gf_reduce_kernel, dim3(blocks), dim3(256), 0, s, g);
  return hipGetLastError();
}

// A product whose result is written as it is (plus what is added), in shares where the
// estimate says so.
template <bool AT, bool BT>
hipError_t gf_product(GfGemm p, float* part, hipStream_t s) {
  const GfTile t = gf_pick(p.M, p.N, p.K, AT || BT, true);
  p.split = t.split;
  if (t.split == 1) return gf_tiled<AT, BT, GF_OUT>(p, t.tiling, s);
  p.part = part;
  const hipError_t e = gf_tiled<AT, BT, GF_PART>(p, t.tiling, s);
  return e != hipSuccess ? e : gf_reduce(&p, 1, s);
}

template <bool GATE, int F = GF_SILU>
hipError_t gf_few(GfFew p, hipStream_t s) {
  // waves that share rows: 4096 in all (16 to a CU), down to one step of the depth each
  const int blocks = (p.R + (GATE ? 1 : 3)) / (GATE ? 2 : 4), steps = (p.K + 511) / 512;
  p.parts = 1;
  while (p.parts < GF_FEW_WAVES && int64_t(blocks) * p.parts < 4096 && 2 * p.parts <= steps) p.parts *= 2;
  const int groups = GF_FEW_WAVES / p.parts;
  const auto kernel = p.M == 1 ? gf_few_kernel<GATE, F, 1> : p.M == 2 ? gf_few_kernel<GATE, F, 2> : gf_few_kernel<GATE, F, 4>;
  hipLaunchKernelGGL(kernel, dim3(unsigned((blocks + groups - 1) / groups)), dim3(64 * GF_FEW_WAVES), 0, s, p);
  return hipGetLastError();
}

// The backward's last three products in one launch: 0 where they are better off one by one.
struct GfTogether {
  int side;                 // 0, 128 (two workgroups to a CU) or 256
  bool parts;               // all of them as partial sums, also those in one share
  int split[3];
};
// their M, N and K
void gf_three(int tokens, int d, int ff, int (&m)[3], int (&n)[3], int (&k)[3]) {
  m[0] = tokens; n[0] = d; k[0] = 2 * ff;
  m[1] = 2 * ff; n[1] = d; k[1] = tokens;
  m[2] = d; n[2] = ff; k[2] = tokens;
}
// By gf_pick's estimate, with the workgroups dealt out in order to whatever place is free first
// (whole backward one by one and together, us: 4001 x 512 x 1368 94 and 69, 2354 x 1984 x 832 108
// and 84, 4503 x 1536 x 5696 619 and 479, 677 x 1024 x 320 35 and 23; left one by one, by 3 %:
// 15899 x 1088 x 4096 1056 and 1067).
GfTogether gf_group_pick(int tokens, int d, int ff) {
  int m[3], n[3], k[3];
  gf_three(tokens, d, ff, m, n, k);
  GfTogether best{0, false, {1, 1, 1}};
  double least = 0;
  for (int j = 0; j < 3; ++j) least += 0.97 * gf_pick(m[j], n[j], k[j], true, true).time;
  for (const int side : {128, 256}) {
    const int places = side == 128 ? 2 * GF_CUS : GF_CUS;
    int64_t tiles[3], all = 0;
    int steps[3];
    for (int j = 0; j < 3; ++j) {
      tiles[j] = int64_t((m[j] + side - 1) / side) * ((n[j] + side - 1) / side);
      steps[j] = (k[j] + 63) / 64;
      all += tiles[j];
    }
    if (all > 4 * places) continue;   // what the last ones leave empty is little
    for (int s = 0; s < 3 * GF_SPLIT; ++s) {   // steps of a workgroup: those of one product in 1 .. GF_SPLIT shares
      const int per = (steps[s / GF_SPLIT] + s % GF_SPLIT) / (s % GF_SPLIT + 1);
      if (per < 4) continue;
      int split[3];
      int64_t count = 0;
      double sums = 0;
      for (int j = 0; j < 3; ++j) {
        split[j] = std::min((steps[j] + per - 1) / per, GF_SPLIT);
        const int own = (steps[j] + split[j] - 1) / split[j];
        split[j] = (steps[j] + own - 1) / own;
        count += tiles[j] * split[j];
        sums += 1.6 * double(m[j]) * n[j] * split[j] / 1e6;
      }
      const bool parts = split[0] > 1 || split[1] > 1 || split[2] > 1;
      if (count > 8 * places) continue;
      const GfOption& o = gf_options[side == 256 ? GF_256 : GF_128_2];
      const double step = o.per_cu == 1 || count <= GF_CUS ? o.lone[1] : o.shared[1];
      // places by when they are free
      struct { double at; int64_t n; } free[8] = {{0, places}};
      int kinds = 1;
      double last = 0;
      for (int j = 0; j < 3; ++j) {
        const double takes = ((steps[j] + split[j] - 1) / split[j]) * step + o.once;
        for (int64_t left = tiles[j] * split[j]; left > 0;) {
          int f = 0;
          for (int q = 1; q < kinds; ++q)
            if (free[q].at < free[f].at) f = q;
          const int64_t now = std::min(left, free[f].n);
          const double until = free[f].at + takes;
          last = std::max(last, until);
          left -= now;
          free[f].n -= now;
          if (free[f].n == 0) free[f] = free[--kinds];
          free[kinds++] = {until, now};
        }
      }
      const double time = last + (parts ? 3.0 + sums : 0.0);
      if (time < least) {
        least = time;
        best = GfTogether{side, parts, {split[0], split[1], split[2]}};
      }
    }
  }
  return best;
}

template <int EPI, int T, int BK, int WM, int WN, int NBUF>
hipError_t gf_group_go(GfGroup& g, hipStream_t s) {
  constexpr size_t ring = size_t(NBUF) * 2 * T * BK * 2, stage = size_t(T) * (T + 4) * 2, lds = ring > stage ? ring : stage;
  const auto kernel = gf_group_kernel<EPI, T, T, BK, WM, WN, NBUF>;
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  int blocks = 0;
  for (int k = 0; k < 3; ++k) {
    g.start[k] = (blocks + 7) / 8 * 8;
    if (!g.job[k].out) g.job[k].M = 0;   // not wanted
    blocks = g.start[k] + gf_plan(g.job[k], T, BK);
  }
  hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(64 * WM * WN), lds, s, g);
  return hipGetLastError();
}

}  // namespace

size_t gf_forward_workspace(int tokens, int d, int ff, bool with_state) {
  if (tokens == 0) return 0;
  if (tokens <= GF_FEW) return size_t(tokens) * ff * 4;
  const size_t h = with_state ? 0 : gf_round(size_t(tokens) * ff * 2);
  return h + gf_pick_bytes(tokens, d, ff, false);
}

hipError_t launch_gated_ffn_forward(const GfFwdArgs& a, hipStream_t s) {
  const int M = a.tokens;
  if (M == 0) return hipSuccess;
  // of the state: the kept factors, h, the factors' further bits
  uint16_t* pa = a.state;
  uint8_t* fine = reinterpret_cast<uint8_t*>(a.state + size_t(M) * 3 * a.ff);
  char* ws = static_cast<char*>(a.ws);
  uint16_t* h = a.state ? a.state + size_t(M) * 2 * a.ff : reinterpret_cast<uint16_t*>(ws);
  float* part = reinterpret_cast<float*>(ws + (a.state ? 0 : gf_round(size_t(M) * a.ff * 2)));
  if (M <= GF_FEW) {
    float* h32 = reinterpret_cast<float*>(ws);
    const GfFew gate{a.x, h32, a.w_in, nullptr, a.state ? h : nullptr, pa, fine, M, a.ff, a.d, 1};
    const hipError_t e = a.gelu ? gf_few<true, GF_GELU>(gate, s) : gf_few<true, GF_SILU>(gate, s);
    return e != hipSuccess ? e : gf_few<false>(GfFew{nullptr, h32, a.w_down, a.add, a.y, nullptr, nullptr, M, a.d, a.ff, 1}, s);
  }
  GfGemm p{};
  p.a = a.x;
  p.b = a.w_in;
  p.lda = p.ldb = p.K = a.d;
  p.M = M;
  p.N = 2 * a.ff;
  p.split = 1;
  p.out = h;
  p.pa = pa;
  p.fine = fine;
  p.ff = a.ff;
  const GfTiling tiling = gf_gate_tiling(M, a.d, a.ff);
  hipError_t e = a.gelu ? gf_tiled<false, false, GF_GATE, GF_GELU>(p, tiling, s) : gf_tiled<false, false, GF_GATE, GF_SILU>(p, tiling, s);
  if (e != hipSuccess) return e;
  p = GfGemm{};
  p.a = h;
  p.b = a.w_down;
  p.lda = p.ldb = p.K = a.ff;
  p.M = M;
  p.N = a.d;
  p.out = a.y;
  p.add16 = a.add;
  return gf_product<false, false>(p, part, s);
}

size_t gf_backward_workspace(int tokens, int d, int ff) {
  if (tokens == 0) return 0;
  int m[3], n[3], k[3];
  gf_three(tokens, d, ff, m, n, k);
  const GfTogether t = gf_group_pick(tokens, d, ff);
  size_t one = 0, all = 0;
  for (int j = 0; j < 3; ++j) {
    one = std::max(one, gf_pick_bytes(m[j], n[j], k[j], true));
    if (t.parts) all += gf_part_bytes(m[j], n[j], t.split[j]);
  }
  return gf_round(size_t(tokens) * 2 * ff * 2) + std::max(one, all);
}

hipError_t launch_gated_ffn_backward(const GfBwdArgs& a, hipStream_t s) {
  const int M = a.tokens;
  if (M == 0) {
    for (auto [p, n] : {std::pair<uint16_t*, size_t>{a.dw_in, size_t(2) * a.ff * a.d}, {a.dw_down, size_t(a.d) * a.ff}}) {
      if (!p) continue;
      hipLaunchKernelGGL(gf_zero_kernel, dim3(unsigned(std::min<size_t>((n + 2047) / 2048, 1024))), dim3(256), 0, s, p, n);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const uint16_t* h = a.state + size_t(M) * 2 * a.ff;
  uint16_t* dgu = static_cast<uint16_t*>(a.ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + gf_round(size_t(M) * 2 * a.ff * 2));
  hipError_t e = hipSuccess;
  if (a.dx || a.dw_in) {
    GfGemm p{};
    p.a = a.dy;
    p.b = a.w_down;
    p.lda = p.K = a.d;
    p.ldb = p.N = p.ff = a.ff;
    p.M = M;
    p.split = 1;
    p.out = dgu;
    p.pa = const_cast<uint16_t*>(a.state);
    p.fine = reinterpret_cast<uint8_t*>(p.pa + size_t(M) * 3 * a.ff);
    const GfTiling tiling = gf_grad_tiling(M, a.d, a.ff);
    e = gf_tiled<false, true, GF_GRAD>(p, tiling, s);
    if (e != hipSuccess) return e;
  }
  GfGroup g{};
  GfGemm &dx = g.job[0], &dw_in = g.job[1], &dw_down = g.job[2];
  dx.a = dw_in.a = dgu;
  dx.lda = dx.K = dw_in.lda = dw_in.M = 2 * a.ff;
  dx.b = a.w_in;
  dw_in.b = a.x;
  dx.ldb = dx.N = dw_in.ldb = dw_in.N = dw_down.lda = dw_down.M = a.d;
  dx.M = dw_in.K = dw_down.K = M;
  dw_down.a = a.dy;
  dw_down.b = h;
  dw_down.ldb = dw_down.N = a.ff;
  dx.add32 = a.dx_add;
  dx.out = a.dx;
  dw_in.out = a.dw_in;
  dw_down.out = a.dw_down;
  if (const GfTogether t = gf_group_pick(M, a.d, a.ff); t.side) {
    for (int k = 0; k < 3; ++k) {
      g.job[k].split = t.split[k];
      g.job[k].part = part;
      if (t.parts) part += gf_part_bytes(g.job[k].M, g.job[k].N, t.split[k]) / 4;
    }
    if (!t.parts) return t.side == 128 ? gf_group_go<GF_OUT, 128, 64, 2, 2, 2>(g, s) : gf_group_go<GF_OUT, 256, 32, 2, 4, 4>(g, s);
    e = t.side == 128 ? gf_group_go<GF_PART, 128, 64, 2, 2, 2>(g, s) : gf_group_go<GF_PART, 256, 32, 2, 4, 4>(g, s);
    return e != hipSuccess ? e : gf_reduce(g.job, 3, s);
  }
  if (a.dx) e = gf_product<false, true>(dx, part, s);
  if (e == hipSuccess && a.dw_in) e = gf_product<true, true>(dw_in, part, s);
  if (e == hipSuccess && a.dw_down) e = gf_product<true, true>(dw_down, part, s);
  return e;
}

GfPlan gated_ffn_plan(int tokens, int d, int ff) {
  GfPlan p{};
  if (tokens == 0) return p;
  p.few = tokens <= GF_FEW;
  const GfTile y = gf_pick(tokens, d, ff, false, true);
  p.gate = gf_gate_tiling(tokens, d, ff);
  p.y = y.tiling;
  p.y_shares = y.split;
  p.grad = gf_grad_tiling(tokens, d, ff);
  const GfTogether t = gf_group_pick(tokens, d, ff);
  p.joint = t.side != 0;
  p.joint_parts = t.parts;
  int m[3], n[3], k[3];
  gf_three(tokens, d, ff, m, n, k);
  for (int j = 0; j < 3; ++j) {
    const GfTile one = gf_pick(m[j], n[j], k[j], true, true);
    p.last[j] = !t.side ? one.tiling : t.side == 128 ? GF_128_2 : GF_256;
    p.last_shares[j] = t.side ? t.split[j] : one.split;
  }
  return p;
}

}  // namespace bmoe
