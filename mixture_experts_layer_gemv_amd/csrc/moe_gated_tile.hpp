// The tile kernels of the gated feed-forward block (gfx950): one template for
// its five products, in bf16 and fp32 (see moe_gated.hpp for what they compute).
//
// A workgroup of WT x WC waves computes 32 TB WT rows by 32 CB WC channels of one
// expert.  Both operands stream through a ring of S stages in LDS, 128 bytes of
// every line a stage (moe_gated_index.hpp), copied with 16 bytes a lane.  The
// weights take the product's row side (MFMA operand A) and the rows its column
// side, so that a lane's accumulators are consecutive channels of one row.
//
// Plain weights lie with their reduction index outermost in the forward pass
// ([E][K][N]); ds_read_b64_tr_b16 turns four lines into a lane's four steps of
// one column, so no transposed copy of the weights is ever made.  A weight
// gradient reduces over rows, which makes both of its operands of that form.
//
// Reduction steps past the end are copied from a zero block in place of the
// operands, so nothing that lies there, NaN included, reaches a sum.
#pragma once

#include <type_traits>

#include "moe_gated.hpp"
#include "moe_gated_index.hpp"
#include "moe_items.hpp"
#include "moe_lds.hpp"

namespace moe {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct Bf16 {
  static constexpr int ES = 2;
  typedef bf16x8_t Frag;  // eight steps of a lane's row or column
};
struct F32 {
  static constexpr int ES = 4;
  typedef f32x4_t Frag;  // four steps
};

enum class Op { kUp, kDown, kGradHidden, kGradX, kGradW };
constexpr bool rows_by_step(Op op) { return op == Op::kGradW; }
constexpr bool weights_by_step(Op op) { return op == Op::kUp || op == Op::kDown || op == Op::kGradW; }

__device__ __attribute__((aligned(16))) const unsigned char g_zeros[16] = {};

// The operand of 32 rows or columns `block`, quarter ks of a stage.
template <class T, bool STEP>
__device__ __forceinline__ typename T::Frag read_operand(const unsigned char* lines, int block, int ks, int lane) {
  if constexpr (!STEP) {
    return *reinterpret_cast<const typename T::Frag*>(lines + block * 4096 + operand32(lane, ks));
  } else if constexpr (std::is_same<T, Bf16>::value) {
    typedef s16x4_t __attribute__((address_space(3))) * Lds;
    const unsigned char* p =
        lines + (block >> 1) * 8192 + (transposed_read(lane, 0, 0, 0) ^ ((block & 1) << 6)) + ks * 2048;
    const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
    const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 512));
    return __builtin_bit_cast(bf16x8_t, (s16x8_t)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    f32x4_t f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float*>(lines + block * 4096 + step_read_f32(lane, ks, i));
    return f;
  }
}

__device__ __forceinline__ f32x16_t multiply(bf16x8_t w, bf16x8_t x, f32x16_t acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t multiply(f32x4_t w, f32x4_t x, f32x16_t acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(w[i], x[i], acc, 0, 0, 0);
  return acc;
}

// n stages of products into acc.  issue(s, j) copies part j of the wave's Sh::CP
// of stage s.  The last stage holds `quarters` quarters of steps.
//
// Every operand read is issued ahead of the products of the quarter before it,
// across the stages too: a stage's last quarter is multiplied after the barrier
// that frees its ring slot, while the copies into that slot and the next stage's
// first reads are under way; a read or copy follows each product, so that the
// matrix cores do not wait for either to issue.
template <class T, int TB, int CB, int WT, int WC, int S, bool XS, bool WS, bool GATED, class Issue>
__device__ __forceinline__ void reduce_stages(f32x16_t (&acc)[CB][TB], const unsigned char* ring, int n, int quarters,
                                              int wt, int wc, int lane, Issue issue) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  struct Frag {
    typename T::Frag x[TB], w[CB];
  };
  if (n <= 0) return;
  const int last = n - 1;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s <= last)
#pragma unroll
      for (int j = 0; j < Sh::CP; ++j) issue(s, j);
  if (S - 1 <= last) __builtin_amdgcn_s_waitcnt(vmcnt_imm(Sh::CP * (S - 1)));
  else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  ring_barrier();
  auto load_one = [&](Frag& f, int s, int ks, int j) {
    const unsigned char* st = ring + (s % S) * (Sh::XB + Sh::WB);
    if (j < CB) f.w[j] = read_operand<T, WS>(st + Sh::XB, channel_block(GATED, WC, CB, wc, j), ks, lane);
    else f.x[j - CB] = read_operand<T, XS>(st, wt * TB + j - CB, ks, lane);
  };
  constexpr int READS = CB + TB, PRODUCTS = TB * CB;
  // The products of `f` between the reads of `next` (quarter ks of stage s) and,
  // with COPY, the copies of stage cs.
  auto pass = [&](const Frag& f, Frag& next, int s, int ks, auto copy, int cs) {
    constexpr int COPIES = decltype(copy)::value ? Sh::CP : 0;
    constexpr int N = PRODUCTS > READS ? (PRODUCTS > COPIES ? PRODUCTS : COPIES) : (READS > COPIES ? READS : COPIES);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j < READS) load_one(next, s, ks, j);
      if (j < PRODUCTS) acc[j % CB][j / CB] = multiply(f.w[j % CB], f.x[j / CB], acc[j % CB][j / CB]);
      if (j < COPIES) issue(cs, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const std::false_type none{};
  Frag f0, f1;
#pragma unroll
  for (int j = 0; j < READS; ++j) load_one(f0, 0, 0, j);
  int s = 0;
  for (; s + S <= last; ++s) {
    pass(f0, f1, s, 1, none, 0);
    pass(f1, f0, s, 2, none, 0);
    pass(f0, f1, s, 3, none, 0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(Sh::CP * (S - 2)));
    ring_barrier();
    pass(f1, f0, s + 1, 0, std::true_type{}, s + S);
  }
  for (; s < last; ++s) {
    pass(f0, f1, s, 1, none, 0);
    pass(f1, f0, s, 2, none, 0);
    pass(f0, f1, s, 3, none, 0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    ring_barrier();
    pass(f1, f0, s + 1, 0, none, 0);
  }
  for (int ks = 0; ks < quarters; ++ks) {
#pragma unroll
    for (int j = 0; j < READS; ++j) load_one(f0, last, ks, j);
#pragma unroll
    for (int j = 0; j < PRODUCTS; ++j) acc[j % CB][j / CB] = multiply(f0.w[j % CB], f0.x[j / CB], acc[j % CB][j / CB]);
  }
}

// ---- epilogues ---------------------------------------------------------------------

// 16 bytes of consecutive values: eight bf16 or four fp32.
template <class T>
struct Vec {
  static constexpr int N = 16 / T::ES;
  float v[N];
};

template <class T>
__device__ __forceinline__ Vec<T> load_vec(const void* p, size_t i) {
  const u32x4_t r = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p) + i * T::ES);
  Vec<T> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T::ES == 2) {
      f.v[2 * j] = __uint_as_float(r[j] << 16);
      f.v[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
    } else {
      f.v[j] = __uint_as_float(r[j]);
    }
  }
  return f;
}

template <class T>
__device__ __forceinline__ void store_vec(void* p, size_t i, const Vec<T>& f) {
  u32x4_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (T::ES == 2)
      r[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{f.v[2 * j], f.v[2 * j + 1]}, bf16x2_t));
    else
      r[j] = __float_as_uint(f.v[j]);
  }
  *reinterpret_cast<u32x4_t*>(static_cast<char*>(p) + i * T::ES) = r;
}

// 1 / (1 + exp(-g)).  In bf16 the fast exponential and reciprocal, good to 2^-21,
// are well within the output's 2^-9; fp32 takes the exact functions.
template <class T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (T::ES == 2) return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
  else return 1.0f / (1.0f + expf(-g));
}

// Hands out the accumulators of row block i as rows: a wave stages 32 rows of its
// 32 CB channels in LDS as fp32 (rows padded by 16 bytes) and f(row, channel,
// values) gets Vec<T>::N channels at `channel` of the first 32 CH and, where CH
// is less than CB, the same of the second.
template <class T, int TB, int CB, int CH, class F>
__device__ __forceinline__ void each_vec(const f32x16_t (&acc)[CB][TB], int i, unsigned char* stage, int lane, F f) {
  constexpr int STR = 32 * CB * 4 + 16, N = Vec<T>::N;
  constexpr int LPR = 32 * CH / N, RPI = 64 / LPR;  // lanes per row, rows a pass
  unsigned char* const mine = stage + (lane & 31) * STR + 16 * (lane >> 5);
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4_t*>(mine + 128 * c + 32 * g) =
          f32x4_t{acc[c][i][4 * g], acc[c][i][4 * g + 1], acc[c][i][4 * g + 2], acc[c][i][4 * g + 3]};
  // other lanes of the wave wrote what a lane reads (a wave's LDS accesses take
  // place in order; the compiler must keep them so across the types)
  asm volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < 32 / RPI; ++q) {
    const int r = q * RPI + lane / LPR, ch = lane % LPR * N;
    Vec<T> a, b;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(stage + r * STR + 4 * (ch + j));
#pragma unroll
      for (int v = 0; v < 4; ++v) a.v[j + v] = lo[v];
      if constexpr (CH < CB) {
        const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(stage + r * STR + 4 * (32 * CH + ch + j));
#pragma unroll
        for (int v = 0; v < 4; ++v) b.v[j + v] = hi[v];
      }
    }
    f(r, ch, a, b);
  }
  asm volatile("" ::: "memory");
}

// The row range of expert e, as find_item reads the offsets; every lane calls.
__device__ __forceinline__ int2 expert_rows(const int32_t* offsets, int E, int R, int e) {
  if (!offsets) return make_int2(0, R);
  const int lane = threadIdx.x & 63;
  auto clamped = [&](int i) { return min(max(i <= E ? offsets[i] : 0, 0), R); };
  int first = clamped(lane);
  const int next = clamped(lane + 1);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int p = __shfl_up(first, d, 64);
    if (lane >= d) first = max(first, p);
  }
  return make_int2(__builtin_amdgcn_readlane(first, e), __builtin_amdgcn_readlane(max(first, next), e));
}

// ---- products over the experts' rows --------------------------------------------

template <class T, Op OP, int TB, int CB, int WT, int WC, int S>
__global__ __launch_bounds__(WT* WC * 64)
    __attribute__((amdgpu_waves_per_eu(TileShape<TB, CB, WT, WC, S>::per_simd, TileShape<TB, CB, WT, WC, S>::per_simd)))
void k_gated_rows(const GatedArgs A, int cg) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  constexpr bool GATED = OP == Op::kUp, WS = weights_by_step(OP), TWO = OP == Op::kGradX;
  constexpr int ES = T::ES, KD = stage_steps(ES);
  constexpr int BN = GATED ? Sh::BN / 2 : Sh::BN;  // output columns of a tile
  static_assert(!GATED || CB % 2 == 0, "a wave takes gate and up channels");
  static_assert(!WS || BN % KD == 0, "whole column groups");
  __shared__ __attribute__((aligned(1024))) unsigned char ring[S * (Sh::XB + Sh::WB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WC, wc = wave % WC;
  const Item it = find_item(A.offsets, A.E, A.R, Sh::BM, (A.N + BN - 1) / BN, cg, (int)blockIdx.x, true);
  if (it.e < 0) return;
  const int row0 = it.row0, rows = it.rows, n0 = it.nb * BN;

  // Copies: the lines past the tile's last row or column re-read the last one.
  const char* xsrc[Sh::CPX];
  uint32_t wsrc[Sh::CPW];
#pragma unroll
  for (int j = 0; j < Sh::CPX; ++j) {
    int r = row0 + min(8 * (Sh::CPX * wave + j) + (lane >> 3), rows - 1);
    if (A.perm) {
      const int t = A.perm[r] / A.topk;
      r = t < 0 ? 0 : (t >= A.T ? A.T - 1 : t);
    }
    xsrc[j] = static_cast<const char*>(A.x) + (size_t)r * A.K * ES;
  }
#pragma unroll
  for (int j = 0; j < Sh::CPW; ++j) {
    const int i = (8 * (Sh::CPW * wave + j) + (lane >> 3)) % (GATED ? Sh::BN / 2 : Sh::BN);
    if (WS) wsrc[j] = (uint32_t)min((n0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), A.N * ES - 16) +
                      (uint32_t)line_step(i, ES) * (uint32_t)(A.N * ES);
    else wsrc[j] = (uint32_t)min(i, A.N - 1 - n0) * (uint32_t)(A.K * ES);
  }
  const size_t wexpert = (size_t)it.e * A.K * A.N * ES;
  const uint32_t lds0 = lds_address(&ring[0]);
  const int per = (A.K + KD - 1) / KD, n = TWO ? 2 * per : per;  // stages of a term, and in all
  const bool tail = A.K % KD != 0;
  const ptrdiff_t second = TWO ? static_cast<const char*>(A.x2) - static_cast<const char*>(A.x) : 0;
  auto issue = [&](int s, int j) {
    const int term = TWO && s >= per, k0 = (s - (term ? per : 0)) * KD;
    const uint32_t at = lds0 + (uint32_t)(s % S) * (Sh::XB + Sh::WB);
    const bool partial = tail && k0 + KD > A.K;
    if (j < Sh::CPX) {
      const int i = Sh::CPX * wave + j, b = k0 * ES + 16 * chunk_of(i, lane);
      const char* p = xsrc[j] + b + (TWO && term ? second : 0);
      if (partial && b >= A.K * ES) p = reinterpret_cast<const char*>(g_zeros);
      copy_at(p, at + i * 1024);
    } else {
      const int jw = j - Sh::CPX, i = Sh::CPW * wave + jw;
      const bool up = GATED && 8 * i >= Sh::BN / 2;
      const char* base = static_cast<const char*>(TWO ? A.w[term] : A.w[up ? 1 : 0]) + wexpert;
      const uint32_t to = at + Sh::XB + i * 1024;
      if (WS) {
        base += (size_t)k0 * A.N * ES;
        if (!partial) copy_frag(base, wsrc[jw], to);
        else copy_at(k0 + line_step(8 * i + (lane >> 3), ES) < A.K ? base + wsrc[jw] : reinterpret_cast<const char*>(g_zeros), to);
      } else {
        base += (size_t)n0 * A.K * ES + (size_t)k0 * ES;
        const int c = 16 * chunk_of(i, lane);
        if (!partial) copy_frag(base, wsrc[jw] + c, to);
        else copy_at(k0 * ES + c < A.K * ES ? base + wsrc[jw] + c : reinterpret_cast<const char*>(g_zeros), to);
      }
    }
  };

  f32x16_t acc[CB][TB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][i][v] = 0.0f;
  const int left = A.K - (per - 1) * KD;
  reduce_stages<T, TB, CB, WT, WC, S, false, WS, GATED>(acc, ring, n, (left + KD / 4 - 1) / (KD / 4), wt, wc, lane, issue);
  __syncthreads();  // the ring is free

  constexpr int CH = GATED ? CB / 2 : CB, N = Vec<T>::N;
  unsigned char* const stage = ring + wave * 32 * (32 * CB * 4 + 16);
  const int nw = n0 + 32 * CH * wc;  // the wave's first output column
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int rb = (wt * TB + i) * 32;
    if (rb >= rows) break;
    each_vec<T, TB, CB, CH>(acc, i, stage, lane, [&](int r, int ch, const Vec<T>& a, const Vec<T>& b) {
      if (rb + r >= rows || nw + ch >= A.N) return;
      const size_t at = (size_t)(row0 + rb + r) * A.N + nw + ch;
      if constexpr (OP == Op::kUp) {
        Vec<T> h;
#pragma unroll
        for (int j = 0; j < N; ++j) h.v[j] = a.v[j] * sigmoid<T>(a.v[j]) * b.v[j];
        store_vec<T>(A.out[0], at, h);
        if (A.out[1]) store_vec<T>(A.out[1], at, a);
        if (A.out[2]) store_vec<T>(A.out[2], at, b);
      } else if constexpr (OP == Op::kGradHidden) {
        // h = g s u with s = sigmoid(g): dg = dh u s (1 + g (1 - s)), du = dh g s
        const Vec<T> g = load_vec<T>(A.in[0], at), u = load_vec<T>(A.in[1], at);
        Vec<T> dg, du, h;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float s = sigmoid<T>(g.v[j]), gs = g.v[j] * s;
          h.v[j] = gs * u.v[j];
          du.v[j] = a.v[j] * gs;
          dg.v[j] = a.v[j] * u.v[j] * (s + gs * (1.0f - s));
        }
        store_vec<T>(A.out[0], at, dg);
        store_vec<T>(A.out[1], at, du);
        if (A.out[2]) store_vec<T>(A.out[2], at, h);
      } else {
        store_vec<T>(A.out[0], at, a);
      }
    });
  }
}

// ---- weight gradients ----------------------------------------------------------------

template <class T, int TB, int CB, int WT, int WC, int S>
__global__ __launch_bounds__(WT* WC * 64)
    __attribute__((amdgpu_waves_per_eu(TileShape<TB, CB, WT, WC, S>::per_simd, TileShape<TB, CB, WT, WC, S>::per_simd)))
void k_gated_grad_w(const GradWArgs A, int cg, int per_expert) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  constexpr int ES = T::ES, KD = stage_steps(ES);
  __shared__ __attribute__((aligned(1024))) unsigned char ring[S * (Sh::XB + Sh::WB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WC, wc = wave % WC;
  // the item: expert, problem, tile
  const int L = xcd_item((int)blockIdx.x, per_expert * A.E, 0);
  if (L < 0) return;
  const int e = L / per_expert;
  int li = L - e * per_expert, q = 0, MB = 0, NB = 0;
  for (;; ++q) {
    MB = (A.p[q].M + Sh::BM - 1) / Sh::BM;
    NB = (A.p[q].N + Sh::BN - 1) / Sh::BN;
    if (li < MB * NB || q + 1 >= A.n) break;
    li -= MB * NB;
  }
  const GradWProblem& P = A.p[q];
  const int g = li / (MB * cg), rem = li - g * MB * cg, gw = min(NB - g * cg, cg);
  const int m0 = rem / gw * Sh::BM, n0 = (g * cg + rem % gw) * Sh::BN;
  const int2 range = expert_rows(A.offsets, A.E, A.R, e);
  const int lo = range.x, K = range.y - range.x;

  uint32_t xsrc[Sh::CPX], wsrc[Sh::CPW];
#pragma unroll
  for (int j = 0; j < Sh::CPX; ++j) {
    const int i = 8 * (Sh::CPX * wave + j) + (lane >> 3);
    xsrc[j] = (uint32_t)min((m0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), P.M * ES - 16) +
              (uint32_t)line_step(i, ES) * (uint32_t)(P.M * ES);
  }
#pragma unroll
  for (int j = 0; j < Sh::CPW; ++j) {
    const int i = 8 * (Sh::CPW * wave + j) + (lane >> 3);
    wsrc[j] = (uint32_t)min((n0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), P.N * ES - 16) +
              (uint32_t)line_step(i, ES) * (uint32_t)(P.N * ES);
  }
  const uint32_t lds0 = lds_address(&ring[0]);
  auto issue = [&](int s, int j) {
    const int k0 = s * KD;
    const bool x = j < Sh::CPX;
    const int i = x ? Sh::CPX * wave + j : Sh::CPW * wave + j - Sh::CPX;
    const char* base = static_cast<const char*>(x ? P.x : P.w) + (size_t)(lo + k0) * (x ? P.M : P.N) * ES;
    const uint32_t from = x ? xsrc[x ? j : 0] : wsrc[x ? 0 : j - Sh::CPX];
    const uint32_t to = lds0 + (uint32_t)(s % S) * (Sh::XB + Sh::WB) + (x ? 0 : Sh::XB) + i * 1024;
    if (k0 + KD <= K) copy_frag(base, from, to);
    else copy_at(k0 + line_step(8 * i + (lane >> 3), ES) < K ? base + from : reinterpret_cast<const char*>(g_zeros), to);
  };

  f32x16_t acc[CB][TB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][i][v] = 0.0f;
  const int n = (K + KD - 1) / KD, left = K - (n - 1) * KD;
  reduce_stages<T, TB, CB, WT, WC, S, true, true, false>(acc, ring, n, (left + KD / 4 - 1) / (KD / 4), wt, wc, lane, issue);
  __syncthreads();

  unsigned char* const stage = ring + wave * 32 * (32 * CB * 4 + 16);
  const int nw = n0 + 32 * CB * wc;
  const size_t out0 = (size_t)e * P.M * P.N;
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int rb = m0 + (wt * TB + i) * 32;
    if (rb >= P.M) break;
    each_vec<T, TB, CB, CB>(acc, i, stage, lane, [&](int r, int ch, const Vec<T>& a, const Vec<T>&) {
      if (rb + r < P.M && nw + ch < P.N) store_vec<T>(P.out, out0 + (size_t)(rb + r) * P.N + nw + ch, a);
    });
  }
}

// ---- launches --------------------------------------------------------------------------

// Upper bound on the row blocks of BM rows.
inline long long row_blocks(const GatedArgs& a, int BM) {
  return a.offsets ? (long long)a.R / BM + (a.R < a.E ? a.R : a.E) : ((long long)a.R + BM - 1) / BM;
}

template <class T, Op OP, int TB, int CB, int WT, int WC, int S>
hipError_t launch_tile(const GatedArgs& a, int cg, hipStream_t s) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  constexpr int BN = OP == Op::kUp ? Sh::BN / 2 : Sh::BN;
  const long long blocks = row_blocks(a, Sh::BM) * ((a.N + BN - 1) / BN);
  if ((blocks + 8) * WT * WC * 64 >= 1LL << 32) return hipErrorInvalidValue;
  k_gated_rows<T, OP, TB, CB, WT, WC, S><<<(unsigned)((blocks + 7) / 8 * 8), WT * WC * 64, 0, s>>>(a, cg);
  return hipGetLastError();
}

template <class T, int TB, int CB, int WT, int WC, int S>
hipError_t launch_grad_w_tile(const GradWArgs& a, int cg, hipStream_t s) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  long long per = 0;
  for (int i = 0; i < a.n; ++i)
    per += (long long)((a.p[i].M + Sh::BM - 1) / Sh::BM) * ((a.p[i].N + Sh::BN - 1) / Sh::BN);
  const long long blocks = per * a.E;
  if ((blocks + 8) * WT * WC * 64 >= 1LL << 32) return hipErrorInvalidValue;
  k_gated_grad_w<T, TB, CB, WT, WC, S><<<(unsigned)((blocks + 7) / 8 * 8), WT * WC * 64, 0, s>>>(a, cg, (int)per);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe
