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
//
// What bounds it: large products (256 x 256 tiles, two waves per SIMD, 128 x 64 each)
// the card's power: 16384 x 4096 x 28672 (gate and up) 2.93 ms, 1.31 PFLOP/s, at about
// 1.65 GHz; over the rows of 8 experts 3.2 ms, over 16 experts' rows 10 to 20 % less, for
// the rows that their last row blocks lack.  Few rows (32-row tiles) their weights'
// bytes: 6.0 to 6.4 TB/s from HBM.  fp32 its products (135 TFLOP/s at 4096 x 2048 x 8192).
// fp32 in small tiles no one resource (333 tokens, top-3 of 12, 1000 x 1720: gate and up 90
// us, down 52): of the CUs' busy cycles the matrix pipe has 73 and 62 %, a sixth of it rows past
// an expert's last; LDS reads take a tenth of the time, and the waves wait for 15 and 23 %
// of theirs, for copies that two stages give one stage's time to arrive; and the launch, about
// one round of tiles, keeps the CUs busy for 83 and 77 % of it.
#pragma once

#include <cstddef>
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

// global -> LDS, 16 bytes a lane from 64-bit addresses (see copy_frag).
__device__ __forceinline__ void copy_at(const void* p, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(p), "s"(lds)
      : "memory");
}

// copy_frag of a line that nothing reads again: not kept in the caches.
__device__ __forceinline__ void copy_frag_once(const void* sbase, uint32_t voff, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2 nt\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(voff), "s"(sbase), "s"(lds)
      : "memory");
}

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

// A tile's buffers.  PAIR: each of its 32 rows has two lines, the high and the low part
// of its values.
template <int TB, int CB, int WT, int WC, int S, bool PAIR>
using RowsShape = TileShape<PAIR ? 2 : TB, CB, WT, WC, S>;

// The stages of a reduction that a workgroup takes: [lo, hi) of TERMS reductions
// of `per` stages, one after the other; with tail each one's last stage ends past
// the reduction (is partial) and holds `quarters` quarters of steps.
struct Stages {
  int lo, hi, per;
  bool tail;
  int quarters;
};
__device__ __forceinline__ Stages stages_of(int K, int KD, int terms) {
  const int per = (K + KD - 1) / KD, left = K - (per - 1) * KD;
  return {0, per * terms, per, left != KD, (left + KD / 4 - 1) / (KD / 4)};
}

__device__ __forceinline__ Stages share_of(Stages st, int split, int splits) {
  const int all = st.hi;
  st.lo = (int)((long long)all * split / splits);
  st.hi = (int)((long long)all * (split + 1) / splits);
  return st;
}

// The products of a workgroup's stages into acc.  at(s) is what the copies of stage
// s start from; issue(at, slot, j, partial) makes copy j of the wave's Sh::CP.
// live: the wave's row blocks that hold rows (an expert's last tile); the others are
// not read or multiplied, and a wave without any only copies.
//
// Every operand read is issued ahead of the products of the quarter before it,
// across the stages too: a stage's last quarter is multiplied after the barrier
// that frees its ring slot, while the copies into that slot and the next stage's
// first reads are under way; a read or copy follows each product, so that the
// matrix cores do not wait for either to issue.
template <class T, int TB, int CB, int WT, int WC, int S, bool XS, bool WS, bool GATED, bool PAIR, int TERMS, int LIVE, class At, class Issue>
__device__ __forceinline__ void reduce_live(f32x16_t (&acc)[CB][TB], const unsigned char* ring, const Stages& st, int wt,
                                            int wc, int lane, At at, Issue issue) {
  using Sh = RowsShape<TB, CB, WT, WC, S, PAIR>;
  constexpr int XB = PAIR ? 2 : LIVE;  // operands of rows; a pair's are multiplied into the same sums
  struct Frag {
    typename T::Frag x[XB ? XB : 1], w[CB];
  };
  const int n = st.hi - st.lo, last = n - 1;
  auto load_one = [&](Frag& f, int s, int ks, int j) {
    const unsigned char* slot = ring + (s % S) * (Sh::XB + Sh::WB);
    if (j < CB) f.w[j] = read_operand<T, WS>(slot + Sh::XB, channel_block(GATED, WC, CB, wc, j), ks, lane);
    else f.x[j - CB] = read_operand<T, XS>(slot, wt * TB + j - CB, ks, lane);
  };
  constexpr int READS = XB ? CB + XB : 0, PRODUCTS = XB * CB;
  auto product = [&](const Frag& f, int j) {
    f32x16_t& sum = acc[j % CB][PAIR ? 0 : j / CB];
    sum = multiply(f.w[j % CB], f.x[j / CB], sum);
  };
  // The products of `f` between the reads of `next` (quarter ks of stage s) and
  // the copies that `copy` makes.
  auto pass = [&](const Frag& f, Frag& next, int s, int ks, auto copy) {
    constexpr int COPIES = std::is_same<decltype(copy), std::nullptr_t>::value ? 0 : Sh::CP;
    constexpr int N = PRODUCTS > READS ? (PRODUCTS > COPIES ? PRODUCTS : COPIES) : (READS > COPIES ? READS : COPIES);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j < READS) load_one(next, s, ks, j);
      if (j < PRODUCTS) product(f, j);
      if constexpr (COPIES > 0)
        if (j < COPIES) copy(j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  Frag f0, f1;
#pragma unroll
  for (int j = 0; j < READS; ++j) load_one(f0, 0, 0, j);
  // stage c - S is multiplied while stage c is copied
  auto turn = [&](int c, auto partial) {
    const int s = c - S;
    pass(f0, f1, s, 1, nullptr);
    pass(f1, f0, s, 2, nullptr);
    pass(f0, f1, s, 3, nullptr);
    const auto a = at(st.lo + c);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(Sh::CP * (S - 2)));
    ring_barrier();
    pass(f1, f0, s + 1, 0, [&](int j) { issue(a, c % S, j, partial); });
  };
  int c = S;
  for (int term = 1; term <= TERMS; ++term) {
    const int whole = term * st.per - (st.tail ? 1 : 0) - st.lo, end = whole < n ? whole : n;
    for (; c < end; ++c) turn(c, std::false_type{});
    if (st.tail && c == whole && c < n) turn(c++, std::true_type{});
  }
  for (int s = c - S > 0 ? c - S : 0; s < last; ++s) {
    pass(f0, f1, s, 1, nullptr);
    pass(f1, f0, s, 2, nullptr);
    pass(f0, f1, s, 3, nullptr);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    ring_barrier();
    pass(f1, f0, s + 1, 0, nullptr);
  }
  const int quarters = st.hi % st.per ? 4 : st.quarters;
  for (int ks = 0; ks < quarters; ++ks) {
#pragma unroll
    for (int j = 0; j < READS; ++j) load_one(f0, last, ks, j);
#pragma unroll
    for (int j = 0; j < PRODUCTS; ++j) product(f0, j);
  }
}

template <class T, int TB, int CB, int WT, int WC, int S, bool XS, bool WS, bool GATED, bool PAIR, int TERMS, class At, class Issue>
__device__ __forceinline__ void reduce_stages(f32x16_t (&acc)[CB][TB], const unsigned char* ring, const Stages& st, int live,
                                              int wt, int wc, int lane, At at, Issue issue) {
  using Sh = RowsShape<TB, CB, WT, WC, S, PAIR>;
  const int n = st.hi - st.lo;
  if (n <= 0) return;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < n) {
      const auto a = at(st.lo + s);
      if (st.tail && (st.lo + s + 1) % st.per == 0) {
#pragma unroll
        for (int j = 0; j < Sh::CP; ++j) issue(a, s, j, std::true_type{});
      } else {
#pragma unroll
        for (int j = 0; j < Sh::CP; ++j) issue(a, s, j, std::false_type{});
      }
    }
  if (S <= n) __builtin_amdgcn_s_waitcnt(vmcnt_imm(Sh::CP * (S - 1)));
  else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  ring_barrier();
  auto go = [&](auto l) {
    reduce_live<T, TB, CB, WT, WC, S, XS, WS, GATED, PAIR, TERMS, decltype(l)::value>(acc, ring, st, wt, wc, lane, at, issue);
  };
  if (PAIR || live >= TB) go(std::integral_constant<int, TB>{});
  else if (live <= 0) go(std::integral_constant<int, 0>{});
  else if (TB == 4 && live == 3) go(std::integral_constant<int, TB == 4 ? 3 : 1>{});
  else if (TB == 4 && live == 2) go(std::integral_constant<int, TB == 4 ? 2 : 1>{});
  else go(std::integral_constant<int, 1>{});
}

// ---- epilogues ---------------------------------------------------------------------

// 16 bytes of consecutive values: eight bf16 or four fp32.
template <class T>
struct Vec {
  static constexpr int N = 16 / T::ES;
  float v[N];
};

template <class T>
__device__ __forceinline__ Vec<T> to_vec(u32x4_t r) {
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

// What one product hands to the next is an operand of the bf16 matrix cores there, and so
// is rounded to bf16.  With `low`, what the rounding of f takes off is stored as well, `low`
// bytes further on: the two parts hold 16 bits of a value.  They double the products that take
// them, 6 R m p operations to 8 forwards and 12 to 22 backwards, which is free where the
// weights' bytes bound the time (gated_pairs) and would cost their share where the products
// do; there a hidden value keeps bf16's 8 bits, as in the packed experts, and an output is off
// by 0.0023 of its size in place of 0.0017, which one rounding leaves.
template <class T>
__device__ __forceinline__ void store_parts(void* p, size_t i, const Vec<T>& f, ptrdiff_t low) {
  store_vec<T>(p, i, f);
  if constexpr (T::ES == 2) {
    if (!low) return;
    Vec<T> rest;
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
      const float high = (float)(__bf16)f.v[j];
      rest.v[j] = fabsf(high) < INFINITY ? f.v[j] - high : 0.0f;
    }
    store_vec<T>(static_cast<char*>(p) + low, i, rest);
  }
}

// 1 / (1 + exp(-g)).  In bf16 the fast exponential and reciprocal: within (2 |g| + 8)
// 2^-24 of the value, where the outputs' half step is 2^-8; fp32 takes the exact functions.
template <class T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (T::ES == 2) return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
  else return 1.0f / (1.0f + expf(-g));
}

// How a wave takes the 32 rows of a block of 32 CH channels, 16 bytes of outputs a
// lane: in pass q of PASSES a lane has row q RPI + lane / LPR, channel N (lane % LPR).
template <class T, int CH>
struct RowWalk {
  static constexpr int N = Vec<T>::N, LPR = 32 * CH / N, RPI = 64 / LPR, PASSES = 32 / RPI;
  static __device__ __forceinline__ int row(int q, int lane) { return q * RPI + lane / LPR; }
  static __device__ __forceinline__ int channel(int lane) { return lane % LPR * N; }
};

// Hands out the accumulators of row block i as rows: a wave stages 32 rows of its
// 32 CB channels in LDS as fp32 (rows padded by 16 bytes) and f(pass, row, channel,
// values) gets Vec<T>::N channels at `channel` of the first 32 CH and, where CH
// is less than CB, the same of the second.
template <class T, int TB, int CB, int CH, class F>
__device__ __forceinline__ void each_vec(const f32x16_t (&acc)[CB][TB], int i, unsigned char* stage, int lane, F f) {
  using Walk = RowWalk<T, CH>;
  constexpr int STR = 32 * CB * 4 + 16, N = Vec<T>::N;
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
  for (int q = 0; q < Walk::PASSES; ++q) {
    const int r = Walk::row(q, lane), ch = Walk::channel(lane);
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
    f(q, r, ch, a, b);
  }
  asm volatile("" ::: "memory");
}

// The row range of expert e, as find_item reads the offsets; every lane calls.
__device__ __forceinline__ int2 expert_rows(const int32_t* offsets, int E, int R, int e) {
  if (!offsets) return make_int2(0, R);
  const int lane = threadIdx.x & 63;
  auto clamped = [&](int i) { return min(max(i <= E ? offsets[i] : 0, 0), R); };
  const int first = scan_max(clamped(lane)), next = clamped(lane + 1);
  return make_int2(__builtin_amdgcn_readlane(first, e), __builtin_amdgcn_readlane(max(first, next), e));
}

// ---- products over the experts' rows --------------------------------------------

// What an output's element `at` takes from memory besides its sums: gate and up for
// the hidden gradients.
struct Saved {
  u32x4_t gate, up;
};
template <Op OP, int ES>
__device__ __forceinline__ Saved load_saved(const GatedArgs& A, size_t at) {
  if constexpr (OP == Op::kGradHidden)
    return {*reinterpret_cast<const u32x4_t*>(static_cast<const char*>(A.in[0]) + at * ES),
            *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(A.in[1]) + at * ES)};
  else return {};
}

// The outputs at element `at` from its sums (gated: a gate's, b up's).
template <class T, Op OP>
__device__ __forceinline__ void finish(const GatedArgs& A, size_t at, const Vec<T>& a, const Vec<T>& b, const Saved& saved) {
  constexpr int V = Vec<T>::N;
  if constexpr (OP == Op::kUp) {
    Vec<T> h;
#pragma unroll
    for (int j = 0; j < V; ++j) h.v[j] = a.v[j] * sigmoid<T>(a.v[j]) * b.v[j];
    store_parts<T>(A.out[0], at, h, A.low);
    if (A.out[1]) store_vec<T>(A.out[1], at, a);
    if (A.out[2]) store_vec<T>(A.out[2], at, b);
  } else if constexpr (OP == Op::kGradHidden) {
    // h = g s u with s = sigmoid(g): dg = dh u s (1 + g (1 - s)), du = dh g s
    const Vec<T> g = to_vec<T>(saved.gate), u = to_vec<T>(saved.up);
    Vec<T> dg, du, h;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float s = sigmoid<T>(g.v[j]), gs = g.v[j] * s;
      h.v[j] = gs * u.v[j];
      du.v[j] = a.v[j] * gs;
      dg.v[j] = a.v[j] * u.v[j] * (s + gs * (1.0f - s));
    }
    store_parts<T>(A.out[0], at, dg, A.low);
    store_parts<T>(A.out[1], at, du, A.low);
    if (A.out[2]) store_parts<T>(A.out[2], at, h, A.low);
  } else {
    store_vec<T>(A.out[0], at, a);
  }
}

// Joins a split reduction: the partial sums added in order, then the outputs.
// The experts' ranges follow one another (find_item), so a row has an expert if it
// lies between the first range's start and the last one's end.
template <class T, Op OP>
__global__ __launch_bounds__(256) void k_gated_join(const GatedArgs A, int splits) {
  constexpr int V = Vec<T>::N;
  constexpr bool GATED = OP == Op::kUp;
  int lo = 0, hi = A.R;
  if (A.offsets) {
    const int lane = threadIdx.x & 63;
    lo = min(max(A.offsets[0], 0), A.R);
    hi = min(max(A.offsets[min(lane, A.E)], 0), A.R);
    hi = max(hi, min(max(A.offsets[A.E], 0), A.R));
    for (int d = 1; d < 64; d <<= 1) hi = max(hi, __shfl_xor(hi, d, 64));
  }
  const int vecs = A.N / V, lines = GATED ? 2 * A.N : A.N;
  const size_t step = (size_t)A.R * lines;
  const long long n = (long long)(hi - lo) * vecs;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256LL * gridDim.x) {
    const int r = lo + (int)(i / vecs), c = (int)(i % vecs) * V;
    const float* p = A.part + (size_t)r * lines + c;
    Vec<T> a = {}, b = {};
    for (int k = 0; k < splits; ++k, p += step)
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(p + j);
#pragma unroll
        for (int v = 0; v < 4; ++v) a.v[j + v] += f[v];
        if constexpr (GATED) {
          const f32x4_t g = *reinterpret_cast<const f32x4_t*>(p + A.N + j);
#pragma unroll
          for (int v = 0; v < 4; ++v) b.v[j + v] += g[v];
        }
      }
    const size_t at = (size_t)r * A.N + c;
    finish<T, OP>(A, at, a, b, load_saved<OP, T::ES>(A, at));
  }
}

// ONCE: the weights are not kept in the caches.  PAIR: the rows come in two parts
// (GatedArgs::low), whose products the same sums take.
template <class T, Op OP, int TB, int CB, int WT, int WC, int S, bool ONCE, bool PAIR>
__global__ __launch_bounds__(WT* WC * 64)
    __attribute__((amdgpu_waves_per_eu(RowsShape<TB, CB, WT, WC, S, PAIR>::per_simd,
                                       RowsShape<TB, CB, WT, WC, S, PAIR>::per_simd)))
void k_gated_rows(const GatedArgs A, int cg, int splits, int cut) {
  using Sh = RowsShape<TB, CB, WT, WC, S, PAIR>;
  static_assert(!PAIR || (TB == 1 && WT == 1), "the pair's lines follow one another");
  constexpr int BM = 32 * TB * WT;  // rows of a tile
  constexpr bool GATED = OP == Op::kUp, WS = weights_by_step(OP), TWO = OP == Op::kGradX;
  constexpr int ES = T::ES, KD = stage_steps(ES);
  constexpr int BN = GATED ? Sh::BN / 2 : Sh::BN;  // output columns of a tile
  static_assert(!GATED || CB % 2 == 0, "a wave takes gate and up channels");
  static_assert(!WS || BN % KD == 0, "whole column groups");
  __shared__ __attribute__((aligned(1024))) unsigned char ring[S * (Sh::XB + Sh::WB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WC, wc = wave % WC;
  const int items = (int)gridDim.x / splits, split = (int)blockIdx.x / items;
  const Item it = find_item(A.offsets, A.E, A.R, BM, (A.N + BN - 1) / BN, cg, (int)blockIdx.x - split * items, true, BM == 256 ? cut : 0);
  if (it.e < 0) return;
  const int row0 = it.row0, rows = it.rows, n0 = it.nb * BN;

  // Copies: the lines past the tile's last row or column re-read the last one.
  const int K = A.K, N = A.N;
  const char* xsrc[Sh::CPX];
  uint32_t wsrc[Sh::CPW];
#pragma unroll
  for (int j = 0; j < Sh::CPX; ++j) {
    const int i = Sh::CPX * wave + j;
    int r = row0 + min((8 * i + (lane >> 3)) % BM, rows - 1);
    if (A.perm) {
      const int t = A.perm[r] / A.topk;
      r = t < 0 ? 0 : (t >= A.T ? A.T - 1 : t);
    }
    xsrc[j] = static_cast<const char*>(A.x) + (size_t)r * K * ES + 16 * chunk_of(i, lane);
    if (PAIR && 8 * i >= BM) xsrc[j] += A.low;
  }
#pragma unroll
  for (int j = 0; j < Sh::CPW; ++j) {
    const int c = Sh::CPW * wave + j, i = (8 * c + (lane >> 3)) % (GATED ? Sh::BN / 2 : Sh::BN);
    if (WS) wsrc[j] = (uint32_t)min((n0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), N * ES - 16) +
                      (uint32_t)line_step(i, ES) * (uint32_t)(N * ES);
    else wsrc[j] = (uint32_t)min(i, N - 1 - n0) * (uint32_t)(K * ES) + 16 * chunk_of(c, lane);
  }
  const uint32_t lds0 = lds_address(&ring[0]);
  Stages st = stages_of(K, KD, TWO ? 2 : 1);
  if (splits > 1) st = share_of(st, split, splits);
  const size_t wstart = ((size_t)it.e * N * K + (WS ? 0 : (size_t)n0 * K)) * ES;
  const char* const w0 = static_cast<const char*>(A.w[0]) + wstart;
  const char* const w1 = GATED || TWO ? static_cast<const char*>(A.w[1]) + wstart : nullptr;
  const ptrdiff_t second = TWO ? static_cast<const char*>(A.x2) - static_cast<const char*>(A.x) : 0;
  struct At {
    const char *w, *up;  // the stage's weights (gated: gate's and up's)
    ptrdiff_t x;         // and the offset of the rows' pointers
    int k0;
  };
  auto at = [&](int s) {
    const bool term = TWO && s >= st.per;
    At a;
    a.k0 = (s - (term ? st.per : 0)) * KD;
    const size_t off = WS ? (size_t)a.k0 * N * ES : (size_t)a.k0 * ES;
    a.w = (term ? w1 : w0) + off;
    a.up = GATED ? w1 + off : nullptr;
    a.x = (ptrdiff_t)a.k0 * ES + (term ? second : 0);
    return a;
  };
  auto issue = [&](const At& a, int slot, int j, auto partial) {
    constexpr bool PART = decltype(partial)::value;
    const char* const zeros = reinterpret_cast<const char*>(g_zeros);
    const uint32_t to = lds0 + (uint32_t)slot * (Sh::XB + Sh::WB);
    if (j < Sh::CPX) {
      const int i = Sh::CPX * wave + j;
      const char* p = xsrc[j] + a.x;
      if (PART && a.k0 * ES + 16 * chunk_of(i, lane) >= K * ES) p = zeros;
      copy_at(p, to + i * 1024);
    } else {
      const int jw = j - Sh::CPX, i = Sh::CPW * wave + jw;
      const char* base = GATED && 8 * i >= Sh::BN / 2 ? a.up : a.w;
      if constexpr (!PART) {
        if constexpr (ONCE) copy_frag_once(base, wsrc[jw], to + Sh::XB + i * 1024);
        else copy_frag(base, wsrc[jw], to + Sh::XB + i * 1024);
      } else {
        const bool in = WS ? a.k0 + line_step(8 * i + (lane >> 3), ES) < K : a.k0 * ES + 16 * chunk_of(i, lane) < K * ES;
        copy_at(in ? base + wsrc[jw] : zeros, to + Sh::XB + i * 1024);
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
  const int live = (rows - wt * TB * 32 + 31) >> 5;
  reduce_stages<T, TB, CB, WT, WC, S, false, WS, GATED, PAIR, TWO ? 2 : 1>(acc, ring, st, live, wt, wc, lane, at, issue);
  __syncthreads();  // the ring is free

  constexpr int CH = GATED ? CB / 2 : CB;
  unsigned char* const stage = ring + wave * 32 * (32 * CB * 4 + 16);
  const int nw = n0 + 32 * CH * wc;  // the wave's first output column
  using Walk = RowWalk<T, CH>;
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int rb = (wt * TB + i) * 32;
    if (rb >= rows) break;
    if (splits > 1) {  // fp32 partial sums, a row's gate and then its up
      const int lines = GATED ? 2 * N : N;
      float* const part = A.part + ((size_t)split * A.R + row0) * lines;
      each_vec<F32, TB, CB, CB>(acc, i, stage, lane, [&](int, int r, int ch, const Vec<F32>& a, const Vec<F32>&) {
        const int col = nw + (GATED ? ch % (32 * CH) : ch);
        if (rb + r < rows && col < N)
          store_vec<F32>(part, (size_t)(rb + r) * lines + col + (GATED && ch >= 32 * CH ? N : 0), a);
      });
      continue;
    }
    // gate and up of the whole row block are loaded together (hidden gradients of 16384
    // rows, 4096 x 6400: 955 us with a wait in each pass, so 948)
    Saved saved[Walk::PASSES] = {};
    if constexpr (OP == Op::kGradHidden)
#pragma unroll
      for (int q = 0; q < Walk::PASSES; ++q) {
        const int r = min(rb + Walk::row(q, lane), rows - 1), c = min(nw + Walk::channel(lane), N - Vec<T>::N);
        saved[q] = load_saved<OP, T::ES>(A, (size_t)(row0 + r) * N + c);
      }
    each_vec<T, TB, CB, CH>(acc, i, stage, lane, [&](int q, int r, int ch, const Vec<T>& a, const Vec<T>& b) {
      if (rb + r >= rows || nw + ch >= N) return;
      const size_t at = (size_t)(row0 + rb + r) * N + nw + ch;
      finish<T, OP>(A, at, a, b, saved[q]);
    });
  }
}

// ---- weight gradients ----------------------------------------------------------------
//
// An expert's rows are the reduction, so each expert has one of its own length; a tile of
// every matrix of every expert, zeros where it has no rows.  16384 rows of 2 experts, three
// gradients of 4096 x 6400: 2.09 ms, 1.23 PFLOP/s; of 16 experts 2.43 ms: a fifth of a
// tile's time goes into its ends.

// PAIR: the hidden operand comes in two parts (GradWProblem::x2, w2), a reduction each.
template <class T, int TB, int CB, int WT, int WC, int S, bool PAIR>
__global__ __launch_bounds__(WT* WC * 64)
    __attribute__((amdgpu_waves_per_eu(TileShape<TB, CB, WT, WC, S>::per_simd, TileShape<TB, CB, WT, WC, S>::per_simd)))
void k_gated_grad_w(const GradWArgs A, int cg, int per_expert, int splits) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  constexpr int ES = T::ES, KD = stage_steps(ES);
  __shared__ __attribute__((aligned(1024))) unsigned char ring[S * (Sh::XB + Sh::WB)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WC, wc = wave % WC;
  // the item: expert, problem, tile
  const int items = (int)gridDim.x / splits, split = (int)blockIdx.x / items;
  const ExpertItem it = expert_item((int)blockIdx.x - split * items, per_expert);
  const int e = it.e;
  if (e >= A.E) return;
  int li = it.tile, q = 0, MB = 0, NB = 0;
  for (;; ++q) {
    MB = (A.problem[q].M + Sh::BM - 1) / Sh::BM;
    NB = (A.problem[q].N + Sh::BN - 1) / Sh::BN;
    if (li < MB * NB || q + 1 >= A.n) break;
    li -= MB * NB;
  }
  const GradWProblem P = A.problem[q];
  const int M = P.M, N = P.N;
  const int g = li / (MB * cg), rem = li - g * MB * cg, gw = min(NB - g * cg, cg);
  const int m0 = rem / gw * Sh::BM, n0 = (g * cg + rem % gw) * Sh::BN;
  const int2 range = expert_rows(A.offsets, A.E, A.R, e);
  const int lo = range.x, K = range.y - range.x;

  uint32_t xsrc[Sh::CPX], wsrc[Sh::CPW];
#pragma unroll
  for (int j = 0; j < Sh::CPX; ++j) {
    const int i = 8 * (Sh::CPX * wave + j) + (lane >> 3);
    xsrc[j] = (uint32_t)min((m0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), M * ES - 16) +
              (uint32_t)line_step(i, ES) * (uint32_t)(M * ES);
  }
#pragma unroll
  for (int j = 0; j < Sh::CPW; ++j) {
    const int i = 8 * (Sh::CPW * wave + j) + (lane >> 3);
    wsrc[j] = (uint32_t)min((n0 + line_group(i, ES) * KD) * ES + 16 * step_chunk(lane), N * ES - 16) +
              (uint32_t)line_step(i, ES) * (uint32_t)(N * ES);
  }
  const uint32_t lds0 = lds_address(&ring[0]);
  Stages st = stages_of(K, KD, PAIR ? 2 : 1);
  if (splits > 1) st = share_of(st, split, splits);
  const char* const x0 = static_cast<const char*>(P.x) + (size_t)lo * M * ES;
  const char* const w0 = static_cast<const char*>(P.w) + (size_t)lo * N * ES;
  const char* const x1 = PAIR ? static_cast<const char*>(P.x2) + (size_t)lo * M * ES : nullptr;
  const char* const w1 = PAIR ? static_cast<const char*>(P.w2) + (size_t)lo * N * ES : nullptr;
  struct At {
    const char *x, *w;
    int k0;
  };
  auto at = [&](int s) {
    const bool second = PAIR && s >= st.per;
    const int k0 = (s - (second ? st.per : 0)) * KD;
    return At{(second ? x1 : x0) + (size_t)k0 * M * ES, (second ? w1 : w0) + (size_t)k0 * N * ES, k0};
  };
  auto issue = [&](const At& a, int slot, int j, auto partial) {
    const bool x = j < Sh::CPX;
    const int i = x ? Sh::CPX * wave + j : Sh::CPW * wave + j - Sh::CPX;
    const char* const base = x ? a.x : a.w;
    const uint32_t from = x ? xsrc[x ? j : 0] : wsrc[x ? 0 : j - Sh::CPX];
    const uint32_t to = lds0 + (uint32_t)slot * (Sh::XB + Sh::WB) + (x ? 0 : Sh::XB) + i * 1024;
    if constexpr (!decltype(partial)::value) copy_frag(base, from, to);
    else copy_at(a.k0 + line_step(8 * i + (lane >> 3), ES) < K ? base + from : reinterpret_cast<const char*>(g_zeros), to);
  };

  f32x16_t acc[CB][TB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][i][v] = 0.0f;
  const int live = (M - m0 - wt * TB * 32 + 31) >> 5;
  reduce_stages<T, TB, CB, WT, WC, S, true, true, false, false, PAIR ? 2 : 1>(acc, ring, st, live, wt, wc, lane, at, issue);
  __syncthreads();

  unsigned char* const stage = ring + wave * 32 * (32 * CB * 4 + 16);
  const int nw = n0 + 32 * CB * wc;
  const size_t out0 = (size_t)e * M * N;
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int rb = m0 + (wt * TB + i) * 32;
    if (rb >= M) break;
    if (splits > 1) {  // fp32 partial sums [problem][split][E][M][N]
      float* const part = A.part + ((size_t)q * splits + split) * A.E * M * N;
      each_vec<F32, TB, CB, CB>(acc, i, stage, lane, [&](int, int r, int ch, const Vec<F32>& a, const Vec<F32>&) {
        if (rb + r < M && nw + ch < N) store_vec<F32>(part, out0 + (size_t)(rb + r) * N + nw + ch, a);
      });
      continue;
    }
    each_vec<T, TB, CB, CB>(acc, i, stage, lane, [&](int, int r, int ch, const Vec<T>& a, const Vec<T>&) {
      if (rb + r < M && nw + ch < N) store_vec<T>(P.out, out0 + (size_t)(rb + r) * N + nw + ch, a);
    });
  }
}

// Joins split weight gradients: blockIdx.y is the problem.
template <class T>
__global__ __launch_bounds__(256) void k_grad_w_join(const GradWArgs A, int splits) {
  constexpr int V = Vec<T>::N;
  const size_t n = (size_t)A.E * A.m * A.p;
  const float* const part = A.part + (size_t)blockIdx.y * splits * n;
  void* const out = A.problem[blockIdx.y].out;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * V; i < n; i += (size_t)gridDim.x * 256 * V) {
    Vec<T> a = {};
    for (int k = 0; k < splits; ++k)
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(part + k * n + i + j);
#pragma unroll
        for (int v = 0; v < 4; ++v) a.v[j + v] += f[v];
      }
    store_vec<T>(out, i, a);
  }
}

// ---- launches --------------------------------------------------------------------------

// Upper bound on the row blocks of BM rows.
inline long long row_blocks(const GatedArgs& a, int BM) {
  return a.offsets ? (long long)a.R / BM + (a.R < a.E ? a.R : a.E) : ((long long)a.R + BM - 1) / BM;
}

template <class T, Op OP, int TB, int CB, int WT, int WC, int S, bool ONCE = false, bool PAIR = false>
hipError_t launch_tile(const GatedArgs& a, int cg, int splits, int cus, hipStream_t s) {
  constexpr int BM = 32 * TB * WT, BN = 32 * CB * WC / (OP == Op::kUp ? 2 : 1);
  const long long most = row_blocks(a, BM) * ((a.N + BN - 1) / BN);
  const int cut = BM == 256 && splits == 1 ? cus : 0;
  const long long blocks = cut ? cut_blocks(most, cut) : (most + 7) / 8 * 8 * splits;
  if (blocks * WT * WC * 64 >= 1LL << 32) return hipErrorInvalidValue;
  k_gated_rows<T, OP, TB, CB, WT, WC, S, ONCE, PAIR><<<(unsigned)blocks, WT * WC * 64, 0, s>>>(a, cg, splits, cut);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || splits == 1) return e;
  const long long vecs = (long long)a.R * (a.N / Vec<T>::N), n = (vecs + 255) / 256;
  k_gated_join<T, OP><<<(unsigned)(n < 1 << 20 ? n : 1 << 20), 256, 0, s>>>(a, splits);
  return hipGetLastError();
}

// The product with the tile that choose_gated names.
template <class T, Op OP>
hipError_t rows_product(const GatedArgs& a, int cus, hipStream_t s) {
  constexpr int cg = 4;  // column blocks that share their rows in an XCD's L2 (2: the same, 8: 2 %, 16: 7 % slower)
  constexpr int KD = stage_steps(T::ES);
  const GatedChoice c = choose_gated(T::ES == 2, a.R, OP == Op::kUp ? 2LL * a.N : a.N,
                                     (a.K + KD - 1) / KD * (OP == Op::kGradX ? 2 : 1), a.E, cus);
  if (c.splits > 1 && !a.part) return hipErrorInvalidValue;
  constexpr bool PAIR = T::ES == 2 && (OP == Op::kDown || OP == Op::kGradX);  // the 32-row tiles of hidden rows
  if (T::ES == 2 && (gated_pairs(true, a.R, a.E) != (a.low != 0))) return hipErrorInvalidValue;
  if constexpr (T::ES == 2) {
    switch (c.tile) {
      case kGated256x256x2: return launch_tile<T, OP, 4, 2, 2, 4, 2>(a, cg, c.splits, cus, s);
      case kGated128x256x3: return launch_tile<T, OP, 2, 2, 2, 4, 3>(a, cg, c.splits, cus, s);
      case kGated128x128x2: return launch_tile<T, OP, 2, 2, 2, 2, 2>(a, cg, c.splits, cus, s);
      case kGated64x128x3: return launch_tile<T, OP, 1, 2, 2, 2, 3>(a, cg, c.splits, cus, s);
      case kGated32x256x2:
        return c.once ? launch_tile<T, OP, 1, 2, 1, 4, 2, true, PAIR>(a, cg, c.splits, cus, s)
                      : launch_tile<T, OP, 1, 2, 1, 4, 2, false, PAIR>(a, cg, c.splits, cus, s);
      case kGated32x256x3:
        return c.once ? launch_tile<T, OP, 1, 2, 1, 4, 3, true, PAIR>(a, cg, c.splits, cus, s)
                      : launch_tile<T, OP, 1, 2, 1, 4, 3, false, PAIR>(a, cg, c.splits, cus, s);
      default: return hipErrorInvalidValue;
    }
  }
  switch (c.tile) {
    case kGated128x128x2: return launch_tile<T, OP, 2, 2, 2, 2, 2>(a, cg, c.splits, cus, s);
    case kGated64x128x3: return launch_tile<T, OP, 1, 2, 2, 2, 3>(a, cg, c.splits, cus, s);
    case kGated32x128x2: return launch_tile<T, OP, 1, 2, 1, 2, 2>(a, cg, c.splits, cus, s);
    default: return hipErrorInvalidValue;
  }
}

template <class T, int TB, int CB, int WT, int WC, int S, bool PAIR>
hipError_t launch_grad_w_tile(const GradWArgs& a, int cg, int splits, hipStream_t s) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  long long per = 0;
  for (int i = 0; i < a.n; ++i)
    per += (long long)((a.problem[i].M + Sh::BM - 1) / Sh::BM) * ((a.problem[i].N + Sh::BN - 1) / Sh::BN);
  const long long blocks = (per + 7) / 8 * 8 * a.E * splits;
  if (blocks * WT * WC * 64 >= 1LL << 32) return hipErrorInvalidValue;
  k_gated_grad_w<T, TB, CB, WT, WC, S, PAIR><<<(unsigned)blocks, WT * WC * 64, 0, s>>>(a, cg, (int)per, splits);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || splits == 1) return e;
  const long long vecs = (long long)a.E * a.m * a.p / Vec<T>::N, n = (vecs + 255) / 256;
  k_grad_w_join<T><<<dim3((unsigned)(n < 1 << 20 ? n : 1 << 20), a.n), 256, 0, s>>>(a, splits);
  return hipGetLastError();
}

template <class T>
hipError_t grad_w_product(const GradWArgs& a, int cus, hipStream_t s) {
  constexpr int cg = 4;  // column blocks that share their rows in an XCD's L2 (2 to 8: within 1 %)
  const GradWChoice c = choose_grad_w(T::ES == 2, a.R, a.m, a.p, a.E, cus);
  if (c.splits > 1 && !a.part) return hipErrorInvalidValue;
  if constexpr (T::ES == 2) {
    bool pair = true;
    for (int i = 0; i < a.n; ++i) pair = pair && a.problem[i].x2 && a.problem[i].w2;
    if (c.wide)
      return pair ? launch_grad_w_tile<T, 4, 2, 2, 4, 2, true>(a, cg, 1, s) : launch_grad_w_tile<T, 4, 2, 2, 4, 2, false>(a, cg, 1, s);
    if (pair) return launch_grad_w_tile<T, 2, 2, 2, 2, 2, true>(a, cg, c.splits, s);
  }
  return launch_grad_w_tile<T, 2, 2, 2, 2, 2, false>(a, cg, c.splits, s);
}

}  // namespace
}  // namespace moe
