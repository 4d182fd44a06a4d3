// int8 x int8 product with a scale per token and per output channel, dense or
// over the experts' row ranges (gfx950):
//   y[r][n] = sx[t] * sw[e][n] * sum_i x[t][i] * w[e][n][i]
// with t = r, or perm[r] / topk.  The int32 sums are exact (K <= kI8MaxK);
// they are converted to fp32, scaled there and rounded once.
//
// Both operands hold the reduction index innermost, so a lane's 16 bytes of a
// row are its MFMA operand as they lie in memory: nothing is repacked.  The
// weights take the product's row side (operand A) and the tokens its column
// side, so that a lane's accumulators are consecutive output channels of one
// token.
#include <type_traits>

#include "moe_items.hpp"
#include "moe_kernels.hpp"
#include "moe_lds.hpp"
#include "moe_rows.hpp"
#include "moe_rows_index.hpp"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// The x row of output row r, kept inside [0, T).
__device__ __forceinline__ int token_of(const I8Args& A, int r) {
  if (!A.perm) return r;
  const int t = A.perm[r] / A.topk;
  return t < 0 ? 0 : (t >= A.T ? A.T - 1 : t);
}

__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// global -> LDS, 16 bytes a lane from 64-bit addresses (see copy_frag).
__device__ __forceinline__ void copy_rows(const void* p, uint32_t lds) {
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

// copy_frag of a weight line that nothing reads again.
__device__ __forceinline__ void copy_once(const void* sbase, uint32_t voff, uint32_t lds) {
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

// Upper bound on the row blocks of BM rows.
long long row_blocks(const I8Args& a, int BM) {
  return a.offsets ? (long long)a.R / BM + (a.R < a.E ? a.R : a.E) : ((long long)a.R + BM - 1) / BM;
}

// go(y_bf16, nt), both known to the compiler.
template <class F>
void dispatch(F go, bool y_bf16, bool nt) {
  const std::true_type yes{};
  const std::false_type no{};
  if (y_bf16) nt ? go(yes, yes) : go(yes, no);
  else nt ? go(no, yes) : go(no, no);
}

// ---- few rows: every wave streams weights of its own -----------------------------
//
// A workgroup owns 16 CB output channels and up to 16 TB rows of one expert;
// its W waves split the reduction and add their int32 sums in LDS.  Each wave
// copies its own lines through a private ring of S stages (128 bytes of every
// row and channel), so no wave waits for another before the final sum.  The
// weights' bytes bound it: 16 x 28672 x 8192 takes 38 us, 6.2 TB/s (a large copy
// reaches 5.0 on this card), 16 x 14336 x 4096 17.9 us, 3.3 TB/s, and with its
// weights in the last-level cache 11.6 us.  Weights
// loaded straight into registers, half a line an instruction, took 13.5 us
// where these copies took 11.1 (16 x 4096 x 14336).  Neighbouring workgroups
// start from different stages, see k_i8_tile (16 x 16384 x 8192: 31 against 24 us).
// NT: weights that only one row block of the expert reads are not kept.
template <int TB, int CB, int W, int S, bool YB, bool NT>
__global__ __launch_bounds__(W * 64) void k_i8_rows(const I8Args A, int cols) {
  constexpr int CPX = 2 * TB, CPW = 2 * CB, CP = CPX + CPW;
  static_assert(CP * S <= 63, "vmcnt holds at most 63");
  constexpr int STAGE = CP * 1024;
  constexpr int RING = W * S * STAGE, PART = W * CB * TB * 1024;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[RING > PART ? RING : PART];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // row blocks outermost: neighbouring workgroups, on different XCDs, read neighbouring channels
  const Item it = find_item(A.offsets, A.E, A.R, 16 * TB, cols, 0, (int)blockIdx.x, false);
  if (it.e < 0) return;
  const int e = it.e, n0 = it.nb * 16 * CB, row0 = it.row0, rows = it.rows;

  const int8_t* xsrc[CPX];
  uint32_t wsrc[CPW];
  const int8_t* const wbase = A.w + ((size_t)e * A.N + n0) * A.K;
#pragma unroll
  for (int j = 0; j < CPX; ++j)
    xsrc[j] = A.x + (size_t)token_of(A, row0 + min(8 * j + (lane >> 3), rows - 1)) * A.K;
#pragma unroll
  for (int j = 0; j < CPW; ++j) wsrc[j] = (uint32_t)min(8 * j + (lane >> 3), A.N - 1 - n0) * (uint32_t)A.K;
  unsigned char* const ring = lds + wave * S * STAGE;
  const uint32_t at0 = lds_address(ring);
  const int steps = (A.K + 127) / 128;
  const int lo = (int)((long long)steps * wave / W), hi = (int)((long long)steps * (wave + 1) / W);
  const int rot = lo < hi ? it.nb % (hi - lo) : 0;
  auto stage_of = [&](int s) { return turned(s, rot, lo, hi); };
  auto issue = [&](int s, int slot, auto once) {
    const int k0 = stage_of(min(s, hi - 1)) * 128;  // past K: any bytes of the row, multiplied by zeros
    const uint32_t at = at0 + (uint32_t)slot * STAGE;
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const uint32_t from = wsrc[j] + (uint32_t)min(k0 + 16 * chunk_of(j, lane), A.K - 16);
      if constexpr (decltype(once)::value) copy_once(wbase, from, at + (CPX + j) * 1024);
      else copy_frag(wbase, from, at + (CPX + j) * 1024);
    }
#pragma unroll
    for (int j = 0; j < CPX; ++j)
      copy_rows(xsrc[j] + min(k0 + 16 * chunk_of(j, lane), A.K - 16), at + j * 1024);
  };
  i32x4_t acc[CB][TB] = {};
  const int quart = lane >> 4;
  auto reduce = [&](auto once) {
#pragma unroll
    for (int s = 0; s < S; ++s) issue(lo + s, s, once);
    int slot = 0;
    for (int s = lo; s < hi; ++s) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(CP * (S - 1)) : "memory");
      const unsigned char* st = ring + slot * STAGE;
      i32x4_t wv[2][CB], xv[2][TB];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int at = operand16(lane, ks);
#pragma unroll
        for (int c = 0; c < CB; ++c) wv[ks][c] = *reinterpret_cast<const i32x4_t*>(st + (CPX + 2 * c) * 1024 + at);
#pragma unroll
        for (int i = 0; i < TB; ++i) xv[ks][i] = *reinterpret_cast<const i32x4_t*>(st + 2 * i * 1024 + at);
      }
      if ((stage_of(s) + 1) * 128 > A.K) {  // the tail: zero weights past K
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int c = 0; c < CB; ++c)
            if (stage_of(s) * 128 + 64 * ks + 16 * quart >= A.K) wv[ks][c] = i32x4_t{0, 0, 0, 0};
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
      issue(s + S, slot, once);
      slot = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
          for (int i = 0; i < TB; ++i)
            acc[c][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[ks][c], xv[ks][i], acc[c][i], 0, 0, 0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the last copies have landed: the ring is reused
  };
  if (lo < hi) {
    if (NT && it.blocks == 1) reduce(std::integral_constant<bool, NT>{});
    else reduce(std::false_type{});
  }
  __syncthreads();
  i32x4_t* const part = reinterpret_cast<i32x4_t*>(lds);  // [W][CB * TB][64]
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < TB; ++i) part[(wave * CB * TB + c * TB + i) * 64 + lane] = acc[c][i];
  __syncthreads();
  // a wave finishes a tile: a lane holds channels 16 c + 4 (lane / 16) .. + 3
  // of row 16 i + lane % 16
  for (int f = wave; f < CB * TB; f += W) {
    const int nn = n0 + 16 * (f / TB) + 4 * (lane >> 4);
    const int r = 16 * (f % TB) + (lane & 15);
    i32x4_t sum = part[f * 64 + lane];
#pragma unroll
    for (int v = 1; v < W; ++v) sum += part[(v * CB * TB + f) * 64 + lane];
    if (r >= rows || nn >= A.N) continue;
    const float sx = A.sx[token_of(A, row0 + r)];
    const float4 sw = *reinterpret_cast<const float4*>(A.sw + (size_t)e * A.N + nn);
    const float o[4] = {(float)sum[0] * sx * sw.x, (float)sum[1] * sx * sw.y, (float)sum[2] * sx * sw.z,
                        (float)sum[3] * sx * sw.w};
    const size_t at = (size_t)(row0 + r) * A.N + nn;
    if constexpr (YB)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + at) = make_uint2(pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(A.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
  }
}

template <int TB, int CB, int W, int S>
hipError_t launch_rows(const I8Args& a, bool y_bf16, bool large, hipStream_t s) {
  const long long cols = (a.N + 16 * CB - 1) / (16 * CB);
  const long long blocks = row_blocks(a, 16 * TB) * cols;
  if (blocks * W * 64 >= 1LL << 32) return hipErrorInvalidValue;
  auto go = [&](auto yb, auto nt) {
    constexpr bool YB = decltype(yb)::value, NT = decltype(nt)::value;
    k_i8_rows<TB, CB, W, S, YB, NT><<<(unsigned)blocks, W * 64, 0, s>>>(a, (int)cols);
  };
  dispatch(go, y_bf16, large);
  return hipGetLastError();
}

// ---- many rows: tiles through LDS ------------------------------------------------
//
// A workgroup of WT x WC waves computes 32 TB WT rows by 32 CB WC channels of
// one expert.  A stage is 128 bytes of the reduction: one cache line of every
// row and channel of the tile, copied into LDS with 16 bytes a lane, eight
// lines a copy, S stages in a ring (see line_place for a line's order in LDS).
//
// What bounds it: large products (256 x 256 tiles, two waves per SIMD, 128 x
// 64 each) the power of products, LDS reads and copies together.  8192 x 4096
// x 14336 takes 408 to 418 us, 2.3 POP/s; the products alone 283 us, products and
// LDS reads 350 us, the copies alone 290 us, while the clock falls to 1.8 GHz.
// A deeper ring (96 KiB under way instead of 64) and four waves of 128 x 128
// (a third fewer LDS reads) measured 2 and 3 % slower.  Products of few rows
// (32 x 256 tiles) stream their weights at 6.5 TB/s.  NT: an expert's weights
// that only one row block reads are not kept.
template <int TB, int CB, int WT, int WC, int S, bool YB, bool NT>
__global__ __launch_bounds__(WT* WC * 64)
    __attribute__((amdgpu_waves_per_eu(TileShape<TB, CB, WT, WC, S>::per_simd, TileShape<TB, CB, WT, WC, S>::per_simd)))
void k_i8_tile(const I8Args A, int cg, bool rotate) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  __shared__ __attribute__((aligned(1024))) unsigned char ring[S][Sh::XB + Sh::WB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WC, wc = wave % WC;
  const Item it = find_item(A.offsets, A.E, A.R, Sh::BM, (A.N + Sh::BN - 1) / Sh::BN, cg, (int)blockIdx.x, true);
  if (it.e < 0) return;
  const int e = it.e, row0 = it.row0, rows = it.rows, n0 = it.nb * Sh::BN;

  // copies: lane l of the copy of lines 8 i .. 8 i + 7 brings chunk
  // chunk_of(i, l) of line 8 i + l / 8 (rows past the tile's last and channels
  // past N re-read the last one)
  const int8_t* xsrc[Sh::CPX];
  uint32_t wsrc[Sh::CPW];
  const int8_t* const wbase = A.w + ((size_t)e * A.N + n0) * A.K;
#pragma unroll
  for (int j = 0; j < Sh::CPX; ++j) {
    const int r = min(8 * (Sh::CPX * wave + j) + (lane >> 3), rows - 1);
    xsrc[j] = A.x + (size_t)token_of(A, row0 + r) * A.K;
  }
#pragma unroll
  for (int j = 0; j < Sh::CPW; ++j)
    wsrc[j] = (uint32_t)min(8 * (Sh::CPW * wave + j) + (lane >> 3), A.N - 1 - n0) * (uint32_t)A.K;
  const uint32_t lds0 = lds_address(&ring[0][0]);
  const int steps = (A.K + 127) / 128;
  const int last = steps - 1;
  // Where a weight tile is read once (rotate), neighbouring column blocks walk
  // the reduction from different stages: in step with one another they read
  // the same offset of rows a power of two apart, few of the memory's channels
  // (16 rows each of 8 experts, 470 MB of weights: 84 against 72 us).  A partial stage
  // stays the last.
  const int full = A.K / 128, rot = rotate && full ? it.nb % full : 0;
  auto stage_of = [&](int s) { return s >= full ? s : turned(s, rot, 0, full); };
  // copy j of the wave's CP of stage s
  auto issue_one = [&](int s, int j, auto once) {
    const uint32_t at = lds0 + (uint32_t)(s % S) * (Sh::XB + Sh::WB);
    const int k0 = stage_of(s) * 128;  // past K: any bytes of the row, multiplied by zeros
    if (j < Sh::CPX) {
      const int i = Sh::CPX * wave + j;
      copy_rows(xsrc[j] + min(k0 + 16 * chunk_of(i, lane), A.K - 16), at + i * 1024);
    } else {
      const int i = Sh::CPW * wave + j - Sh::CPX;
      const uint32_t from = wsrc[j - Sh::CPX] + (uint32_t)min(k0 + 16 * chunk_of(i, lane), A.K - 16);
      if constexpr (decltype(once)::value) copy_once(wbase, from, at + Sh::XB + i * 1024);
      else copy_frag(wbase, from, at + Sh::XB + i * 1024);
    }
  };

  i32x16_t acc[CB][TB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[c][i][v] = 0;

  const int half = lane >> 5;
  struct Frag {
    i32x4_t x[TB], w[CB];
  };
  // Every operand read is issued ahead of the products of the quarter stage
  // before it, across the stages too: a stage's last quarter is multiplied
  // after the barrier that frees its ring slot, while the copies into that
  // slot and the next stage's first reads are under way.  LIVE: the wave's row
  // blocks that hold rows (an expert's last tile); the others are not read or
  // multiplied, and a wave without any only copies.
  auto reduce = [&](auto live, auto once) {
    constexpr int LIVE = decltype(live)::value;
    // operand j of quarter ks of stage s: the channel blocks, then the row blocks
    auto load_one = [&](Frag& f, int s, int ks, int j) {
      const unsigned char* st = ring[s % S];
      const int at = operand32(lane, ks);
      if (j < CB) f.w[j] = *reinterpret_cast<const i32x4_t*>(st + Sh::XB + (wc * CB + j) * 4096 + at);
      else f.x[j - CB] = *reinterpret_cast<const i32x4_t*>(st + (wt * TB + j - CB) * 4096 + at);
    };
    constexpr int READS = LIVE ? CB + LIVE : 0, PRODUCTS = LIVE * CB;
    // The products of `f`, and after each one a read of the next quarter's
    // operands (`next`, quarter ks of stage s) and, with COPY, a copy of stage
    // `cs`: reads and copies issued together would leave the matrix cores idle
    // for as long as they take to issue.
    auto pass = [&](const Frag& f, Frag& next, int s, int ks, auto copy, int cs) {
      constexpr int COPIES = decltype(copy)::value ? Sh::CP : 0;
      constexpr int N = PRODUCTS > READS ? (PRODUCTS > COPIES ? PRODUCTS : COPIES) : (READS > COPIES ? READS : COPIES);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j < READS) load_one(next, s, ks, j);
        if (j < PRODUCTS)
          acc[j % CB][j / CB] =
              __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[j % CB], f.x[j / CB], acc[j % CB][j / CB], 0, 0, 0);
        if (j < COPIES) issue_one(cs, j, once);
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
    const int left = A.K - last * 128;  // the last stage: up to 128 bytes
    for (int ks = 0; 32 * ks < left; ++ks) {
#pragma unroll
      for (int j = 0; j < READS; ++j) load_one(f0, last, ks, j);
      if (LIVE > 0 && 32 * ks + 16 * half >= left)
#pragma unroll
        for (int c = 0; c < CB; ++c) f0.w[c] = i32x4_t{0, 0, 0, 0};  // weights past K
#pragma unroll
      for (int j = 0; j < PRODUCTS; ++j)
        acc[j % CB][j / CB] =
            __builtin_amdgcn_mfma_i32_32x32x32_i8(f0.w[j % CB], f0.x[j / CB], acc[j % CB][j / CB], 0, 0, 0);
    }
  };
  auto run = [&](auto once) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s <= last)
#pragma unroll
        for (int j = 0; j < Sh::CP; ++j) issue_one(s, j, once);
    if (S - 1 <= last) __builtin_amdgcn_s_waitcnt(vmcnt_imm(Sh::CP * (S - 1)));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    ring_barrier();
    const int live = min(TB, (rows - wt * TB * 32 + 31) >> 5);
    if (live == TB) reduce(std::integral_constant<int, TB>{}, once);
    else if (live <= 0) reduce(std::integral_constant<int, 0>{}, once);
    else if (TB == 4 && live == 3) reduce(std::integral_constant<int, TB == 4 ? 3 : 1>{}, once);
    else if (TB == 4 && live == 2) reduce(std::integral_constant<int, TB == 4 ? 2 : 1>{}, once);
    else reduce(std::integral_constant<int, 1>{}, once);
  };
  if (NT && it.blocks == 1) run(std::integral_constant<bool, NT>{});
  else run(std::false_type{});
  __syncthreads();  // the ring is free

  // Epilogue: element v of acc[c][i] in lane l is channel acc_channel(l, v) of
  // channel block c and row l % 32 of row block i.  A wave
  // stages one row block at a time (32 rows by its 32 CB channels, rows padded
  // by 16 bytes) and stores it 16 bytes a lane, whole lines of a row together.
  constexpr int ES = YB ? 2 : 4;
  constexpr int RB = Sh::row_bytes(ES), STR = Sh::stride(ES);
  unsigned char* const stage = &ring[0][0] + wave * 32 * STR;
  const int nw = n0 + wc * 32 * CB;  // the wave's first channel
  float sw[CB][16];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int n = nw + 32 * c + 8 * g + 4 * half;
      const float4 f = n < A.N ? *reinterpret_cast<const float4*>(A.sw + (size_t)e * A.N + n) : make_float4(0, 0, 0, 0);
      sw[c][4 * g] = f.x, sw[c][4 * g + 1] = f.y, sw[c][4 * g + 2] = f.z, sw[c][4 * g + 3] = f.w;
    }
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    const int rb = (wt * TB + i) * 32;  // the block's first row in the tile
    if (rb >= rows) break;
    const int r = min(rb + (lane & 31), rows - 1);
    const float sx = A.sx[token_of(A, row0 + r)];
    unsigned char* const mine = stage + (lane & 31) * STR + 4 * half * ES;
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = (float)acc[c][i][4 * g + v] * sx * sw[c][4 * g + v];
        unsigned char* const p = mine + (32 * c + 8 * g) * ES;
        if constexpr (YB)
          *reinterpret_cast<uint2*>(p) = make_uint2(pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3]));
        else
          *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
      }
    constexpr int LPR = RB / 16;   // lanes per row
    constexpr int RPI = 64 / LPR;  // rows per store
    // other lanes of the wave wrote what a lane reads (a wave's LDS accesses
    // take place in order; the compiler must keep them so across the types)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int rr = q * RPI + lane / LPR, col = lane % LPR;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * STR + col * 16);
      const int n = nw + col * (16 / ES);
      if (rb + rr < rows && n < A.N)
        *reinterpret_cast<uint4*>(static_cast<char*>(A.y) + ((size_t)(row0 + rb + rr) * A.N + n) * ES) = v;
    }
    asm volatile("" ::: "memory");
  }
}

template <int TB, int CB, int WT, int WC, int S>
hipError_t launch_tile(const I8Args& a, bool y_bf16, int cg, bool single, bool large, hipStream_t s) {
  using Sh = TileShape<TB, CB, WT, WC, S>;
  const long long blocks = row_blocks(a, Sh::BM) * ((a.N + Sh::BN - 1) / Sh::BN);
  if ((blocks + 8) * WT * WC * 64 >= 1LL << 32) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)((blocks + 7) / 8 * 8);
  auto go = [&](auto yb, auto nt) {
    constexpr bool YB = decltype(yb)::value, NT = decltype(nt)::value;
    k_i8_tile<TB, CB, WT, WC, S, YB, NT><<<grid, WT * WC * 64, 0, s>>>(a, cg, single);
  };
  dispatch(go, y_bf16, single && large);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_i8(const I8Args& a, bool y_bf16, int cus, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  if (a.K <= 0 || a.K % 16 || a.K > kI8MaxK || a.N <= 0 || a.N % 8 || a.E < 1 || (!a.offsets && a.E != 1))
    return hipErrorInvalidValue;
  const I8Choice c = choose_i8(a.R, a.N, a.E, cus);
  const bool once = c.once, large = i8_weights_once(a.w, a.K, a.N, a.E);
  const int cg = 4;  // column blocks that share their rows in an XCD's L2 (2 and 8: within 2 %; 1: 10 % slower)
  switch (c.kernel) {
    case kTile32x256x3: return launch_tile<1, 2, 1, 4, 3>(a, y_bf16, cg, once, large, s);
    case kTile64x256x3: return launch_tile<2, 2, 1, 4, 3>(a, y_bf16, cg, once, large, s);
    case kTile32x256x2: return launch_tile<1, 2, 1, 4, 2>(a, y_bf16, cg, once, large, s);
    case kTile64x256x2: return launch_tile<2, 2, 1, 4, 2>(a, y_bf16, cg, once, large, s);
    case kTile256x256x2: return launch_tile<4, 2, 2, 4, 2>(a, y_bf16, cg, once, large, s);
    case kTile128x256x3: return launch_tile<2, 2, 2, 4, 3>(a, y_bf16, cg, once, large, s);
    case kTile128x128x4: return launch_tile<2, 1, 2, 4, 4>(a, y_bf16, cg, once, large, s);
    case kTile64x128x3: return launch_tile<1, 2, 2, 2, 3>(a, y_bf16, cg, once, large, s);
    case kTile64x64x4: return launch_tile<1, 1, 2, 2, 4>(a, y_bf16, cg, once, large, s);
    case kRing16x32: return launch_rows<1, 2, 4, 2>(a, y_bf16, large, s);
    case kRing64x32: return launch_rows<4, 2, 4, 2>(a, y_bf16, large, s);
    case kRing32x32: return launch_rows<2, 2, 4, 2>(a, y_bf16, large, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
