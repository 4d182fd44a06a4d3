// Row operators around the experts for gfx950: the input norm's forward and
// backward pass, also with the residual's addition and int8 codes, token rows
// copied into expert order, expert rows combined back to their tokens, and the
// gradients of both.
//
// All of them move each row through HBM once and do 1 to 16 operations per
// element, so bytes bound them; sums and statistics are fp32, and a value is
// rounded once, when it is stored.  Measured at 8192 rows of 4096 bf16, in
// parentheses the algorithmic bytes over the time (a large copy reaches 5.0
// TB/s on this card): layer norm 24.5 us (5.5 TB/s), its gradients 41.4 us (4.9),
// top-2 permute 38.4 us (5.2), its gradient and the combine 34.5 us (5.8), the
// combine's gradient 66.4 us (5.1); the residual added, normalised and quantised
// 54 us (5.6), its gradient with the residual stream's 46 us (5.8).
#include <type_traits>

#include "moe_convert.hpp"
#include "moe_kernels.hpp"
#include "moe_rows.hpp"
#include "moe_rows_index.hpp"

namespace moe {
namespace {

// (HIP's own uint4 is a struct whose arrays the compiler does not keep in
// registers once their loads are conditional)
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// 16 bytes; ONCE: of data that the caches need not keep.
template <bool ONCE>
__device__ __forceinline__ u32x4_t load16(const void* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
  else return *static_cast<const u32x4_t*>(p);
}

// Eight consecutive bf16 starting at element i (a multiple of 8).
template <bool ONCE>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&f)[8]) {
  const u32x4_t v = load16<ONCE>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(v[j] << 16);
    f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
  }
}

// Two fp32 -> two bf16, round to nearest even (the hardware conversion).
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

__device__ __forceinline__ void store8(void* p, size_t i, const float (&f)[8]) {
  *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) =
      u32x4_t{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7])};
}

// v plus the value that the DPP control CTRL moves to each lane (0 where none does).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, ROWS, 0xF, true));
}

// Sum over the wave, the same in every lane: four shifts within rows of 16
// lanes, then the rows' totals carried to the last lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Sum over aligned groups of n = 8, 16 or 32 lanes, the same in each of them:
// a step adds lanes whose values are equal within the half that they come from.
__device__ __forceinline__ float group_sum(float v, int n) {
  v = dpp_add<0xB1, 0xF>(v);   // lane ^ 1
  v = dpp_add<0x4E, 0xF>(v);   // lane ^ 2
  v = dpp_add<0x141, 0xF>(v);  // the other half of 8 lanes
  if (n > 8) v = dpp_add<0x140, 0xF>(v);  // the other half of 16
  if (n > 16) v += __shfl_xor(v, 16, 64);
  return v;
}

// ---- norm -----------------------------------------------------------------------
//
// A team of NT threads (8, 16, 32 or a multiple of 64) owns a row; a block
// holds one or more teams.  A thread keeps V times eight elements (norm_cols).
template <bool BF16, bool ONCE>
__device__ __forceinline__ void load_raw(u32x4_t (&v)[BF16 ? 1 : 2], const void* p, size_t row, NormCols c, int m) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
    const int at = i ? c.hi : c.lo;
    v[i] = u32x4_t{0, 0, 0, 0};
    if (at < m) v[i] = load16<ONCE>(static_cast<const char*>(p) + (row + at) * (BF16 ? 2 : 4));
  }
}

template <bool BF16>
__device__ __forceinline__ void from_raw(const u32x4_t (&v)[BF16 ? 1 : 2], float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16) {
      f[2 * j] = __uint_as_float(v[0][j] << 16);
      f[2 * j + 1] = __uint_as_float(v[0][j] & 0xFFFF0000u);
    } else {
      f[j] = __uint_as_float(v[0][j]);
      f[4 + j] = __uint_as_float(v[1][j]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store_row(void* p, size_t row, NormCols c, int m, const float (&f)[8]) {
  if constexpr (BF16) {
    if (c.lo < m) store8(p, row + c.lo, f);
  } else {
    if (c.lo < m) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + row + c.lo) = f32x4_t{f[0], f[1], f[2], f[3]};
    if (c.hi < m) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + row + c.hi) = f32x4_t{f[4], f[5], f[6], f[7]};
  }
}

// The same columns of an fp32 vector (gamma, beta, a row of partial sums); 0 past m.
template <bool BF16>
__device__ __forceinline__ void load_vec(const float* p, NormCols c, int m, float (&f)[8]) {
  const f32x4_t zero = {0, 0, 0, 0};
  const f32x4_t a = c.lo < m ? *reinterpret_cast<const f32x4_t*>(p + c.lo) : zero;
  const f32x4_t b = c.hi < m ? *reinterpret_cast<const f32x4_t*>(p + c.hi) : zero;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = a[j];
    f[4 + j] = b[j];
  }
}

template <bool BF16>
__device__ __forceinline__ void store_vec(float* p, NormCols c, int m, const float (&f)[8]) {
  if (c.lo < m) *reinterpret_cast<f32x4_t*>(p + c.lo) = f32x4_t{f[0], f[1], f[2], f[3]};
  if (c.hi < m) *reinterpret_cast<f32x4_t*>(p + c.hi) = f32x4_t{f[4], f[5], f[6], f[7]};
}

// Sum over a team, the same in all of its threads.  slot is an LDS row of 16
// per wave of the block; consecutive sums use different rows, so one barrier
// each is enough: a row is written again only after a barrier that every wave
// reaches after reading it.
__device__ __forceinline__ float team_sum(float v, int NT, int first, float* slot) {
  if (NT < 64) return group_sum(v, NT);
  v = wave_sum(v);
  if (NT == 64) return v;
  const int lane = threadIdx.x & 63, waves = NT >> 6;
  if (lane == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  return group_sum((lane & 15) < waves ? slot[first + (lane & 15)] : 0.0f, 16);
}

// The largest value of a team, as team_sum.
__device__ __forceinline__ float team_max(float v, int NT, int first, float* slot) {
  for (int o = 1; o < (NT < 64 ? NT : 64); o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  if (NT <= 64) return v;
  const int lane = threadIdx.x & 63, waves = NT >> 6;
  if (lane == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (lane & 15) < waves ? slot[first + (lane & 15)] : 0.0f;
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// y = (x - mu) r gamma + beta, mu the row's mean (0 for the RMS norm), r = 1 /
// sqrt(mean((x - mu)^2) + eps).  gamma and beta stay in registers from row to
// row; the next row is loaded while this one is summed.
//
// ADD: x + residual in place of x, kept in fp32 for the norm and rounded once to
// be stored as sum; y may be absent, and its int8 codes with the row's power-of-two
// scale (act_scale_exponent) are taken from the fp32 values, not from rounded
// ones.  sum and y may lie over x or residual: a row is read whole by the team
// that writes it, before it does.
template <bool BF16, int V, bool LAYER, bool ONCE, bool ADD>
__global__ __launch_bounds__(1024) void k_norm_fwd(const NormArgs A, int NT) {
  __shared__ float red[3][16];
  const int team = threadIdx.x / NT, teams = blockDim.x / NT, tid = threadIdx.x - team * NT;
  const int first = team * NT >> 6;  // the team's first wave
  const int m = A.m;
  const float inv_m = 1.0f / (float)m;
  float g[V][8], b[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const NormCols c = norm_cols(BF16, tid, NT, v);
    load_vec<BF16>(A.gamma, c, m, g[v]);
    if (LAYER && A.beta) load_vec<BF16>(A.beta, c, m, b[v]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
  }
  u32x4_t next[V][BF16 ? 1 : 2], nres[ADD ? V : 1][BF16 ? 1 : 2];
  auto fetch = [&](long long t) {
    if (t >= A.T) t = A.T - 1;  // read, never written
#pragma unroll
    for (int v = 0; v < V; ++v) {
      load_raw<BF16, ONCE>(next[v], A.x, (size_t)t * m, norm_cols(BF16, tid, NT, v), m);
      if (ADD && A.residual)
        load_raw<BF16, ONCE>(nres[v], A.residual, (size_t)t * m, norm_cols(BF16, tid, NT, v), m);
    }
  };
  const long long stride = (long long)gridDim.x * teams;
  fetch((long long)blockIdx.x * teams + team);
  int turn = 0;
  for (long long t0 = (long long)blockIdx.x * teams; t0 < A.T; t0 += stride, turn ^= 1) {  // the same count for every team
    const long long t = t0 + team;
    float f[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      from_raw<BF16>(next[v], f[v]);
      if (ADD && A.residual) {
        float r[8];
        from_raw<BF16>(nres[v], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[v][j] += r[j];
      }
    }
    if (t0 + stride < A.T) fetch(t + stride);
    if constexpr (ADD)
      if (A.sum && t < A.T)
#pragma unroll
        for (int v = 0; v < V; ++v) store_row<BF16>(A.sum, (size_t)t * m, norm_cols(BF16, tid, NT, v), m, f[v]);
    float mu = 0.0f;
    if constexpr (LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += f[v][j];
      mu = team_sum(s, NT, first, red[0]) * inv_m;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const NormCols c = norm_cols(BF16, tid, NT, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = (j < 4 ? c.lo : c.hi) < m ? f[v][j] - mu : 0.0f;
        f[v][j] = d;
        q = fmaf(d, d, q);
      }
    }
    const float var = team_sum(q, NT, first, red[LAYER ? 1 : turn]) * inv_m;
    float r = 1.0f / sqrtf(var + A.eps);
    float rest = 0.0f;  // of r, to 40 bits: one step of Newton's method on r^-2 = var + eps
    if constexpr (ADD) {
      const float v = var + A.eps, q1 = v * r, e = fmaf(-q1, r, 1.0f) - fmaf(v, r, -q1) * r;
      if (r > 0.0f && r < INFINITY && e > -1.0f && e < 1.0f) {
        rest = 0.5f * r * e;
        const float near = r + rest;
        rest -= near - r;
        r = near;
      }
    }
    if (tid == 0 && t < A.T) {
      if (LAYER && A.mean) A.mean[t] = mu;
      if (A.rstd) A.rstd[t] = r;
    }
    if constexpr (!ADD) {
      if (t >= A.T) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = LAYER ? fmaf(f[v][j] * r, g[v][j], b[v][j]) : f[v][j] * r * g[v][j];
        store_row<BF16>(A.out, (size_t)t * m, norm_cols(BF16, tid, NT, v), m, o);
      }
    } else {
      float top = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)  // past the row's end gamma and beta are 0, and so is y
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // h = f r as a sum of two, so that y is rounded once: codes are rounded
          // from it, and each error moves some of them over a tie
          const float h = f[v][j] * r, low = fmaf(f[v][j], r, -h) + f[v][j] * rest;
          f[v][j] = LAYER ? fmaf(h, g[v][j], fmaf(low, g[v][j], b[v][j])) : fmaf(h, g[v][j], low * g[v][j]);
          top = fmaxf(top, fabsf(f[v][j]));
        }
      if (A.out && t < A.T)
#pragma unroll
        for (int v = 0; v < V; ++v) store_row<BF16>(A.out, (size_t)t * m, norm_cols(BF16, tid, NT, v), m, f[v]);
      if (!A.codes) continue;
      const int X = act_scale_exponent<true>(team_max(top, NT, first, red[2]));
      if (t >= A.T) continue;
      if (tid == 0) A.scale[t] = ldexpf(1.0f, X);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const NormCols c = norm_cols(BF16, tid, NT, v);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          q[h] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[h] |= ((uint32_t)(int)rintf(ldexpf(f[v][4 * h + j], -X)) & 0xFFu) << (8 * j);
        }
        int8_t* const row = A.codes + (size_t)t * m;
        if constexpr (BF16) {
          if (c.lo < m) *reinterpret_cast<u32x2_t*>(row + c.lo) = u32x2_t{q[0], q[1]};
        } else {
          if (c.lo < m) *reinterpret_cast<uint32_t*>(row + c.lo) = q[0];
          if (c.hi < m) *reinterpret_cast<uint32_t*>(row + c.hi) = q[1];
        }
      }
    }
  }
}

// The gradients.  With h = (x - mu) r and u = gamma dy:
//   dx = r (u - h <u, h> / m - [layer] <u, 1> / m)
//   dgamma = sum_t dy h,  dbeta = sum_t dy
// A thread adds its columns' dy h and dy over the rows its team takes.  The
// block's sums are added in LDS and written as one row of partial sums, and
// k_norm_wgrad adds those in block order: nothing depends on timing.
// ADD: dsum, the gradient that reaches the sum of x and residual directly, is
// added to dx, which may lie over dsum or dy as the forward's rows may.
template <bool BF16, int V, bool LAYER, bool ONCE, bool ADD>
__global__ __launch_bounds__(1024) void k_norm_bwd(const NormArgs A, int NT) {
  __shared__ float red[4][16];
  extern __shared__ float acc[];  // [2][m] where the block's sums are added
  const int team = threadIdx.x / NT, teams = blockDim.x / NT, tid = threadIdx.x - team * NT;
  const int first = team * NT >> 6;
  const int m = A.m;
  const float inv_m = 1.0f / (float)m;
  float g[V][8], ag[V][8], ab[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_vec<BF16>(A.gamma, norm_cols(BF16, tid, NT, v), m, g[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ag[v][j] = ab[v][j] = 0.0f;
  }
  u32x4_t nx[V][BF16 ? 1 : 2], ny[V][BF16 ? 1 : 2], ns[ADD ? V : 1][BF16 ? 1 : 2];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](long long t) {
    const long long row = t < A.T ? t : A.T - 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const NormCols c = norm_cols(BF16, tid, NT, v);
      load_raw<BF16, ONCE>(nx[v], A.x, (size_t)row * m, c, m);
      load_raw<BF16, ONCE>(ny[v], A.dy, (size_t)row * m, c, m);
      if (ADD && A.dsum) load_raw<BF16, ONCE>(ns[v], A.dsum, (size_t)row * m, c, m);
    }
    nmu = LAYER ? A.mean[row] : 0.0f;
    nr = A.rstd[row];
  };
  // The next row loaded during this one's sums.  With V = 2 it takes 16 (bf16) or
  // 32 registers, and of the 128 that 1024 threads leave a thread 104 (RMS, bf16)
  // to 128 (layer norm, fp32) are in use: there is room for it in the bf16 RMS
  // form only, which has no form of its own.
  constexpr bool AHEAD = V == 1;
  const long long stride = (long long)gridDim.x * teams;
  if (AHEAD) fetch((long long)blockIdx.x * teams + team);
  int turn = 0;
  for (long long t0 = (long long)blockIdx.x * teams; t0 < A.T; t0 += stride, turn ^= 2) {  // the same count for every team
    const long long t = t0 + team;
    const bool live = t < A.T;
    if (!AHEAD) fetch(t);
    const float mu = nmu, r = nr;
    float h[V][8], u[V][8];
    u32x4_t ds[ADD ? V : 1][BF16 ? 1 : 2];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      from_raw<BF16>(nx[v], h[v]);
      from_raw<BF16>(ny[v], u[v]);
      if constexpr (ADD)
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) ds[v][i] = ns[v][i];
    }
    if (AHEAD && t0 + stride < A.T) fetch(t + stride);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const NormCols c = norm_cols(BF16, tid, NT, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // outside the row x and dy are 0: h would be -mu r, times 0; kept finite
        const bool in = live && (j < 4 ? c.lo : c.hi) < m;
        h[v][j] = in ? (h[v][j] - mu) * r : 0.0f;
        const float d = live ? u[v][j] : 0.0f;
        ag[v][j] = fmaf(d, h[v][j], ag[v][j]);
        if (LAYER) ab[v][j] += d;
        u[v][j] = d * g[v][j];
        s1 = fmaf(u[v][j], h[v][j], s1);
        if (LAYER) s2 += u[v][j];
      }
    }
    if (!A.out) continue;
    // both sums share a barrier
    float m1, m2 = 0.0f;
    if (NT < 64) {
      m1 = group_sum(s1, NT);
      if (LAYER) m2 = group_sum(s2, NT);
    } else {
      m1 = wave_sum(s1);
      if (LAYER) m2 = wave_sum(s2);
      if (NT > 64) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = NT >> 6;
        if (lane == 0) {
          red[turn][wave] = m1;
          if (LAYER) red[turn + 1][wave] = m2;
        }
        __syncthreads();
        const bool mine = (lane & 15) < waves;
        const int at = first + (mine ? lane & 15 : 0);
        m1 = group_sum(mine ? red[turn][at] : 0.0f, 16);
        if (LAYER) m2 = group_sum(mine ? red[turn + 1][at] : 0.0f, 16);
      }
    }
    m1 *= inv_m;
    m2 *= inv_m;
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (LAYER ? u[v][j] - m2 - h[v][j] * m1 : u[v][j] - h[v][j] * m1) * r;
      if constexpr (ADD)
        if (A.dsum) {
          float d[8];
          from_raw<BF16>(ds[v], d);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] += d[j];
        }
      store_row<BF16>(A.out, (size_t)t * m, norm_cols(BF16, tid, NT, v), m, o);
    }
  }
  if (!A.partial) return;
  for (int o = NT; o < 64; o <<= 1)  // teams that share a wave
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ag[v][j] += __shfl_xor(ag[v][j], o, 64);
        if (LAYER) ab[v][j] += __shfl_xor(ab[v][j], o, 64);
      }
  const int per = NT < 64 ? 64 : NT, groups = blockDim.x / per, group = threadIdx.x / per;
  const bool owner = NT >= 64 || (threadIdx.x & 63) < NT;
  for (int k = 1; k < groups; ++k) {
    __syncthreads();
    if (group == k && owner)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const NormCols c = norm_cols(BF16, tid, NT, v);
        store_vec<BF16>(acc, c, m, ag[v]);
        if (LAYER) store_vec<BF16>(acc + m, c, m, ab[v]);
      }
    __syncthreads();
    if (group == 0 && owner)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const NormCols c = norm_cols(BF16, tid, NT, v);
        float f[8];
        load_vec<BF16>(acc, c, m, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ag[v][j] += f[j];
        if (LAYER) {
          load_vec<BF16>(acc + m, c, m, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) ab[v][j] += f[j];
        }
      }
  }
  if (group || !owner) return;
  // a single block's sums are the gradients
  const bool one = gridDim.x == 1;
  float* const pg = one ? A.dgamma : A.partial + (size_t)blockIdx.x * m;
  float* const pb = one ? A.dbeta : A.partial + (size_t)(gridDim.x + blockIdx.x) * m;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const NormCols c = norm_cols(BF16, tid, NT, v);
    if (pg) store_vec<BF16>(pg, c, m, ag[v]);
    if (LAYER && pb) store_vec<BF16>(pb, c, m, ab[v]);
  }
}

// Sums the partial rows: a block owns 32 columns of one gradient (blockIdx.y:
// 0 gamma, 1 beta), eight lanes of four columns; its 64 groups of lanes take
// every 64th row, then add up in LDS.
__global__ __launch_bounds__(512) void k_norm_wgrad(const float* __restrict__ partial, int blocks, int m,
                                                    float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ f32x4_t part[64][8];
  float* const out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int q = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * q;
  const float* p = partial + (size_t)blockIdx.y * blocks * m + c;
  f32x4_t s = {0, 0, 0, 0};
  if (c < m)
#pragma unroll 4
    for (int b = grp; b < blocks; b += 64) s += *reinterpret_cast<const f32x4_t*>(p + (size_t)b * m);
  part[grp][q] = s;
#pragma unroll
  for (int n = 32; n; n >>= 1) {
    __syncthreads();
    if (grp < n) {
      s += part[grp + n][q];
      part[grp][q] = s;
    }
  }
  if (grp == 0 && c < m) *reinterpret_cast<f32x4_t*>(out + c) = s;
}

// ---- rows in expert order ---------------------------------------------------------
//
// One wave per (token, slice of its row).  An assignment's row is
// inv[t*k + j]; a value outside [0, R) means that it has none (dropped): it
// is not written, adds nothing and gets a zero weight gradient.
constexpr int kSlice = 4;  // 16-byte vectors per lane of a permuted slice

// The k rows of token t, one per lane (k <= 64).
__device__ __forceinline__ int token_rows(const RowsArgs& A, int t, int lane) {
  const int r = lane < A.k ? A.inv[(size_t)t * A.k + lane] : -1;
  return r >= 0 && r < A.R ? r : -1;
}

// out[inv[t*k+j]] = tok[t]: 16-byte chunks, whatever the type.
template <bool ONCE>
__global__ __launch_bounds__(256) void k_permute_rows(const RowsArgs A, int chunks, int slices) {
  const int lane = threadIdx.x & 63;
  const long long items = (long long)A.T * slices;
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += 4LL * gridDim.x) {
    const int t = (int)(item / slices), c0 = (int)(item % slices) * 64 * kSlice + lane;
    const int mine = token_rows(A, t, lane);
    const u32x4_t* src = static_cast<const u32x4_t*>(A.tok) + (size_t)t * chunks;
    u32x4_t v[kSlice];
#pragma unroll
    for (int i = 0; i < kSlice; ++i)
      if (c0 + 64 * i < chunks) v[i] = load16<ONCE>(src + c0 + 64 * i);
    for (int j = 0; j < A.k; ++j) {
      const int r = __builtin_amdgcn_readlane(mine, j);
      if (r < 0) continue;
      u32x4_t* dst = static_cast<u32x4_t*>(A.out) + (size_t)r * chunks;
#pragma unroll
      for (int i = 0; i < kSlice; ++i)
        if (c0 + 64 * i < chunks) dst[c0 + 64 * i] = v[i];
    }
  }
}

// The eight elements of a row at columns c (slab_cols), 0 past m: lanes past it
// load the row's end, so that the loads depend on no branch.  ONCE as in load16.
template <bool BF16, bool FOURS, bool ONCE>
__device__ __forceinline__ void load_cols(const void* p, size_t row, NormCols c, int m, float (&f)[8]) {
  if constexpr (!FOURS) {
    load8<ONCE>(p, row + min(c.lo, m - 8), f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const size_t at = row + min(h ? c.hi : c.lo, m - 4);
      if constexpr (BF16) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[4 * h + 2 * j] = __uint_as_float(v[j] << 16);
          f[4 * h + 2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
      } else {
        const u32x4_t v = load16<ONCE>(static_cast<const float*>(p) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[4 * h + j] = __uint_as_float(v[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (j < 4 ? c.lo : c.hi) < m ? f[j] : 0.0f;
}

template <bool BF16, bool FOURS>
__device__ __forceinline__ void store_cols(void* p, size_t row, NormCols c, int m, const float (&f)[8]) {
  if constexpr (!FOURS) {
    if (c.lo < m) store8(p, row + c.lo, f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = h ? c.hi : c.lo;
      if (at >= m) continue;
      const float* g = f + 4 * h;
      if constexpr (BF16)
        *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + row + at) =
            u32x2_t{pack2_bf16(g[0], g[1]), pack2_bf16(g[2], g[3])};
      else
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + row + at) = f32x4_t{g[0], g[1], g[2], g[3]};
    }
  }
}

// out[t] = sum_j w[t,j] rows[inv[t*k+j]], in order of j.
template <bool RB, bool OB, bool ONCE>
__global__ __launch_bounds__(256) void k_combine_rows(const RowsArgs A, int slices) {
  constexpr int V = 2;
  constexpr bool FOURS = !RB || !OB;
  const int lane = threadIdx.x & 63;
  const long long items = (long long)A.T * slices;
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += 4LL * gridDim.x) {
    const int t = (int)(item / slices), slab = (int)(item % slices) * V;
    const int mine = token_rows(A, t, lane);
    const float wl = lane < A.k ? (A.w ? A.w[(size_t)t * A.k + lane] : 1.0f) : 0.0f;
    float s[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[v][j] = 0.0f;
    for (int j = 0; j < A.k; ++j) {
      const int r = __builtin_amdgcn_readlane(mine, j);
      if (r < 0) continue;
      const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        load_cols<RB, FOURS, ONCE>(A.rows, (size_t)r * A.m, slab_cols(FOURS, lane, slab + v), A.m, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) s[v][q] = fmaf(wj, f[q], s[v][q]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      store_cols<OB, FOURS>(A.out, (size_t)t * A.m, slab_cols(FOURS, lane, slab + v), A.m, s[v]);
  }
}

// The combine's gradient, one block of up to four waves per token:
// out[inv[t*k+j]] = w[t,j] dy[t], dw[t,j] = <dy[t], rows[inv[t*k+j]]>.
// out may be rows: a lane writes the columns that it has read itself (lanes past
// the row's end read columns of others and drop them).
template <bool TB, bool RB, bool ONCE>
__global__ __launch_bounds__(256) void k_combine_rows_bwd(const RowsArgs A) {
  constexpr int V = 2;
  constexpr bool FOURS = !TB || !RB;
  __shared__ float dots[4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int slabs = row_slabs(A.m);
  for (long long i = blockIdx.x; i < A.T; i += gridDim.x) {  // the step past the last token may pass 2^31
    const int t = (int)i;
    const int mine = token_rows(A, t, lane);
    const float wl = lane < A.k && A.w ? A.w[(size_t)t * A.k + lane] : 0.0f;
    dots[wave][lane] = 0.0f;
    for (int slab = wave; slab < slabs; slab += waves * V) {
      float d[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v)
        load_cols<TB, FOURS, ONCE>(A.tok, (size_t)t * A.m, slab_cols(FOURS, lane, slab + v * waves), A.m, d[v]);
      for (int j = 0; j < A.k; ++j) {
        const int r = __builtin_amdgcn_readlane(mine, j);
        if (r < 0) continue;
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const NormCols c = slab_cols(FOURS, lane, slab + v * waves);
          if (A.dw) {
            float f[8];
            load_cols<RB, FOURS, ONCE>(A.rows, (size_t)r * A.m, c, A.m, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot = fmaf(d[v][q], f[q], dot);
          }
          if (A.out) {
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = wj * d[v][q];
            store_cols<RB, FOURS>(A.out, (size_t)r * A.m, c, A.m, o);
          }
        }
        if (A.dw) {
          dot = wave_sum(dot);
          if (lane == 0) dots[wave][j] += dot;
        }
      }
    }
    if (!A.dw) continue;
    __syncthreads();
    if (tid < A.k) {
      float s = 0.0f;
      for (int i = 0; i < waves; ++i) s += dots[i][tid];
      A.dw[(size_t)t * A.k + tid] = s;
    }
    __syncthreads();  // dots is cleared for the next token
  }
}

// Blocks of a launch: its threads must stay below 2^32, and the kernels walk
// what is left.
constexpr int kMaxGrid = 1 << 22;
unsigned wave_grid(long long items) {  // four waves a block, an item each
  const long long blocks = (items + 3) / 4;
  return blocks < kMaxGrid ? (unsigned)blocks : (unsigned)kMaxGrid;
}

// f(flags ...) with each flag known to the compiler.
template <class F>
void dispatch(F f) {
  f();
}
template <class F, class... Flags>
void dispatch(F f, bool flag, Flags... rest) {
  if (flag) dispatch([&](auto... r) { f(std::true_type{}, r...); }, rest...);
  else dispatch([&](auto... r) { f(std::false_type{}, r...); }, rest...);
}

// A call that moves half of the 256 MB last-level cache or more reads its
// inputs as data not to be kept (ONCE), which leaves the cache to what it writes
// for the next operator.  8192 x 4096 bf16: layer norm 27.3 -> 24.6 us, its
// gradients 43.2 -> 41.4, top-2 permute 39.9 -> 38.7, combine 41.1 -> 34.7; norm,
// permute and combine in turn 95 -> 84 us, their gradients 140 -> 128.  Below it
// the inputs may still be cached (16384 x 1024, norm, called again on the same
// rows: 12.8 -> 14.5 us).  Outputs written past the caches would take 22.6, 42.6,
// 30.2 and 37.7 us, and their next reader would pay for it (the three in turn:
// 100 us).
bool large(long long bytes) { return bytes >= 128 << 20; }
long long bytes_of(long long rows, int m, bool bf16) { return rows * m * (bf16 ? 2 : 4); }

}  // namespace

namespace {

template <bool ADD>
hipError_t norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, long long bytes, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const int V = norm_vecs(a.m), nt = norm_threads(a.m), teams = norm_fwd_teams(nt), threads = nt * teams;
  // the threads that a CU's registers hold: 2048 with up to 64 a thread, 1792 with 72, 1536
  // with 80 (more blocks than fit make a second round of a share each: 6802 x 2416 fp32,
  // residual added: 56.7 us with 2048, 54.1 with 1792)
  const int room = !ADD ? 2048 : bf16 ? (layer ? 1792 : 2048) : (layer ? 1536 : 1792);
  const long long blocks = ((long long)a.T + teams - 1) / teams, most = (long long)cus * (V == 1 ? room / threads : 1);
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  dispatch(
      [&](auto b, auto l, auto big) {
        constexpr bool B = decltype(b)::value, L = decltype(l)::value, ONCE = decltype(big)::value;
        if (V == 1) k_norm_fwd<B, 1, L, ONCE, ADD><<<grid, threads, 0, s>>>(a, nt);
        else k_norm_fwd<B, 2, L, ONCE, ADD><<<grid, threads, 0, s>>>(a, nt);
      },
      bf16, layer, large(bytes));
  return hipGetLastError();
}

template <bool ADD>
hipError_t norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, long long bytes, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const int V = norm_vecs(a.m), nt = norm_threads(a.m), threads = nt * norm_bwd_teams(nt);
  const unsigned grid = (unsigned)norm_bwd_blocks(a.T, a.m, cus);
  const size_t lds = threads > (nt < 64 ? 64 : nt) ? 2 * sizeof(float) * (size_t)a.m : 0;  // at most 2048 columns
  dispatch(
      [&](auto b, auto l, auto big) {
        constexpr bool B = decltype(b)::value, L = decltype(l)::value, ONCE = decltype(big)::value;
        if (V == 1) k_norm_bwd<B, 1, L, ONCE, ADD><<<grid, threads, lds, s>>>(a, nt);
        else k_norm_bwd<B, 2, L, ONCE, ADD><<<grid, threads, lds, s>>>(a, nt);
      },
      bf16, layer, large(bytes));
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.partial || grid == 1) return e;
  k_norm_wgrad<<<dim3((unsigned)((a.m + 31) / 32), layer ? 2 : 1), 512, 0, s>>>(a.partial, (int)grid, a.m, a.dgamma,
                                                                               layer ? a.dbeta : nullptr);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  return norm_forward<false>(a, bf16, layer, cus, 2 * bytes_of(a.T, a.m, bf16), s);
}

hipError_t launch_add_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  const int passes = 1 + (a.residual ? 1 : 0) + (a.sum ? 1 : 0) + (a.out ? 1 : 0);
  return norm_forward<true>(a, bf16, layer, cus, passes * bytes_of(a.T, a.m, bf16) + (a.codes ? (long long)a.T * a.m : 0), s);
}

hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  return norm_backward<false>(a, bf16, layer, cus, (a.out ? 3 : 2) * bytes_of(a.T, a.m, bf16), s);
}

hipError_t launch_add_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  return norm_backward<true>(a, bf16, layer, cus, (a.out ? (a.dsum ? 4 : 3) : 2) * bytes_of(a.T, a.m, bf16), s);
}

hipError_t launch_permute_rows(const RowsArgs& a, bool bf16, hipStream_t s) {
  if (a.T <= 0 || a.R <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int chunks = bf16 ? a.m / 8 : a.m / 4;
  const int slices = (chunks + 64 * kSlice - 1) / (64 * kSlice);
  const unsigned g = wave_grid((long long)a.T * slices);
  dispatch([&](auto big) { k_permute_rows<decltype(big)::value><<<g, 256, 0, s>>>(a, chunks, slices); },
           large(bytes_of((long long)a.T + a.R, a.m, bf16)));
  return hipGetLastError();
}

hipError_t launch_combine_rows(const RowsArgs& a, bool rows_bf16, bool out_bf16, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int slices = (a.m / 8 + 127) / 128;
  const unsigned g = wave_grid((long long)a.T * slices);
  dispatch(
      [&](auto rb, auto ob, auto big) {
        k_combine_rows<decltype(rb)::value, decltype(ob)::value, decltype(big)::value><<<g, 256, 0, s>>>(a, slices);
      },
      rows_bf16, out_bf16, large(bytes_of(a.R, a.m, rows_bf16) + bytes_of(a.T, a.m, out_bf16)));
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const RowsArgs& a, bool tok_bf16, bool rows_bf16, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  int waves = (a.m / 8 + 127) / 128;
  if (waves > 4) waves = 4;
  const unsigned g = a.T < kMaxGrid ? (unsigned)a.T : (unsigned)kMaxGrid;
  const int passes = (a.dw ? 1 : 0) + (a.out ? 1 : 0);
  dispatch(
      [&](auto tb, auto rb, auto big) {
        k_combine_rows_bwd<decltype(tb)::value, decltype(rb)::value, decltype(big)::value><<<g, waves * 64, 0, s>>>(a);
      },
      tok_bf16, rows_bf16, large(bytes_of(a.T, a.m, tok_bf16) + passes * bytes_of(a.R, a.m, rows_bf16)));
  return hipGetLastError();
}

}  // namespace moe
