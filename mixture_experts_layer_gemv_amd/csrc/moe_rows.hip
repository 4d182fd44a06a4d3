// Row operators around the experts for gfx950: the input norm's forward and
// backward pass, token rows copied into expert order, expert rows combined
// back to their tokens, and the gradients of both.
//
// All of them move each row through HBM once and do 1 to 16 operations per
// element, so bytes bound them; sums and statistics are fp32, and a value is
// rounded once, when it is stored.
#include "moe_kernels.hpp"
#include "moe_rows.hpp"

namespace moe {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Eight consecutive elements starting at element i (a multiple of 8).
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&f)[8]) {
  if constexpr (BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

// Two fp32 -> two bf16, round to nearest even (the hardware conversion).
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&f)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// One DPP step of a wave sum: v plus the value that CTRL moves to each lane
// (0 where none does).
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

// Eight elements as loaded, converted only when they are used.
template <bool BF16>
struct Raw8 {
  uint4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    if constexpr (BF16) {
      v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    } else {
      v[0] = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)[0];
      v[1] = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)[1];
    }
  }
  __device__ __forceinline__ void clear() {
    v[0] = make_uint4(0, 0, 0, 0);
    if constexpr (!BF16) v[1] = v[0];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (BF16) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
    }
  }
};

// Adds the waves' values of a team: slot[0 .. waves) in LDS, written before a barrier.
__device__ __forceinline__ float slot_sum(const float* slot, int waves) {
  float r = 0.0f;
  for (int i = 0; i < waves; ++i) r += slot[i];
  return r;
}

// ---- norm -----------------------------------------------------------------------
//
// y = (x - mu) r gamma + beta, mu the row's mean (0 for the RMS norm), r = 1 /
// sqrt(mean((x - mu)^2) + eps).  One block per row, the row in registers (V
// vectors of 8 per thread), gamma and beta kept there from row to row; the
// next row is loaded while this one is summed.
template <bool BF16, int V, bool LAYER>
__global__ __launch_bounds__(V == 1 ? 256 : 1024) void k_norm_fwd(const NormArgs A) {
  // consecutive sums use different rows, so one barrier each is enough: a row
  // is written again only after a barrier that every wave reaches after reading it
  __shared__ float red[2][16];
  const int tid = threadIdx.x, NT = blockDim.x, wave = tid >> 6, waves = NT >> 6;
  const int mv = A.m / 8;
  const float inv_m = 1.0f / (float)A.m;
  float g[V][8], b[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * NT;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[v][j] = b[v][j] = 0.0f;
    if (i < mv) {
      load8<false>(A.gamma, (size_t)i * 8, g[v]);
      if (LAYER && A.beta) load8<false>(A.beta, (size_t)i * 8, b[v]);
    }
  }
  Raw8<BF16> next[V];
  auto fetch = [&](int t) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      next[v].clear();
      if (tid + v * NT < mv) next[v].load(A.x, (size_t)t * A.m + (size_t)(tid + v * NT) * 8);
    }
  };
  auto team_sum = [&](float v, float* slot) {
    v = wave_sum(v);
    if (waves == 1) return v;
    if ((tid & 63) == 0) slot[wave] = v;
    __syncthreads();
    return slot_sum(slot, waves);
  };
  fetch(blockIdx.x);
  int turn = 0;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 1) {
    float f[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) next[v].get(f[v]);
    if (t + (int)gridDim.x < A.T) fetch(t + gridDim.x);
    float mu = 0.0f;
    if constexpr (LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += f[v][j];
      mu = team_sum(s, red[0]) * inv_m;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = tid + v * NT < mv;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = in ? f[v][j] - mu : 0.0f;
        f[v][j] = d;
        q = fmaf(d, d, q);
      }
    }
    const float var = team_sum(q, red[LAYER ? 1 : turn]) * inv_m;
    const float r = 1.0f / sqrtf(var + A.eps);
    if (tid == 0) {
      if (LAYER && A.mean) A.mean[t] = mu;
      if (A.rstd) A.rstd[t] = r;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * NT;
      if (i < mv) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = LAYER ? fmaf(f[v][j] * r, g[v][j], b[v][j]) : f[v][j] * r * g[v][j];
        store8<BF16>(A.out, (size_t)t * A.m + (size_t)i * 8, o);
      }
    }
  }
}

// The gradients.  With h = (x - mu) r and u = gamma dy:
//   dx = r (u - h <u, h> / m - [layer] <u, 1> / m)
//   dgamma = sum_t dy h,  dbeta = sum_t dy
// A block holds several teams of NT threads, one row each per step; a thread
// adds its columns' dy h and dy over the rows its team takes.  The teams' sums
// are added in LDS, the block writes them as one row of partial sums, and
// k_norm_wgrad adds those in block order: nothing depends on timing.
template <bool BF16, int V, bool LAYER, int MAXT>
__global__ __launch_bounds__(MAXT) __attribute__((amdgpu_waves_per_eu(4))) void k_norm_bwd(const NormArgs A, int NT) {
  __shared__ float red[4][16];
  extern __shared__ float acc[];  // gamma [m]; after the rows, with more than one team, [2][m] sums
  const int team = threadIdx.x / NT, teams = blockDim.x / NT, tid = threadIdx.x - team * NT;
  const int wave = threadIdx.x >> 6, waves = NT >> 6, first = team * waves;  // the team's first wave
  const int mv = A.m / 8;
  const float inv_m = 1.0f / (float)A.m;
  float ag[V][8], ab[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * NT;
#pragma unroll
    for (int j = 0; j < 8; ++j) ag[v][j] = ab[v][j] = 0.0f;
    if (i < mv && team == 0) {
      float f[8];
      load8<false>(A.gamma, (size_t)i * 8, f);
      store8<false>(acc, (size_t)i * 8, f);
    }
  }
  __syncthreads();
  Raw8<BF16> nx[V], ny[V];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](long long t) {  // rows past the last are zeros
#pragma unroll
    for (int v = 0; v < V; ++v) {
      nx[v].clear();
      ny[v].clear();
      if (t < A.T && tid + v * NT < mv) {
        nx[v].load(A.x, (size_t)t * A.m + (size_t)(tid + v * NT) * 8);
        ny[v].load(A.dy, (size_t)t * A.m + (size_t)(tid + v * NT) * 8);
      }
    }
    nmu = LAYER && t < A.T ? A.mean[t] : 0.0f;
    nr = t < A.T ? A.rstd[t] : 0.0f;
  };
  const long long stride = (long long)gridDim.x * teams;
  fetch((long long)blockIdx.x * teams + team);
  int turn = 0;
  for (long long t0 = (long long)blockIdx.x * teams; t0 < A.T; t0 += stride, turn ^= 2) {  // the same count for every team
    const long long t = t0 + team;
    const float mu = nmu, r = nr;
    float h[V][8], u[V][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      nx[v].get(h[v]);
      ny[v].get(u[v]);
    }
    if (t0 + stride < A.T) fetch(t + stride);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = tid + v * NT < mv;
      float g[8];
      load8<false>(acc, in ? (size_t)(tid + v * NT) * 8 : 0, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[v][j] = in ? (h[v][j] - mu) * r : 0.0f;
        ag[v][j] = fmaf(u[v][j], h[v][j], ag[v][j]);
        if (LAYER) ab[v][j] += u[v][j];
        u[v][j] *= g[j];
        s1 = fmaf(u[v][j], h[v][j], s1);
        if (LAYER) s2 += u[v][j];
      }
    }
    if (!A.out) continue;
    s1 = wave_sum(s1);
    if (LAYER) s2 = wave_sum(s2);
    if (waves > 1) {
      if ((threadIdx.x & 63) == 0) {
        red[turn][wave] = s1;
        if (LAYER) red[turn + 1][wave] = s2;
      }
      __syncthreads();
      s1 = slot_sum(red[turn] + first, waves);
      if (LAYER) s2 = slot_sum(red[turn + 1] + first, waves);
    }
    s1 *= inv_m;
    s2 *= inv_m;
    if (t >= A.T) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * NT;
      if (i < mv) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (LAYER ? u[v][j] - s2 - h[v][j] * s1 : u[v][j] - h[v][j] * s1) * r;
        store8<BF16>(A.out, (size_t)t * A.m + (size_t)i * 8, o);
      }
    }
  }
  if (!A.partial) return;
  for (int k = 1; k < teams; ++k) {
    __syncthreads();
    if (team == k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = tid + v * NT;
        if (i < mv) {
          store8<false>(acc, (size_t)i * 8, ag[v]);
          if (LAYER) store8<false>(acc + A.m, (size_t)i * 8, ab[v]);
        }
      }
    }
    __syncthreads();
    if (team == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = tid + v * NT;
        if (i < mv) {
          float f[8];
          load8<false>(acc, (size_t)i * 8, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) ag[v][j] += f[j];
          if (LAYER) {
            load8<false>(acc + A.m, (size_t)i * 8, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) ab[v][j] += f[j];
          }
        }
      }
    }
  }
  if (team) return;
  float* const pg = A.partial + (size_t)blockIdx.x * A.m;
  float* const pb = pg + (size_t)gridDim.x * A.m;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * NT;
    if (i < mv) {
      store8<false>(pg, (size_t)i * 8, ag[v]);
      if (LAYER) store8<false>(pb, (size_t)i * 8, ab[v]);
    }
  }
}

// Sums the partial rows: a block owns 32 columns of one gradient (blockIdx.y:
// 0 gamma, 1 beta), eight lanes of four columns; its 64 groups of lanes take
// every 64th row, then add up in LDS.
__global__ __launch_bounds__(512) void k_norm_wgrad(const float* __restrict__ partial, int blocks, int m,
                                                    float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float4 part[64][8];
  float* const out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int q = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * q;
  const float* p = partial + (size_t)blockIdx.y * blocks * m + c;
  float4 s = make_float4(0, 0, 0, 0);
  if (c < m)
#pragma unroll 4
    for (int b = grp; b < blocks; b += 64) {
      const float4 f = *reinterpret_cast<const float4*>(p + (size_t)b * m);
      s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
    }
  part[grp][q] = s;
#pragma unroll
  for (int n = 32; n; n >>= 1) {
    __syncthreads();
    if (grp < n) {
      const float4 f = part[grp + n][q];
      s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
      part[grp][q] = s;
    }
  }
  if (grp == 0 && c < m) *reinterpret_cast<float4*>(out + c) = s;
}

// ---- rows in expert order ---------------------------------------------------------
//
// One wave per (token, 256-vector slice of its row).  An assignment's row is
// inv[t*k + j]; a value outside [0, R) means that it has none (dropped): it
// is not written, adds nothing and gets a zero weight gradient.
constexpr int kSlice = 4;  // 8-element vectors per lane

// The k rows of token t, one per lane (k <= 64).
__device__ __forceinline__ int token_rows(const RowsArgs& A, int t, int lane) {
  const int r = lane < A.k ? A.inv[(size_t)t * A.k + lane] : -1;
  return r >= 0 && r < A.R ? r : -1;
}

// out[inv[t*k+j]] = tok[t]: 16-byte chunks, whatever the type.
__global__ __launch_bounds__(256) void k_permute_rows(const RowsArgs A, int chunks, int slices) {
  const int lane = threadIdx.x & 63;
  const long long items = (long long)A.T * slices;
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += 4LL * gridDim.x) {
    const int t = (int)(item / slices), c0 = (int)(item % slices) * 64 * kSlice + lane;
    const int mine = token_rows(A, t, lane);
    const uint4* src = static_cast<const uint4*>(A.tok) + (size_t)t * chunks;
    uint4 v[kSlice];
#pragma unroll
    for (int i = 0; i < kSlice; ++i)
      if (c0 + 64 * i < chunks) v[i] = src[c0 + 64 * i];
    for (int j = 0; j < A.k; ++j) {
      const int r = __builtin_amdgcn_readlane(mine, j);
      if (r < 0) continue;
      uint4* dst = static_cast<uint4*>(A.out) + (size_t)r * chunks;
#pragma unroll
      for (int i = 0; i < kSlice; ++i)
        if (c0 + 64 * i < chunks) dst[c0 + 64 * i] = v[i];
    }
  }
}

// out[t] = sum_j w[t,j] rows[inv[t*k+j]], in order of j.
template <bool RB, bool OB>
__global__ __launch_bounds__(256) void k_combine_rows(const RowsArgs A, int slices) {
  constexpr int V = 2;
  const int lane = threadIdx.x & 63, mv = A.m / 8;
  const long long items = (long long)A.T * slices;
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < items; item += 4LL * gridDim.x) {
    const int t = (int)(item / slices), c0 = (int)(item % slices) * 64 * V + lane;
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
      for (int v = 0; v < V; ++v)
        if (c0 + 64 * v < mv) {
          float f[8];
          load8<RB>(A.rows, (size_t)r * A.m + (size_t)(c0 + 64 * v) * 8, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) s[v][q] = fmaf(wj, f[q], s[v][q]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c0 + 64 * v < mv) store8<OB>(A.out, (size_t)t * A.m + (size_t)(c0 + 64 * v) * 8, s[v]);
  }
}

// The combine's gradient, one block of up to four waves per token:
// out[inv[t*k+j]] = w[t,j] dy[t], dw[t,j] = <dy[t], rows[inv[t*k+j]]>.
template <bool TB, bool RB>
__global__ __launch_bounds__(256) void k_combine_rows_bwd(const RowsArgs A) {
  constexpr int V = 2;
  __shared__ float dots[4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, NT = blockDim.x, waves = NT >> 6;
  const int mv = A.m / 8;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const int mine = token_rows(A, t, lane);
    const float wl = lane < A.k && A.w ? A.w[(size_t)t * A.k + lane] : 0.0f;
    dots[wave][lane] = 0.0f;
    for (int c0 = tid; c0 < (mv + 63) / 64 * 64; c0 += NT * V) {
      float d[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * NT;
#pragma unroll
        for (int q = 0; q < 8; ++q) d[v][q] = 0.0f;
        if (c < mv) load8<TB>(A.tok, (size_t)t * A.m + (size_t)c * 8, d[v]);
      }
      for (int j = 0; j < A.k; ++j) {
        const int r = __builtin_amdgcn_readlane(mine, j);
        if (r < 0) continue;
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = c0 + v * NT;
          if (c < mv) {
            const size_t at = (size_t)r * A.m + (size_t)c * 8;
            if (A.dw) {
              float f[8];
              load8<RB>(A.rows, at, f);
#pragma unroll
              for (int q = 0; q < 8; ++q) dot = fmaf(d[v][q], f[q], dot);
            }
            if (A.out) {
              float o[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) o[q] = wj * d[v][q];
              store8<RB>(A.out, at, o);
            }
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

// Threads of a team (one row) of the norm kernels, with V vectors per thread.
int norm_vecs(int m) { return m <= 2048 ? 1 : 2; }
int norm_threads(int m) {
  const int per = 8 * norm_vecs(m);
  return ((m + per - 1) / per + 63) / 64 * 64;
}
// Teams of a block and blocks per CU of the backward pass.
int norm_teams(int m) { return norm_threads(m) <= 512 ? 512 / norm_threads(m) : 1; }

}  // namespace

#define MOE_NORM(KERNEL, ...)                               \
  do {                                                      \
    if (bf16 && layer) KERNEL(true, true)<<<__VA_ARGS__;     \
    else if (bf16) KERNEL(true, false)<<<__VA_ARGS__;        \
    else if (layer) KERNEL(false, true)<<<__VA_ARGS__;       \
    else KERNEL(false, false)<<<__VA_ARGS__;                 \
  } while (0)

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const int nt = norm_threads(a.m), most = cus * (2048 / nt);
  const unsigned grid = (unsigned)(a.T < most ? a.T : most);
#define MOE_FWD1(B, L) k_norm_fwd<B, 1, L>
#define MOE_FWD2(B, L) k_norm_fwd<B, 2, L>
  if (norm_vecs(a.m) == 1) MOE_NORM(MOE_FWD1, grid, nt, 0, s>>>(a));
  else MOE_NORM(MOE_FWD2, grid, nt, 0, s>>>(a));
#undef MOE_FWD1
#undef MOE_FWD2
  return hipGetLastError();
}

int norm_backward_blocks(int T, int m, int cus) {
  const int teams = norm_teams(m), most = 2 * cus;
  const long long blocks = ((long long)T + teams - 1) / teams;
  return blocks < most ? (int)blocks : most;
}

hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)norm_backward_blocks(a.T, a.m, cus);
  const int nt = norm_threads(a.m), teams = norm_teams(a.m), threads = nt * teams;
  const size_t lds = (teams > 1 ? 2 : 1) * sizeof(float) * (size_t)a.m;
#define MOE_BWD1(B, L) k_norm_bwd<B, 1, L, 512>
#define MOE_BWD2(B, L) k_norm_bwd<B, 2, L, 512>
#define MOE_BWD3(B, L) k_norm_bwd<B, 2, L, 1024>
  if (norm_vecs(a.m) == 1) MOE_NORM(MOE_BWD1, grid, threads, lds, s>>>(a, nt));
  else if (threads <= 512) MOE_NORM(MOE_BWD2, grid, threads, lds, s>>>(a, nt));
  else MOE_NORM(MOE_BWD3, grid, threads, lds, s>>>(a, nt));
#undef MOE_BWD1
#undef MOE_BWD2
#undef MOE_BWD3
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.partial) return e;
  k_norm_wgrad<<<dim3((unsigned)((a.m + 31) / 32), layer ? 2 : 1), 512, 0, s>>>(a.partial, (int)grid, a.m, a.dgamma,
                                                                               layer ? a.dbeta : nullptr);
  return hipGetLastError();
}
#undef MOE_NORM

hipError_t launch_permute_rows(const RowsArgs& a, bool bf16, hipStream_t s) {
  if (a.T <= 0 || a.R <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int chunks = bf16 ? a.m / 8 : a.m / 4;
  const int slices = (chunks + 64 * kSlice - 1) / (64 * kSlice);
  k_permute_rows<<<wave_grid((long long)a.T * slices), 256, 0, s>>>(a, chunks, slices);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const RowsArgs& a, bool rows_bf16, bool out_bf16, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int slices = (a.m / 8 + 127) / 128;
  const unsigned g = wave_grid((long long)a.T * slices);
  if (rows_bf16 && out_bf16) k_combine_rows<true, true><<<g, 256, 0, s>>>(a, slices);
  else if (rows_bf16) k_combine_rows<true, false><<<g, 256, 0, s>>>(a, slices);
  else if (out_bf16) k_combine_rows<false, true><<<g, 256, 0, s>>>(a, slices);
  else k_combine_rows<false, false><<<g, 256, 0, s>>>(a, slices);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const RowsArgs& a, bool tok_bf16, bool rows_bf16, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  int waves = (a.m / 8 + 127) / 128;
  if (waves > 4) waves = 4;
  const unsigned g = a.T < kMaxGrid ? (unsigned)a.T : (unsigned)kMaxGrid;
  if (tok_bf16 && rows_bf16) k_combine_rows_bwd<true, true><<<g, waves * 64, 0, s>>>(a);
  else if (tok_bf16) k_combine_rows_bwd<true, false><<<g, waves * 64, 0, s>>>(a);
  else if (rows_bf16) k_combine_rows_bwd<false, true><<<g, waves * 64, 0, s>>>(a);
  else k_combine_rows_bwd<false, false><<<g, waves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
