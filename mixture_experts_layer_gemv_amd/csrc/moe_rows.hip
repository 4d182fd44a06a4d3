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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over a team of `waves` waves, the same bits in every lane.  `slot` is a
// [16] LDS row of the team; consecutive reductions use different rows, so one
// barrier each is enough: a row is written again only after a barrier that
// every wave reaches after reading it.
__device__ __forceinline__ float team_sum(float v, float* slot, int wave, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[wave] = v;
  __syncthreads();
  float r = 0.0f;
  for (int i = 0; i < waves; ++i) r += slot[i];
  return r;
}

// ---- norm -----------------------------------------------------------------------
//
// y = (x - mu) r gamma + beta, mu the row's mean (0 for the RMS norm), r = 1 /
// sqrt(mean((x - mu)^2) + eps).  One block per row, the row in registers (V
// vectors of 8 per thread), gamma and beta kept there from row to row.
template <bool BF16, int V, bool LAYER>
__global__ __launch_bounds__(V == 1 ? 256 : 1024) void k_norm_fwd(const NormArgs A) {
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
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const size_t row = (size_t)t * A.m;
    float f[V][8];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * NT;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[v][j] = 0.0f;
      if (i < mv) load8<BF16>(A.x, row + (size_t)i * 8, f[v]);
    }
    float mu = 0.0f;
    if constexpr (LAYER) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += f[v][j];
      mu = team_sum(s, red[0], wave, waves) * inv_m;
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
    // a block-wide barrier separates the rows' uses of red[1] for the RMS norm too
    const float var = team_sum(q, red[LAYER ? 1 : (t / gridDim.x) & 1], wave, waves) * inv_m;
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
        store8<BF16>(A.out, row + (size_t)i * 8, o);
      }
    }
  }
}

// The gradients.  With h = (x - mu) r and u = gamma dy:
//   dx = r (u - h <u, h> / m - [layer] <u, 1> / m)
//   dgamma = sum_t dy h,  dbeta = sum_t dy
// One block per row and step; each thread adds its columns' dy h and dy over
// the rows its block takes and writes them as one row of partial sums, which
// k_norm_wgrad adds in block order (the result does not depend on timing).
template <bool BF16, int V, bool LAYER>
__global__ __launch_bounds__(V == 1 ? 256 : 1024) void k_norm_bwd(const NormArgs A) {
  __shared__ float red[4][16];
  const int tid = threadIdx.x, NT = blockDim.x, wave = tid >> 6, waves = NT >> 6;
  const int mv = A.m / 8;
  const float inv_m = 1.0f / (float)A.m;
  float g[V][8], ag[V][8], ab[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * NT;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[v][j] = ag[v][j] = ab[v][j] = 0.0f;
    if (i < mv) load8<false>(A.gamma, (size_t)i * 8, g[v]);
  }
  int turn = 0;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 2) {
    const size_t row = (size_t)t * A.m;
    const float mu = LAYER ? A.mean[t] : 0.0f, r = A.rstd[t];
    float h[V][8], u[V][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * NT;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = u[v][j] = 0.0f;
      if (i < mv) {
        load8<BF16>(A.x, row + (size_t)i * 8, h[v]);
        load8<BF16>(A.dy, row + (size_t)i * 8, u[v]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[v][j] = (h[v][j] - mu) * r;
          ag[v][j] = fmaf(u[v][j], h[v][j], ag[v][j]);
          if (LAYER) ab[v][j] += u[v][j];
          u[v][j] *= g[v][j];
          s1 = fmaf(u[v][j], h[v][j], s1);
          if (LAYER) s2 += u[v][j];
        }
      }
    }
    if (!A.out) continue;
    s1 = wave_sum(s1);
    if (LAYER) s2 = wave_sum(s2);
    if (waves > 1) {
      if ((tid & 63) == 0) {
        red[turn][wave] = s1;
        if (LAYER) red[turn + 1][wave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
      for (int i = 0; i < waves; ++i) {
        s1 += red[turn][i];
        if (LAYER) s2 += red[turn + 1][i];
      }
    }
    s1 *= inv_m;
    s2 *= inv_m;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * NT;
      if (i < mv) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (LAYER ? u[v][j] - s2 - h[v][j] * s1 : u[v][j] - h[v][j] * s1) * r;
        store8<BF16>(A.out, row + (size_t)i * 8, o);
      }
    }
  }
  if (!A.partial) return;
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

// Sums the partial rows: a block owns 64 columns of one gradient (blockIdx.y:
// 0 gamma, 1 beta), its four waves a quarter of the rows each.
__global__ __launch_bounds__(256) void k_norm_wgrad(const float* __restrict__ partial, int blocks, int m,
                                                    float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float part[4][64];
  float* const out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = partial + (size_t)blockIdx.y * blocks * m;
  const int lo = (int)((long long)blocks * wave / 4), hi = (int)((long long)blocks * (wave + 1) / 4);
  float s = 0.0f;
  if (c < m)
    for (int b = lo; b < hi; ++b) s += p[(size_t)b * m + c];
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < m) out[c] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

// Blocks of a launch: its threads must stay below 2^32, and the kernels walk
// what is left.
constexpr int kMaxGrid = 1 << 22;
unsigned wave_grid(long long items) {  // four waves a block, an item each
  const long long blocks = (items + 3) / 4;
  return blocks < kMaxGrid ? (unsigned)blocks : (unsigned)kMaxGrid;
}

// Threads of a block for rows of m, with V vectors per thread.
int norm_vecs(int m) { return m <= 2048 ? 1 : 2; }
int norm_threads(int m) {
  const int per = 8 * norm_vecs(m);
  return ((m + per - 1) / per + 63) / 64 * 64;
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

}  // namespace

#define MOE_NORM(KERNEL, GRID)                                                                \
  do {                                                                                        \
    const int nt = norm_threads(a.m);                                                         \
    if (norm_vecs(a.m) == 1) {                                                                \
      if (bf16 && layer) KERNEL<true, 1, true><<<GRID, nt, 0, s>>>(a);                        \
      else if (bf16) KERNEL<true, 1, false><<<GRID, nt, 0, s>>>(a);                           \
      else if (layer) KERNEL<false, 1, true><<<GRID, nt, 0, s>>>(a);                          \
      else KERNEL<false, 1, false><<<GRID, nt, 0, s>>>(a);                                    \
    } else {                                                                                  \
      if (bf16 && layer) KERNEL<true, 2, true><<<GRID, nt, 0, s>>>(a);                        \
      else if (bf16) KERNEL<true, 2, false><<<GRID, nt, 0, s>>>(a);                           \
      else if (layer) KERNEL<false, 2, true><<<GRID, nt, 0, s>>>(a);                          \
      else KERNEL<false, 2, false><<<GRID, nt, 0, s>>>(a);                                    \
    }                                                                                         \
  } while (0)

hipError_t launch_norm_forward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const int most = cus * (2048 / norm_threads(a.m));
  const unsigned grid = (unsigned)(a.T < most ? a.T : most);
  MOE_NORM(k_norm_fwd, grid);
  return hipGetLastError();
}

int norm_backward_blocks(int T, int m, int cus) {
  const int nt = norm_threads(m);
  const int most = cus * (nt <= 512 ? 512 / nt : 1);
  return T < most ? T : most;
}

hipError_t launch_norm_backward(const NormArgs& a, bool bf16, bool layer, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.m > kNormMaxCols) return hipErrorInvalidValue;
  const unsigned grid = (unsigned)norm_backward_blocks(a.T, a.m, cus);
  MOE_NORM(k_norm_bwd, grid);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !a.partial) return e;
  k_norm_wgrad<<<dim3((unsigned)((a.m + 63) / 64), layer ? 2 : 1), 256, 0, s>>>(a.partial, (int)grid, a.m, a.dgamma,
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
