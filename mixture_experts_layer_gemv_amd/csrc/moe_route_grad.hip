// The gradient of the routing for gfx950.  With l = x Wr + b, the k chosen logits
// of a token softmaxed to gate weights w:
//   dl[t][e] = add[t][e] + sum over j with idx[t][j] = e of w_j (dw_j - sum_i w_i dw_i)
//   dx = dx_add + dl Wr^T,  dWr = x^T dl,  db = sum_t dl
// All products run on the fp32 matrix cores (16 x 16 x 4), whose operands are
// single fp32 values a lane: x and Wr are used as they lie in memory.  x and
// dx_add are read and dx is written once: bytes bound it.
#include <type_traits>

#include "moe_gated.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kCols = 128;  // columns of a wave

// The token groups that the gradient of Wr is summed in, each with a partial sum
// of its own: two blocks a CU over the column slabs, of 64 tokens or more.
int token_groups(int T, int m, int cus) {
  const long long slabs = (m + kCols - 1) / kCols, want = (2LL * cus + slabs - 1) / slabs, most = ((long long)T + 63) / 64;
  const long long g = want < most ? want : most;
  return (int)(g < 1 ? 1 : g);
}
int padded_experts(int E) { return E <= 16 ? 16 : E <= 32 ? 32 : 64; }

// One wave a token: lane j holds choice j, then lane e logit e.
__global__ __launch_bounds__(256) void k_route_dl(const RouteGradArgs A) {
  const int lane = threadIdx.x & 63;
  for (long long i = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); i < A.T; i += 4LL * gridDim.x) {
    const size_t t = (size_t)i;
    const bool mine = lane < A.k;
    const float w = mine ? A.w[t * A.k + lane] : 0.0f, dw = mine ? A.dw[t * A.k + lane] : 0.0f;
    const int id = mine ? A.idx[t * A.k + lane] : -1;
    float s = w * dw;
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    const float v = w * (dw - s);
    float dl = lane < A.E && A.dl_add ? A.dl_add[t * A.E + lane] : 0.0f;
    for (int j = 0; j < A.k; ++j)
      if (__builtin_amdgcn_readlane(id, j) == lane) dl += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
    if (lane < A.E) A.dl[t * A.E + lane] = dl;
  }
}

// Eight columns of a lane, of the 128 from c0: eight together in bf16, twice four
// in fp32 (whole lines a load); 0 where the row is not `live` or past m.
template <bool BF16>
__device__ __forceinline__ int lane_col(int l16, int j) {
  return BF16 ? 8 * l16 + j : (j < 4 ? 4 * l16 + j : 64 + 4 * l16 + j - 4);
}
template <bool BF16>
__device__ __forceinline__ void load_cols(const void* p, size_t row, int c0, int l16, int m, bool live, float (&f)[8]) {
  const u32x4_t zero = {0, 0, 0, 0};
  if constexpr (BF16) {
    const int c = c0 + 8 * l16;
    const u32x4_t v = live && c < m ? *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + row + c) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(v[j] << 16);
      f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 64 * h + 4 * l16;
      const u32x4_t v = live && c < m ? *reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p) + row + c) : zero;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * h + j] = __uint_as_float(v[j]);
    }
  }
}

// KK steps of four experts.  Blocks below gw take the gradient of Wr (slab of 128
// columns, token group), the others dx.
template <bool BF16, int KK>
__global__ __launch_bounds__(256) void k_route_grad(const RouteGradArgs A, int slabs, int groups, int gw) {
  constexpr int EB = KK < 4 ? 1 : KK / 4, EP = 16 * EB;
  __shared__ f32x4_t part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, quart = lane >> 4;
  const int b = (int)blockIdx.x < gw ? (int)blockIdx.x : (int)blockIdx.x - gw;
  const int slab = b % slabs, group = b / slabs, c0 = slab * kCols;
  const int t0 = (int)((long long)A.T * group / groups), t1 = (int)((long long)A.T * (group + 1) / groups);
  if ((int)blockIdx.x < gw) {
    f32x4_t acc[EB][8];
    float sum[EB];
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      sum[e] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[e][j] = f32x4_t{0, 0, 0, 0};
    }
    // four tokens a step, one per quarter of the wave
    for (int t4 = t0 + 4 * wave; t4 < t1; t4 += 16) {
      const int t = t4 + quart;
      const bool live = t < t1;
      float f[8];
      load_cols<BF16>(A.x, (size_t)(live ? t : t0) * A.m, c0, l16, A.m, live && A.dwr, f);
#pragma unroll
      for (int e = 0; e < EB; ++e) {
        const int id = 16 * e + l16;
        const float d = live && id < A.E ? A.dl[(size_t)t * A.E + id] : 0.0f;
        sum[e] += d;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(d, f[j], acc[e][j], 0, 0, 0);
      }
    }
    // the four waves' sums in order; lane: column l16 of set j, experts 16 e + 4 quart .. + 3
    float* const out = A.partial + (size_t)group * A.m * EP;
#pragma unroll
    for (int e = 0; e < EB; ++e) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        __syncthreads();
        part[wave][lane] = acc[e][j];
        __syncthreads();
        const int c = c0 + lane_col<BF16>(l16, j);
        if (wave == 0 && c < A.m)
          *reinterpret_cast<f32x4_t*>(out + (size_t)c * EP + 16 * e + 4 * quart) =
              part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane];
      }
      if (slab == 0) {
        __syncthreads();
        float s = sum[e];
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        part[wave][lane][0] = s;
        __syncthreads();
        if (wave == 0 && lane < 16)
          A.partial[(size_t)groups * A.m * EP + (size_t)group * EP + 16 * e + lane] =
              part[0][lane][0] + part[1][lane][0] + part[2][lane][0] + part[3][lane][0];
      }
    }
    return;
  }
  // dx: 16 tokens a step.  Row r of the product's 16-column block q is column
  // column(q, r), so that a lane's four rows of two blocks are eight columns in
  // a row in bf16.
  auto column = [&](int q, int r) {
    return BF16 ? 32 * (q >> 1) + 8 * (r >> 2) + 4 * (q & 1) + (r & 3) : 16 * q + r;
  };
  float wr[8][KK];
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int c = c0 + column(q, l16), e = 4 * kk + quart;
      wr[q][kk] = c < A.m && e < A.E ? A.wr[(size_t)c * A.E + e] : 0.0f;
    }
  for (int t16 = t0 + 16 * wave; t16 < t1; t16 += 64) {
    const int t = t16 + l16;
    const bool live = t < t1;
    float d[KK];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int e = 4 * kk + quart;
      d[kk] = live && e < A.E ? A.dl[(size_t)t * A.E + e] : 0.0f;
    }
    f32x4_t acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      acc[q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) acc[q] = __builtin_amdgcn_mfma_f32_16x16x4f32(wr[q][kk], d[kk], acc[q], 0, 0, 0);
    }
    if (!live) continue;
    const size_t row = (size_t)t * A.m;
    if constexpr (BF16) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + 32 * u + 8 * quart;
        if (c >= A.m) continue;
        u32x4_t a = {0, 0, 0, 0}, o;
        if (A.dx_add) a = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(A.dx_add) + row + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t& s = acc[2 * u + (i >> 1)];
          const f32x2_t v = {s[2 * (i & 1)] + __uint_as_float(a[i] << 16), s[2 * (i & 1) + 1] + __uint_as_float(a[i] & 0xFFFF0000u)};
          o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
        }
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(A.dx) + row + c) = o;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int c = c0 + 16 * q + 4 * quart;
        if (c >= A.m) continue;
        f32x4_t s = acc[q];
        if (A.dx_add) s += *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(A.dx_add) + row + c);
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(A.dx) + row + c) = s;
      }
    }
  }
}

// The token groups' partial sums added in order: thread (column, expert), then db.
__global__ __launch_bounds__(256) void k_route_join(const RouteGradArgs A, int groups, int EP) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long n = (long long)A.m * A.E;
  if (i >= n + A.E) return;
  const bool bias = i >= n;
  const int c = bias ? 0 : (int)(i / A.E), e = bias ? (int)(i - n) : (int)(i - (long long)c * A.E);
  const size_t step = bias ? (size_t)EP : (size_t)A.m * EP;
  const float* p = A.partial + (bias ? (size_t)groups * A.m * EP : (size_t)c * EP) + e;
  float s = 0.0f;
  for (int g = 0; g < groups; ++g) s += p[g * step];
  if (bias) {
    if (A.db) A.db[e] = s;
  } else if (A.dwr) {
    A.dwr[i] = s;
  }
}

}  // namespace

size_t route_grad_bytes(int T, int m, int E, int cus) {
  return (size_t)token_groups(T, m, cus) * ((size_t)m + 1) * padded_experts(E) * sizeof(float);
}

hipError_t launch_route_backward(const RouteGradArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.E < 1 || a.E > 64 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int blocks = (int)(((long long)a.T + 3) / 4 < 1 << 22 ? ((long long)a.T + 3) / 4 : 1 << 22);
  k_route_dl<<<blocks, 256, 0, s>>>(a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const int slabs = (a.m + kCols - 1) / kCols, groups = token_groups(a.T, a.m, cus);
  const bool wgrad = a.dwr || a.db;
  const long long one = (long long)slabs * groups, total = one * ((wgrad ? 1 : 0) + (a.dx ? 1 : 0));
  if (total * 256 >= 1LL << 32) return hipErrorInvalidValue;
  if (total) {
    auto go = [&](auto b) {
      constexpr bool B = decltype(b)::value;
      const int gw = wgrad ? (int)one : 0;
      const unsigned grid = (unsigned)total;
      if (a.E <= 8) k_route_grad<B, 2><<<grid, 256, 0, s>>>(a, slabs, groups, gw);
      else if (a.E <= 16) k_route_grad<B, 4><<<grid, 256, 0, s>>>(a, slabs, groups, gw);
      else if (a.E <= 32) k_route_grad<B, 8><<<grid, 256, 0, s>>>(a, slabs, groups, gw);
      else k_route_grad<B, 16><<<grid, 256, 0, s>>>(a, slabs, groups, gw);
    };
    if (bf16) go(std::true_type{});
    else go(std::false_type{});
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!wgrad) return hipSuccess;
  const int EP = padded_experts(a.E);
  const long long n = ((long long)a.m + 1) * a.E;
  k_route_join<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, groups, EP);
  return hipGetLastError();
}

}  // namespace moe
