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

constexpr int kCols = 128;  // columns of a block

// 16 bytes; ONCE: of data that the caches need not keep (8192 x 4096: 61 -> 56 us; the
// rule is the row operators').
template <bool ONCE>
__device__ __forceinline__ u32x4_t load16(const char* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  else return *reinterpret_cast<const u32x4_t*>(p);
}

// The token groups that the gradients are computed in, each with a partial sum of
// Wr's: two blocks a CU over the column slabs, of 64 tokens or more.
int token_groups(int T, int m, int cus) {
  const long long slabs = (m + kCols - 1) / kCols, want = (2LL * cus + slabs - 1) / slabs, most = ((long long)T + 63) / 64;
  const long long g = want < most ? want : most;
  return (int)(g < 1 ? 1 : g);
}
int padded_experts(int E) { return (E + 15) / 16 * 16; }

// Sixteen bytes of a row's columns: eight in a row in bf16, twice four in fp32 (whole
// lines a load), of the 128 from c0; 0 where the row is not `live` or past m.
template <bool BF16, bool ONCE>
struct Cols {
  static constexpr int N = BF16 ? 1 : 2;
  u32x4_t v[N];
  __device__ __forceinline__ void load(const void* p, size_t row, int c0, int l16, int m, bool live) {
#pragma unroll
    for (int h = 0; h < N; ++h) {
      const int c = c0 + (BF16 ? 8 * l16 : 64 * h + 4 * l16);
      v[h] = u32x4_t{0, 0, 0, 0};
      if (live && c < m) v[h] = load16<ONCE>(static_cast<const char*>(p) + (row + c) * (BF16 ? 2 : 4));
    }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (BF16) return __uint_as_float(j & 1 ? v[0][j >> 1] & 0xFFFF0000u : v[0][j >> 1] << 16);
    else return __uint_as_float(v[j >> 2][j & 3]);
  }
  static __device__ __forceinline__ int column(int l16, int j) {
    return BF16 ? 8 * l16 + j : 64 * (j >> 2) + 4 * l16 + (j & 3);
  }
};

// The logits' gradient of tokens from .. from + TC - 1 in LDS, rows of STR values (0
// past token t1 and past the experts); with `store`, in memory too.  Every block
// computes what its tokens need rather than wait for a launch of its own that would.
template <int TC, int STR>
__device__ __forceinline__ void logits_gradient(const RouteGradArgs& A, float* lds, int from, int t1, bool store) {
  const int n = min(TC, t1 - from);
  constexpr int threads = 256;
  __syncthreads();
  if (A.dl_add) {
    for (int i = threadIdx.x; i < TC * STR; i += threads) {
      const int t = i / STR, e = i % STR;
      lds[i] = t < n && e < A.E ? A.dl_add[(size_t)(from + t) * A.E + e] : 0.0f;
    }
  } else {
    for (int i = threadIdx.x; i < TC * STR; i += threads) lds[i] = 0.0f;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {  // a thread a token
    const size_t at = (size_t)(from + threadIdx.x) * A.k;
    float* const d = lds + threadIdx.x * STR;
    float s = 0.0f;
#pragma unroll 4
    for (int j = 0; j < A.k; ++j) s = fmaf(A.w[at + j], A.dw[at + j], s);
#pragma unroll 4
    for (int j = 0; j < A.k; ++j) {
      const int e = A.idx[at + j];
      const float v = A.w[at + j] * (A.dw[at + j] - s);
      if (e >= 0 && e < A.E) d[e] += v;
    }
  }
  __syncthreads();
  if (store)
    for (int i = threadIdx.x; i < n * A.E; i += threads) A.dl[(size_t)from * A.E + i] = lds[i / A.E * STR + i % A.E];
}

// A block takes a slab of 128 columns of a token group: below gw the partial gradient
// of Wr, the others dx.  KK steps of four experts.
//
// 8192 x 4096, 8 experts: 56 us, 3.6 TB/s.  The gradient of Wr in a launch before dx's, joined in
// dx's: 69 us; in blocks of 64 columns and all tokens, without a join: 92 us; the
// logits' gradient in a launch of its own: 72 us.
template <bool BF16, int KK, bool ONCE>
__global__ __launch_bounds__(256, 2) void k_route_grad(const RouteGradArgs A, int slabs, int groups, int gw) {
  constexpr int EB = (KK + 3) / 4, EP = 16 * EB;
  constexpr int TC = KK <= 8 ? 256 : 128, STR = 4 * KK + 1;  // tokens of a chunk, its row (one bank further a token)
  constexpr int PART = 4 * 8 * 64 * 4;                     // 16 experts' sums of every wave
  __shared__ __attribute__((aligned(16))) float lds[TC * STR > PART ? TC * STR : PART];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, quart = lane >> 4, m = A.m;
  const bool wgrad = (int)blockIdx.x < gw;
  const int b = wgrad ? (int)blockIdx.x : (int)blockIdx.x - gw;
  const int slab = b % slabs, group = b / slabs, c0 = slab * kCols;
  const int t0 = (int)((long long)A.T * group / groups), t1 = (int)((long long)A.T * (group + 1) / groups);
  const bool store = slab == 0 && (!wgrad || gw == (int)gridDim.x);
  if (wgrad) {
    f32x4_t acc[EB][8];
    float sum[EB];
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      sum[e] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[e][j] = f32x4_t{0, 0, 0, 0};
    }
    for (int from = t0; from < t1; from += TC) {
      // a product takes four tokens, one per quarter of the wave; four products' rows are loaded together
      constexpr int AHEAD = 4;
      Cols<BF16, ONCE> x[AHEAD];
      auto fetch = [&](int i) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const int t = from + i + 4 * a + quart;
          x[a].load(A.x, (size_t)(t < t1 ? t : t0) * m, c0, l16, m, t < t1 && A.dwr);
        }
      };
      const int n = min(TC, t1 - from), first = 4 * AHEAD * wave;
      if (first < n) fetch(first);
      logits_gradient<TC, STR>(A, lds, from, t1, store);
      for (int i = first; i < n; i += 16 * AHEAD) {
        if (i != first) fetch(i);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const float* const d = lds + (i + 4 * a + quart) * STR;
#pragma unroll
          for (int e = 0; e < EB; ++e) {
            const float v = 16 * e + l16 < 4 * KK ? d[16 * e + l16] : 0.0f;
            sum[e] += v;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[e][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, x[a].at(j), acc[e][j], 0, 0, 0);
          }
        }
      }
    }
    // the waves' sums in order; lane: column l16 of set j, experts 16 e + 4 quart .. + 3
    float* const out = A.partial + (size_t)group * m * EP;
    f32x4_t* const part = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) part[(wave * 8 + j) * 64 + lane] = acc[e][j];
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * wave + h, c = c0 + Cols<BF16, ONCE>::column(l16, j);
        f32x4_t s = part[j * 64 + lane];
        for (int v = 1; v < 4; ++v) s += part[(v * 8 + j) * 64 + lane];
        if (c < m) *reinterpret_cast<f32x4_t*>(out + (size_t)c * EP + 16 * e + 4 * quart) = s;
      }
    }
    if (slab == 0)
#pragma unroll
      for (int e = 0; e < EB; ++e) {
        float s = sum[e];
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        __syncthreads();
        lds[wave * 64 + lane] = s;
        __syncthreads();
        if (wave == 0 && lane < 16)
          A.partial[(size_t)groups * m * EP + (size_t)group * EP + 16 * e + lane] =
              lds[lane] + lds[64 + lane] + lds[128 + lane] + lds[192 + lane];
      }
    return;
  }
  // dx: 16 tokens a step and wave.  Row r of the product's 16-column block q is column
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
      wr[q][kk] = A.dx && c < m && e < A.E ? A.wr[(size_t)c * A.E + e] : 0.0f;
    }
  constexpr int U = BF16 ? 4 : 8;  // vectors of a lane's columns, 16 bytes each
  for (int from = t0; from < t1; from += TC) {
    const int n = min(TC, t1 - from);
    u32x4_t add[U];
    auto col = [&](int u) { return c0 + (BF16 ? 32 * u + 8 * quart : 16 * u + 4 * quart); };
    auto fetch = [&](int i) {
      const int t = from + i + l16;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        add[u] = u32x4_t{0, 0, 0, 0};
        if (A.dx_add && t < t1 && col(u) < m)
          add[u] = load16<ONCE>(static_cast<const char*>(A.dx_add) + ((size_t)t * m + col(u)) * (BF16 ? 2 : 4));
      }
    };
    fetch(16 * wave);
    logits_gradient<TC, STR>(A, lds, from, t1, store);
    if (!A.dx) continue;
    for (int i = 16 * wave; i < n; i += 64) {
      const int t = from + i + l16;
      if (i != 16 * wave) fetch(i);
      float d[KK];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) d[kk] = lds[(i + l16) * STR + 4 * kk + quart];
      f32x4_t acc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        acc[q] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) acc[q] = __builtin_amdgcn_mfma_f32_16x16x4f32(wr[q][kk], d[kk], acc[q], 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        u32x4_t o;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if constexpr (BF16) {
            const f32x4_t& s = acc[2 * u + (h >> 1)];
            const f32x2_t v = {s[2 * (h & 1)] + __uint_as_float(add[u][h] << 16),
                               s[2 * (h & 1) + 1] + __uint_as_float(add[u][h] & 0xFFFF0000u)};
            o[h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
          } else {
            o[h] = __float_as_uint(acc[u][h] + __uint_as_float(add[u][h]));
          }
        }
        if (t < t1 && col(u) < m)
          *reinterpret_cast<u32x4_t*>(static_cast<char*>(A.dx) + ((size_t)t * m + col(u)) * (BF16 ? 2 : 4)) = o;
      }
    }
  }
}

// The token groups' partial sums added in order: thread (column, expert), then db.
__global__ __launch_bounds__(256) void k_route_join(const RouteGradArgs A, int groups, int EP) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, n = (long long)A.m * A.E;
  if (i >= n + A.E) return;
  const bool bias = i >= n;
  const int c = bias ? 0 : (int)(i / A.E), e = bias ? (int)(i - n) : (int)(i - (long long)c * A.E);
  const size_t step = bias ? (size_t)EP : (size_t)A.m * EP;
  const float* p = A.partial + (bias ? (size_t)groups * A.m * EP : (size_t)c * EP) + e;
  float* const out = bias ? A.db : A.dwr;
  if (!out) return;
  float s = 0.0f;
#pragma unroll 8
  for (int g = 0; g < groups; ++g) s += p[g * step];
  out[bias ? e : i] = s;
}

}  // namespace

size_t route_grad_bytes(int T, int m, int E, int cus) {
  return (size_t)token_groups(T, m, cus) * ((size_t)m + 1) * padded_experts(E) * sizeof(float);
}

hipError_t launch_route_backward(const RouteGradArgs& a, bool bf16, int cus, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  if (a.m <= 0 || a.m % 8 || a.E < 1 || a.E > 64 || a.k < 1 || a.k > 64) return hipErrorInvalidValue;
  const int groups = token_groups(a.T, a.m, cus);
  const bool wgrad = a.dwr || a.db;
  const int slabs = a.dx || a.dwr ? (a.m + kCols - 1) / kCols : 1;  // without them only the first slab's sums are wanted
  const long long one = (long long)slabs * groups, total = one * (wgrad && a.dx ? 2 : 1);
  if (total * 256 >= 1LL << 32) return hipErrorInvalidValue;
  const long long passes = (a.dwr ? 1 : 0) + (a.dx ? (a.dx_add ? 2 : 1) : 0);
  const bool large = passes * a.T * a.m * (bf16 ? 2 : 4) >= 128 << 20;
  auto go = [&](auto b, auto steps) {
    constexpr bool B = decltype(b)::value;
    constexpr int KK = decltype(steps)::value;
    const int gw = wgrad ? (int)one : 0;
    if (large) k_route_grad<B, KK, true><<<(unsigned)total, 256, 0, s>>>(a, slabs, groups, gw);
    else k_route_grad<B, KK, false><<<(unsigned)total, 256, 0, s>>>(a, slabs, groups, gw);
  };
  auto by_experts = [&](auto b) {
    if (a.E <= 8) go(b, std::integral_constant<int, 2>{});
    else if (a.E <= 16) go(b, std::integral_constant<int, 4>{});
    else if (a.E <= 32) go(b, std::integral_constant<int, 8>{});
    else if (a.E <= 48) go(b, std::integral_constant<int, 12>{});
    else go(b, std::integral_constant<int, 16>{});
  };
  if (bf16) by_experts(std::true_type{});
  else by_experts(std::false_type{});
  if (hipError_t e = hipGetLastError(); e != hipSuccess || !wgrad) return e;
  const long long n = ((long long)a.m + 1) * a.E;
  k_route_join<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, groups, padded_experts(a.E));
  return hipGetLastError();
}

}  // namespace moe
