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
#include "moe_kernels.hpp"
#include "moe_rows.hpp"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// The row range of expert e, kept inside [0, R] whatever the offsets hold.
__device__ __forceinline__ int row_at(const I8Args& A, int e) {
  if (!A.offsets) return e ? A.R : 0;
  const int o = A.offsets[e];
  return o < 0 ? 0 : (o > A.R ? A.R : o);
}

// The x row of output row r, kept inside [0, T).
__device__ __forceinline__ int token_of(const I8Args& A, int r) {
  if (!A.perm) return r;
  const int t = A.perm[r] / A.topk;
  return t < 0 ? 0 : (t >= A.T ? A.T - 1 : t);
}

// Four consecutive channels n .. n + 3 of output row r (N is a multiple of 8).
template <bool YB>
__device__ __forceinline__ void store4(const I8Args& A, int e, int r, int t, int n, const i32x4_t& acc) {
  const float sx = A.sx[t];
  const float4 sw = *reinterpret_cast<const float4*>(A.sw + (size_t)e * A.N + n);
  const float o[4] = {(float)acc[0] * sx * sw.x, (float)acc[1] * sx * sw.y, (float)acc[2] * sx * sw.z,
                      (float)acc[3] * sx * sw.w};
  const size_t at = (size_t)r * A.N + n;
  if constexpr (YB) {
    const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{o[0], o[1]}, bf16x2_t));
    const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{o[2], o[3]}, bf16x2_t));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + at) = make_uint2(lo, hi);
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(A.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
  }
}

// A workgroup owns 16 output channels and up to 16 MT rows of one expert; its
// waves split the reduction and add their int32 sums in LDS.
template <int MT, bool YB>
__global__ __launch_bounds__(256) void k_i8_rows(const I8Args A, int pairs) {
  __shared__ i32x4_t part[4][MT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = (int)(blockIdx.x / (unsigned)pairs) * 16;
  int pair = (int)(blockIdx.x % (unsigned)pairs);
  int e = 0, row0 = 0, end = 0;
  for (; e < A.E; ++e) {
    row0 = row_at(A, e);
    end = row_at(A, e + 1);
    const int c = end > row0 ? (end - row0 + 16 * MT - 1) / (16 * MT) : 0;
    if (pair < c) break;
    pair -= c;
  }
  if (e == A.E) return;
  row0 += pair * 16 * MT;
  const int rows = min(16 * MT, end - row0);

  const int q = 16 * (lane >> 4);  // the lane's bytes of a 64-byte step
  const int n = min(n0 + (lane & 15), A.N - 1);
  const int8_t* wrow = A.w + ((size_t)e * A.N + n) * A.K + q;
  const int8_t* xrow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = row0 + min(16 * i + (lane & 15), rows - 1);
    xrow[i] = A.x + (size_t)token_of(A, r) * A.K + q;
  }
  i32x4_t acc[MT] = {};
  const int steps = (A.K + 63) / 64;
  const int lo = steps * wave / 4, hi = steps * (wave + 1) / 4;
  for (int s = lo; s < hi; ++s) {
    const int k = s * 64;
    const bool in = k + q < A.K;  // K is a multiple of 16
    const i32x4_t zero = {0, 0, 0, 0};
    const i32x4_t wv = in ? *reinterpret_cast<const i32x4_t*>(wrow + k) : zero;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const i32x4_t xv = in ? *reinterpret_cast<const i32x4_t*>(xrow[i] + k) : zero;
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // wave i finishes row tile i: a lane holds channels n0 + 4 (lane / 16) .. + 3
  // of row 16 i + lane % 16
  const int nn = n0 + 4 * (lane >> 4);
  for (int i = wave; i < MT; i += 4) {
    const i32x4_t sum = part[0][i][lane] + part[1][i][lane] + part[2][i][lane] + part[3][i][lane];
    const int r = 16 * i + (lane & 15);
    if (r < rows && nn < A.N) store4<YB>(A, e, row0 + r, token_of(A, row0 + r), nn, sum);
  }
}

}  // namespace

hipError_t launch_matmul_i8(const I8Args& a, bool y_bf16, int cus, hipStream_t s) {
  (void)cus;
  if (a.R <= 0) return hipSuccess;
  if (a.K <= 0 || a.K % 16 || a.K > kI8MaxK || a.N <= 0 || a.N % 8 || a.E < 1 || (!a.offsets && a.E != 1))
    return hipErrorInvalidValue;
  const long long pairs = (long long)a.R / 64 + (a.R < a.E ? a.R : a.E);
  const long long blocks = pairs * ((a.N + 15) / 16);
  if (blocks >= 1LL << 24) return hipErrorInvalidValue;
  if (y_bf16) k_i8_rows<4, true><<<(unsigned)blocks, 256, 0, s>>>(a, (int)pairs);
  else k_i8_rows<4, false><<<(unsigned)blocks, 256, 0, s>>>(a, (int)pairs);
  return hipGetLastError();
}

}  // namespace moe
