// quarot_fp8_gemm and quarot_fp8_gated_gemm: products of e4m3 codes with block
// scales on both operands.
//
//   P[i, j] = sum_b a_scale[b, i] w_scale[j / 128, b] sum_{k in block b} a[i, k] w[j, k]
//   gemm:  y = P rounded to fp16 / bf16
//   gated: z = silu(P_gate) P_up in fp32, quantized to e4m3 with a scale for
//          each token and 128 columns
//
// One CTA per 32 tokens x 128 columns on the CUDA cores.
#include <cuda_fp8.h>

#include "fp8.cuh"

namespace quarot {
namespace fp8 {
namespace gemm {

constexpr int TM = 32, TN = BLK, TK = 32;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3);
  return __half2float(__half(h));
}

template <bool GATED, typename T>
__global__ void __launch_bounds__(256)
fp8_gemm_kernel(const uint8_t* __restrict__ a, const float* __restrict__ as, const uint8_t* __restrict__ w0,
                const float* __restrict__ ws0, const uint8_t* __restrict__ w1, const float* __restrict__ ws1, int M,
                int N, int K, T* __restrict__ y, uint8_t* __restrict__ q, float* __restrict__ qs) {
  constexpr int NW = GATED ? 2 : 1;
  __shared__ float sa[TM][TK + 1], sw[NW][TN][TK + 1];
  const int nblk_n = (N + TN - 1) / TN, nkb = (K + BLK - 1) / BLK;
  const int nb = int(blockIdx.x) % nblk_n;
  const int m0 = int(blockIdx.x) / nblk_n * TM, n0 = nb * TN;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[NW][4][4] = {};
  for (int kb = 0; kb < nkb; ++kb) {
    float part[NW][4][4] = {};
    for (int k0 = kb * BLK; k0 < min(K, (kb + 1) * BLK); k0 += TK) {
      __syncthreads();
      for (int i = threadIdx.x; i < TM * TK; i += 256) {
        const int r = i / TK, c = i % TK;
        sa[r][c] = m0 + r < M && k0 + c < K ? e4m3_value(a[size_t(m0 + r) * K + k0 + c]) : 0.f;
      }
      for (int i = threadIdx.x; i < TN * TK; i += 256) {
        const int r = i / TK, c = i % TK;
        const bool in = n0 + r < N && k0 + c < K;
        sw[0][r][c] = in ? e4m3_value(w0[size_t(n0 + r) * K + k0 + c]) : 0.f;
        if constexpr (GATED) sw[1][r][c] = in ? e4m3_value(w1[size_t(n0 + r) * K + k0 + c]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < TK; ++k)
#pragma unroll
        for (int p = 0; p < NW; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              part[p][i][j] = fmaf(sa[4 * ty + i][k], sw[p][tx + 32 * j][k], part[p][i][j]);
    }
#pragma unroll
    for (int p = 0; p < NW; ++p) {
      const float wsc = (p == 0 ? ws0 : ws1)[size_t(nb) * nkb + kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + 4 * ty + i;
        const float s = m < M ? as[size_t(kb) * M + m] * wsc : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[p][i][j] = fmaf(part[p][i][j], s, acc[p][i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 4 * ty + i;
    if constexpr (!GATED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 32 * j;
        if (m < M && n < N) y[size_t(m) * N + n] = T(acc[0][i][j]);
      }
    } else {
      float z[4], mx = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[j] = __fdiv_rn(acc[0][i][j], 1.0f + expf(-acc[0][i][j])) * acc[1][i][j];
        mx = max_nan(mx, fabsf(z[j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = block_amax(mx);
      const Quotient quo(mx);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 32 * j;
        if (m < M && n < N) q[size_t(m) * N + n] = uint8_t(cvt_e4m3x2(quo(make_float2(z[j], 0.f))) & 0xFF);
      }
      if (m < M && tx == 0) qs[size_t(nb) * M + m] = block_scale(mx);
    }
  }
}

// ------------------------------------------------------------------ host
static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

static int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K <= 0) return QUAROT_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if (K % 16 != 0 || K > (int64_t(1) << 20) || M > lim || N > lim) return QUAROT_ERR_UNSUPPORTED;
  return QUAROT_OK;
}

}  // namespace gemm
}  // namespace fp8
}  // namespace quarot

using namespace quarot;

extern "C" int quarot_fp8_gemm(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q, const float* w_scale,
                               int64_t M, int64_t N, int64_t K, void* y, int dtype, void* stream) {
  using namespace quarot::fp8;
  using namespace quarot::fp8::gemm;
  if (dtype != QUAROT_FP16 && dtype != QUAROT_BF16) return QUAROT_ERR_INVALID_ARG;
  const int e = check_sizes(M, N, K);
  if (e != QUAROT_OK || M == 0 || N == 0) return e;
  if (!a_q || !a_scale || !w_q || !w_scale || !y) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(a_q, 16) || misaligned(w_q, 16) || misaligned(y, 16) || misaligned(a_scale, 4) || misaligned(w_scale, 4))
    return QUAROT_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned((M + TM - 1) / TM * ((N + TN - 1) / TN));
  if (dtype == QUAROT_FP16)
    fp8_gemm_kernel<false, __half><<<grid, 256, 0, st>>>(a_q, a_scale, w_q, w_scale, nullptr, nullptr, int(M), int(N),
                                                         int(K), static_cast<__half*>(y), nullptr, nullptr);
  else
    fp8_gemm_kernel<false, __nv_bfloat16><<<grid, 256, 0, st>>>(a_q, a_scale, w_q, w_scale, nullptr, nullptr, int(M),
                                                                int(N), int(K), static_cast<__nv_bfloat16*>(y), nullptr,
                                                                nullptr);
  return cudaGetLastError() == cudaSuccess ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}

extern "C" int quarot_fp8_gated_gemm(const uint8_t* a_q, const float* a_scale, const uint8_t* wg_q,
                                     const float* wg_scale, const uint8_t* wu_q, const float* wu_scale, int64_t M,
                                     int64_t I, int64_t K, uint8_t* q_out, float* scale_out, void* stream) {
  using namespace quarot::fp8;
  using namespace quarot::fp8::gemm;
  const int e = check_sizes(M, I, K);
  if (e != QUAROT_OK) return e;
  if (I % 16 != 0) return QUAROT_ERR_UNSUPPORTED;
  if (M == 0 || I == 0) return QUAROT_OK;
  if (!a_q || !a_scale || !wg_q || !wg_scale || !wu_q || !wu_scale || !q_out || !scale_out) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(a_q, 16) || misaligned(wg_q, 16) || misaligned(wu_q, 16) || misaligned(q_out, 16) ||
      misaligned(a_scale, 4) || misaligned(wg_scale, 4) || misaligned(wu_scale, 4) || misaligned(scale_out, 4))
    return QUAROT_ERR_ALIGNMENT;
  const unsigned grid = unsigned((M + TM - 1) / TM * ((I + TN - 1) / TN));
  fp8_gemm_kernel<true, __half><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      a_q, a_scale, wg_q, wg_scale, wu_q, wu_scale, int(M), int(I), int(K), nullptr, q_out, scale_out);
  return cudaGetLastError() == cudaSuccess ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}
