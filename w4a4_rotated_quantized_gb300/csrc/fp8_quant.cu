// The 8-bit quantizers: quarot_quant_fp8 (tokens, one scale for each token and
// 128 columns), quarot_quant_fp8_block (weights, one scale for each 128 x 128
// block) and quarot_add_rmsnorm_quant_fp8 (residual addition, RMSNorm and the
// token quantizer in one pass).
//
// [S] Stage 2b (symmetric abs-max quantization of the tokens, online) and
// Stage 1a (RMSNorm before the quantized projections); [G] "Online Activation
// Rotation Fused into RMSNorm".  The 8-bit form serves the layers that stay
// above 4 bits.
#include "fp8.cuh"

namespace quarot {
namespace fp8 {

// Eight columns of a row: 16 bytes of input, 8 codes.
template <typename T>
struct Chunk {
  float2 v[4];
  __device__ __forceinline__ explicit Chunk(uint4 r) {
    v[0] = to_f2<T>(r.x);
    v[1] = to_f2<T>(r.y);
    v[2] = to_f2<T>(r.z);
    v[3] = to_f2<T>(r.w);
  }
  __device__ __forceinline__ float amax() const {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max_nan(fabsf(v[i].x), fabsf(v[i].y));
    return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
  }
  __device__ __forceinline__ uint2 codes(const Quotient& q) const {
    return make_uint2(cvt_e4m3x4(q(v[0]), q(v[1])), cvt_e4m3x4(q(v[2]), q(v[3])));
  }
};

// Abs-max of 16-bit pairs, as they are (a NaN wins); exact, so the same as in fp32.
template <typename T>
struct Pair;
template <>
struct Pair<__half> {
  using V = __half2;
  static __device__ __forceinline__ V abs_max(V a, V b) { return __hmax2_nan(__habs2(a), __habs2(b)); }
  static __device__ __forceinline__ float2 value(V a) { return __half22float2(a); }
};
template <>
struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static __device__ __forceinline__ V abs_max(V a, V b) { return __hmax2_nan(__habs2(a), __habs2(b)); }
  static __device__ __forceinline__ float2 value(V a) { return __bfloat1622float2(a); }
};
template <typename T, int N>
__device__ __forceinline__ float raw_amax(const uint4 (&r)[N]) {
  using P = Pair<T>;
  typename P::V m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const typename P::V* v = reinterpret_cast<const typename P::V*>(&r[i]);
    m[i] = P::abs_max(P::abs_max(v[0], v[1]), P::abs_max(v[2], v[3]));
  }
#pragma unroll
  for (int i = 1; i < N; ++i) m[0] = P::abs_max(m[0], m[i]);
  const float2 f = P::value(m[0]);
  return max_nan(f.x, f.y);
}

// Maximum over the 16 lanes (one block of 128 columns) of a half warp.
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// ------------------------------------------------------------------ tokens
// Eight lanes own a block, 16 columns each (two 16-byte loads, one 16-byte
// store); a lane group takes U blocks, all loaded before the first is
// quantized.  Blocks are numbered along the rows, so a warp reads 1 KB without
// a gap.  Bound by HBM, 3 B an element: 8192 x 12288 46.6 us (6.5 TB/s, 95 % of a
// copy; 48.7 with the registers that the compiler would take, 49.7 with those and
// 256 threads, then 55.4 with one block to a lane group and 56.8 with four),
// 2048 x 12288 bf16 13.5 us (5.6 TB/s), of which a launch and a first load are 1.4.
constexpr int QT = 128, QU = 2, QG = QT / 8;

template <typename T>
__global__ void __launch_bounds__(QT, 10) quant_tokens_kernel(const T* __restrict__ x, uint32_t M, uint32_t d, int64_t ld,
                                                          uint32_t nb, uint32_t total, uint8_t* __restrict__ q,
                                                          float* __restrict__ scale) {
  const uint32_t l = threadIdx.x & 7u, g = threadIdx.x >> 3;
  uint4 raw[QU][2];
  uint32_t row[QU], col[QU];
  bool in[QU];
  next_may_start();
  wait_for_previous();
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    const uint32_t i = (blockIdx.x * QU + u) * QG + g;
    row[u] = i / nb;
    col[u] = (i - row[u] * nb) * BLK + l * 16;
    in[u] = i < total && col[u] < d;
    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
    if (in[u]) {
      const uint4* src = reinterpret_cast<const uint4*>(x + int64_t(row[u]) * ld + col[u]);
      raw[u][0] = __ldg(src);
      raw[u][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    float m = raw_amax<T>(raw[u]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = block_amax(m);
    const Quotient quo(m);
    const uint2 a = Chunk<T>(raw[u][0]).codes(quo), b = Chunk<T>(raw[u][1]).codes(quo);
    if (in[u]) {
      *reinterpret_cast<uint4*>(q + size_t(row[u]) * d + col[u]) = make_uint4(a.x, a.y, b.x, b.y);
      if (l == 0) scale[size_t(col[u] / BLK) * M + row[u]] = block_scale(m);
    }
  }
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 block, held in registers (8 chunks a thread): one read.
// Bound by HBM, 3 B an element: 12288 x 4096 25.4 us (5.9 TB/s, 88 % of a copy;
// 26.1 with three CTAs on an SM instead of four), 4096 x 4096 10.8 us (4.7 TB/s).
template <typename T>
__global__ void __launch_bounds__(256, 4) quant_block_kernel(const T* __restrict__ x, uint32_t N, uint32_t d, int64_t ld,
                                                          uint32_t nb, uint8_t* __restrict__ q,
                                                          float* __restrict__ scale) {
  __shared__ float wmax[8];
  const uint32_t c0 = (blockIdx.x % nb) * BLK + (threadIdx.x & 15u) * 8u;
  const uint32_t r0 = (blockIdx.x / nb) * BLK + (threadIdx.x >> 4);
  uint4 raw[8];
  next_may_start();
  wait_for_previous();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (c0 < d && r0 + 16 * i < N) raw[i] = __ldg(reinterpret_cast<const uint4*>(x + int64_t(r0 + 16 * i) * ld + c0));
  }
  float m = raw_amax<T>(raw);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, wmax[i]);
  m = block_amax(m);
  const Quotient quo(m);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 < d && r0 + 16 * i < N) *reinterpret_cast<uint2*>(q + size_t(r0 + 16 * i) * d + c0) = Chunk<T>(raw[i]).codes(quo);
  if (threadIdx.x == 0) scale[blockIdx.x] = block_scale(m);
}

// ------------------------------------------------------------------ residual + norm
// One CTA per row.  With h = rnd(x + residual) and r = sqrt(mean h^2 + eps),
// the codes of h w / r do not depend on r, a factor that all blocks of the row
// share: every block is quantized as soon as it is read, and r enters the
// scales (amax(h w) / 448 / r) at the end of the row.  So a row of any length
// is read once and nothing of it is kept but its blocks' abs-max.  Traffic: 2
// + 2 B read, 2 + 1 B written for each element.
//
// A thread has NU chunks in flight.  8192 x 12288 fp16: 103.5 us, 6.8 TB/s, as
// fast as a copy; 8192 x 4096: 36.9 us, 6.4 TB/s; 509 x 12288: 9.6 us, one
// wave of CTAs that waits for its loads six chunks a thread; 1 x 4096: 2.1 us,
// the latency of one row.
template <typename T, bool RES, bool WGT, int NU>
__global__ void norm_quant_kernel(const T* x, int64_t ld_x, const T* res, int64_t ld_r,
                                  const T* __restrict__ w, uint32_t M, uint32_t d, uint32_t nb, float eps, T* h_out,
                                  int64_t ld_h, uint8_t* __restrict__ q, float* __restrict__ scale) {
  extern __shared__ float amax_s[];  // [nb]
  __shared__ float part[32];
  const uint32_t row = blockIdx.x;
  const T* xr = x + int64_t(row) * ld_x;
  const T* rr = RES ? res + int64_t(row) * ld_r : nullptr;
  T* hr = h_out != nullptr ? h_out + int64_t(row) * ld_h : nullptr;
  uint8_t* qr = q + size_t(row) * d;
  const uint32_t step = blockDim.x * 8u;
  float2 ss = make_float2(0.f, 0.f);
  next_may_start();
  wait_for_previous();
  for (uint32_t base = 0; base < nb * BLK; base += NU * step) {
    uint4 a[NU], b[NU], g[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint32_t c = base + u * step + threadIdx.x * 8u;
      a[u] = b[u] = g[u] = make_uint4(0, 0, 0, 0);
      if (c < d) {
        a[u] = *reinterpret_cast<const uint4*>(xr + c);
        if constexpr (RES) b[u] = *reinterpret_cast<const uint4*>(rr + c);
        if constexpr (WGT) g[u] = __ldg(reinterpret_cast<const uint4*>(w + c));
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint32_t c = base + u * step + threadIdx.x * 8u;
      if (base + u * step >= nb * BLK) break;
      uint32_t hw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
      if constexpr (RES) {
        const uint32_t rw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) hw[i] = from_f2<T>(__fadd2_rn(to_f2<T>(hw[i]), to_f2<T>(rw[i])));
      }
      const uint4 h4 = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      if (c < d && hr != nullptr) *reinterpret_cast<uint4*>(hr + c) = h4;
      Chunk<T> v(h4);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __ffma2_rn(v.v[i], v.v[i], ss);
      if constexpr (WGT) {
        const Chunk<T> gv(g[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = __fmul2_rn(v.v[i], gv.v[i]);
      }
      const float m = block_amax(half_warp_max(v.amax()));
      if (c < d) {
        *reinterpret_cast<uint2*>(qr + c) = v.codes(Quotient(m));
        if ((threadIdx.x & 15u) == 0) amax_s[c / BLK] = m;
      }
    }
  }
  float s = ss.x + ss.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (uint32_t i = 0; i < (blockDim.x >> 5); ++i) s += part[i];
  const float rms = __fsqrt_rn(__fadd_rn(__fdiv_rn(s, float(d)), eps));
  for (uint32_t b = threadIdx.x; b < nb; b += blockDim.x)
    scale[size_t(b) * M + row] = __fdiv_rn(block_scale(amax_s[b]), rms);
}

// ------------------------------------------------------------------ host
static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxWidth = int64_t(1) << 20;

static int check_matrix(const void* x, int dtype, int64_t M, int64_t d, int64_t ld, const void* q, const void* s) {
  if (M < 0 || d <= 0 || ld < d || (dtype != QUAROT_FP16 && dtype != QUAROT_BF16)) return QUAROT_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > kMaxWidth || M > (int64_t(1) << 31) - BLK || M * ((d + BLK - 1) / BLK) >= (int64_t(1) << 31))
    return QUAROT_ERR_UNSUPPORTED;
  if (ld % 8 != 0) return QUAROT_ERR_ALIGNMENT;
  if (M == 0) return QUAROT_OK;
  if (!x || !q || !s) return QUAROT_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return QUAROT_ERR_ALIGNMENT;
  return QUAROT_OK;
}

template <typename T>
static int launch_norm(const void* x, int64_t ld_x, const void* res, int64_t ld_r, const void* w, int64_t M,
                        int64_t d, float eps, void* h, int64_t ld_h, uint8_t* q, float* scale, cudaStream_t st) {
  const uint32_t nb = uint32_t((d + BLK - 1) / BLK);
  const int64_t chunks = int64_t(nb) * (BLK / 8);
  // Few rows: as many threads as 256 to a row, its latency counts (600 x 4096: 5.3 us,
  // 6.7 with 128).  Many: smaller CTAs, more of them, as rows end at different
  // times (8192 x 4096: 36.9 us with 128 threads, 41.6 with 256; 8192 x 1024: 12.1
  // with 64, 14.5 with 128).  Long rows: 256 threads with three chunks in flight, at
  // any number of rows (8192 x 12288: 103.5 us, with two 109.2, with two and 128
  // threads 105.9; 509 x 12288: 9.6, 9.8, 14.4).
  const bool is_long = chunks > 1024;
  const int64_t most = is_long || M < 1024 ? 256 : chunks > 256 ? 128 : 64;
  const unsigned threads = unsigned(chunks < most ? (chunks + 31) / 32 * 32 : most);
  const size_t smem = nb * sizeof(float);
  auto go = [&](auto kern) {
    return launch_dependent(kern, dim3(unsigned(M)), threads, smem, 1, st, static_cast<const T*>(x), ld_x,
                            static_cast<const T*>(res), ld_r, static_cast<const T*>(w), M, d, nb, eps,
                            static_cast<T*>(h), ld_h, q, scale);
  };
  if (is_long) {
    if (res && w) return go(norm_quant_kernel<T, true, true, 3>);
    if (res) return go(norm_quant_kernel<T, true, false, 3>);
    if (w) return go(norm_quant_kernel<T, false, true, 3>);
    return go(norm_quant_kernel<T, false, false, 3>);
  }
  if (res && w) return go(norm_quant_kernel<T, true, true, 2>);
  if (res) return go(norm_quant_kernel<T, true, false, 2>);
  if (w) return go(norm_quant_kernel<T, false, true, 2>);
  return go(norm_quant_kernel<T, false, false, 2>);
}

}  // namespace fp8
}  // namespace quarot

using namespace quarot;

extern "C" int quarot_quant_fp8(const void* x, int dtype, int64_t M, int64_t d, int64_t ld_x, uint8_t* q_out,
                                float* scale_out, void* stream) {
  using namespace quarot::fp8;
  const int e = check_matrix(x, dtype, M, d, ld_x, q_out, scale_out);
  if (e != QUAROT_OK || M == 0) return e;
  const uint32_t nb = uint32_t((d + BLK - 1) / BLK), total = uint32_t(M) * nb;
  const unsigned grid = (total + QU * QG - 1) / (QU * QG);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == QUAROT_FP16)
    return launch_dependent(quant_tokens_kernel<__half>, dim3(grid), QT, 0, 1, st, static_cast<const __half*>(x), M, d,
                            ld_x, nb, total, q_out, scale_out);
  return launch_dependent(quant_tokens_kernel<__nv_bfloat16>, dim3(grid), QT, 0, 1, st,
                          static_cast<const __nv_bfloat16*>(x), M, d, ld_x, nb, total, q_out, scale_out);
}

extern "C" int quarot_quant_fp8_block(const void* w, int dtype, int64_t N, int64_t K, int64_t ld_w, uint8_t* q_out,
                                      float* scale_out, void* stream) {
  using namespace quarot::fp8;
  const int e = check_matrix(w, dtype, N, K, ld_w, q_out, scale_out);
  if (e != QUAROT_OK || N == 0) return e;
  const uint32_t nb = uint32_t((K + BLK - 1) / BLK);
  const unsigned grid = unsigned((N + BLK - 1) / BLK) * nb;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == QUAROT_FP16)
    return launch_dependent(quant_block_kernel<__half>, dim3(grid), 256, 0, 1, st, static_cast<const __half*>(w), N, K,
                            ld_w, nb, q_out, scale_out);
  return launch_dependent(quant_block_kernel<__nv_bfloat16>, dim3(grid), 256, 0, 1, st,
                          static_cast<const __nv_bfloat16*>(w), N, K, ld_w, nb, q_out, scale_out);
}

extern "C" int quarot_add_rmsnorm_quant_fp8(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                                            const void* weight, int dtype, int64_t M, int64_t d, float eps,
                                            void* residual_out, int64_t ld_out, uint8_t* q_out, float* scale_out,
                                            void* stream) {
  using namespace quarot::fp8;
  if (!(eps > 0.f) || !(eps < INFINITY)) return QUAROT_ERR_INVALID_ARG;
  const int e = check_matrix(x, dtype, M, d, ld_x, q_out, scale_out);
  if (e != QUAROT_OK) return e;
  if ((residual && ld_r < d) || (residual_out && ld_out < d)) return QUAROT_ERR_INVALID_ARG;
  if ((residual && ld_r % 8 != 0) || (residual_out && ld_out % 8 != 0)) return QUAROT_ERR_ALIGNMENT;
  if (M == 0) return QUAROT_OK;
  if (!aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16)) return QUAROT_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == QUAROT_FP16)
    return launch_norm<__half>(x, ld_x, residual, ld_r, weight, M, d, eps, residual_out, ld_out, q_out, scale_out, st);
  return launch_norm<__nv_bfloat16>(x, ld_x, residual, ld_r, weight, M, d, eps, residual_out, ld_out, q_out, scale_out, st);
}
