// quarot_paged_attn: attention over the paged INT4 cache.
//
// For new token i at position p of sequence b, and query head h of group
// g = h / (Hq / Hkv):
//   q~ = q H_d / sqrt(d),  s_t = sm_scale * q~ . (k_s[t] kcode_t)  for t <= p
//   out = sum_t softmax(s)_t v_s[t] vcode_t
#include "paged.cuh"

namespace quarot {
namespace paged {

constexpr int SW = 4;  // warps

// One CTA per (token, query head); each warp takes every fourth cached token
// with an online softmax of its own, lanes share a head's dims.
template <typename T, int D>
__global__ void __launch_bounds__(32 * SW)
attn_kernel(const T* __restrict__ q, int64_t ld_q, int Hq, int Hkv, const uint8_t* __restrict__ k_q,
            const __half* __restrict__ k_s, const uint8_t* __restrict__ v_q, const __half* __restrict__ v_s, Batch t,
            int shared_len, float qscale, int unrotate, T* __restrict__ out, int64_t ld_out) {
  constexpr int E = D / 32;
  __shared__ float qs[D], os[SW][D], ms[SW], ls[SW];
  const int n = blockIdx.x / Hq, h = blockIdx.x % Hq, g = h / (Hq / Hkv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place p = place_of(t, n);
  if (p.b < 0) return;
  const int len = p.pos + 1;
  auto hadamard = [&](float* x) {
    for (int span = 1; span < D; span <<= 1) {
      float y = 0.f;
      const int e = threadIdx.x;
      if (e < D) y = (e & span) ? x[e ^ span] - x[e] : x[e] + x[e ^ span];
      __syncthreads();
      if (e < D) x[e] = y;
      __syncthreads();
    }
  };
  if (threadIdx.x < D) {
    const T v = q[n * ld_q + int64_t(h) * D + threadIdx.x];
    qs[threadIdx.x] = float(v);
  }
  __syncthreads();
  hadamard(qs);
  float x[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    x[i] = qs[lane * E + i] * qscale;
    o[i] = 0.f;
  }
  for (int tok = warp; tok < len; tok += SW) {
    const int page = page_at(t, tok < shared_len ? 0 : p.b, tok / t.ps);
    if (page < 0) continue;
    const int64_t at = (int64_t(page) * Hkv + g) * t.ps + tok % t.ps;
    float s = 0.f;
    for (int i = 0; i < E; i += 2) {
      const uint8_t c = k_q[at * (D / 2) + (lane * E + i) / 2];
      s += x[i] * float(int(c << 28) >> 28) + x[i + 1] * float(int(c << 24) >> 28);
    }
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= __half2float(k_s[at]);
    const float mn = fmaxf(m, s), a = exp2f(m - mn), e = exp2f(s - mn);
    const float w = e * __half2float(v_s[at]);
    m = mn;
    l = l * a + e;
    for (int i = 0; i < E; i += 2) {
      const uint8_t c = v_q[at * (D / 2) + (lane * E + i) / 2];
      o[i] = o[i] * a + w * float(int(c << 28) >> 28);
      o[i + 1] = o[i + 1] * a + w * float(int(c << 24) >> 28);
    }
  }
  for (int i = 0; i < E; ++i) os[warp][lane * E + i] = o[i];
  if (lane == 0) {
    ms[warp] = m;
    ls[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float mm = -INFINITY, num = 0.f, den = 0.f;
    for (int w = 0; w < SW; ++w) mm = fmaxf(mm, ms[w]);
    for (int w = 0; w < SW; ++w) {
      const float f = mm == -INFINITY ? 0.f : exp2f(ms[w] - mm);
      num += f * os[w][threadIdx.x];
      den += f * ls[w];
    }
    qs[threadIdx.x] = den > 0.f ? num / den : 0.f;
  }
  __syncthreads();
  if (unrotate) hadamard(qs);
  if (threadIdx.x < D)
    out[n * ld_out + int64_t(h) * D + threadIdx.x] = T(qs[threadIdx.x] * (unrotate ? 1.0f / sqrtf(float(D)) : 1.0f));
}

}  // namespace paged
}  // namespace quarot

using namespace quarot;
using namespace quarot::paged;

extern "C" size_t quarot_paged_workspace_bytes(int64_t N, int64_t B, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_q,
                                               int64_t shared_len) {
  if (N <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128) || max_q <= 0 ||
      shared_len < 0)
    return 0;
  return 256;
}

extern "C" int quarot_paged_attn(const void* q, int64_t ld_q, int dtype, int64_t N, int64_t Hq, int64_t Hkv, int64_t d,
                                 const uint8_t* k_q, const void* k_s, const uint8_t* v_q, const void* v_s, int64_t n_pages,
                                 int64_t page_size, const int32_t* page_table, int64_t B, int64_t max_pages,
                                 const int32_t* lengths, const int32_t* cu_q, int64_t max_q, int64_t shared_len,
                                 float sm_scale, int unrotate_out, void* out, int64_t ld_out, void* workspace,
                                 size_t ws_bytes, void* stream) {
  int rc = check_sizes(dtype, N, Hkv, d, n_pages, page_size, B, max_pages, cu_q);
  if (rc != QUAROT_OK) return rc;
  if (Hq <= 0 || Hq % Hkv != 0 || max_q <= 0 || shared_len < 0 || shared_len > max_pages * page_size ||
      (unrotate_out != 0 && unrotate_out != 1) || isnan(sm_scale) || isinf(sm_scale))
    return QUAROT_ERR_INVALID_ARG;
  if (Hq > kMaxHeads) return QUAROT_ERR_UNSUPPORTED;
  if (N == 0 || B == 0) return QUAROT_OK;
  if ((rc = check_heads(q, ld_q, Hq, d)) != QUAROT_OK || (rc = check_heads(out, ld_out, Hq, d)) != QUAROT_OK) return rc;
  if ((rc = check_cache(k_q, k_s, v_q, v_s, page_table, lengths, cu_q, max_pages)) != QUAROT_OK) return rc;
  if (!workspace || ws_bytes < quarot_paged_workspace_bytes(N, B, Hq, Hkv, d, max_q, shared_len)) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(workspace, 256)) return QUAROT_ERR_ALIGNMENT;
  const Batch t = {page_table, lengths, cu_q, int(B), int(max_pages), int(n_pages), int(page_size)};
  const float qscale = (sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(float(d))) * 1.4426950408889634f / sqrtf(float(d));
  auto go = [&](auto kern, auto* qp, auto* op) {
    kern<<<unsigned(N * Hq), 32 * SW, 0, static_cast<cudaStream_t>(stream)>>>(
        qp, ld_q, int(Hq), int(Hkv), k_q, static_cast<const __half*>(k_s), v_q, static_cast<const __half*>(v_s), t,
        int(shared_len), qscale, unrotate_out, op, ld_out);
  };
  if (dtype == QUAROT_FP16) {
    auto* qp = static_cast<const __half*>(q);
    auto* op = static_cast<__half*>(out);
    d == 64 ? go(attn_kernel<__half, 64>, qp, op) : go(attn_kernel<__half, 128>, qp, op);
  } else {
    auto* qp = static_cast<const __nv_bfloat16*>(q);
    auto* op = static_cast<__nv_bfloat16*>(out);
    d == 64 ? go(attn_kernel<__nv_bfloat16, 64>, qp, op) : go(attn_kernel<__nv_bfloat16, 128>, qp, op);
  }
  return cuda_ok(cudaGetLastError()) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}
