// Rotary positions and the paged INT4 cache's writing and reading:
// quarot_rope, quarot_paged_append, quarot_paged_read.
//
// The cache holds what quarot_kv_write stores (the head-wise rotation of
// [S] Stages 1c and 1d, the symmetric quantizer of Stage 2c's procedure), in
// pages: codes [n_pages, Hkv, page_size, d / 2], scales [n_pages, Hkv,
// page_size].  Token p of sequence b is slot p % page_size of page
// table[b][p / page_size].
#include "paged.cuh"

namespace quarot {
namespace paged {

// ------------------------------------------------------------------ rotary positions
// A head is d / 16 units of 16 elements: 8 pairs that are turned (elements
// 16 u .. 16 u + 15 of interleaved pairs, 8 u .. 8 u + 7 with their partners
// rot / 2 further of the half layout), or 16 elements that stay.  A thread owns
// a unit of every HSth head of a token: it makes the 8 angles once for them.
struct Heads {
  const void* in;
  void* out;
  int64_t ld_in, ld_out;
  int H;
};

template <typename T>
__device__ __forceinline__ void rope_unit(const T* src, T* dst, int u, int rot, bool inter, const float2* cs) {
  const int units = rot >> 4;
  int e0, e1;
  if (u >= units || inter) {
    e0 = 16 * u;
    e1 = e0 + 8;
  } else {
    e0 = 8 * u;
    e1 = e0 + (rot >> 1);
  }
  uint4 r0 = *reinterpret_cast<const uint4*>(src + e0), r1 = *reinterpret_cast<const uint4*>(src + e1);
  if (u < units) {
    float a[8], b[8];
    unpack8<T>(r0, a);
    unpack8<T>(r1, b);
    if (inter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        turn(a[2 * i], a[2 * i + 1], cs[i]);
        turn(b[2 * i], b[2 * i + 1], cs[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(a[i], b[i], cs[i]);
    }
    r0 = pack8<T>(a);
    r1 = pack8<T>(b);
  }
  *reinterpret_cast<uint4*>(dst + e0) = r0;
  *reinterpret_cast<uint4*>(dst + e1) = r1;
}

template <typename T>
__global__ void __launch_bounds__(256)
rope_kernel(Heads q, Heads k, int64_t N, int d, const int32_t* __restrict__ positions,
            const double* __restrict__ inv_freq, int rot, int inter, float scale, int HS) {
  const int U = d >> 4;
  const int64_t gt = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int lane_unit = int(gt % U);
  const int64_t slot = gt / U;  // (token, first head)
  const int64_t n = slot / HS;
  if (n >= N) return;
  float2 cs[8];
  if (16 * lane_unit < rot) {
    const int pos = positions[n];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = turn_of(pos, turn_step(inv_freq[8 * lane_unit + i]), scale);
  }
  for (int h = int(slot % HS); h < q.H + k.H; h += HS) {
    const bool isq = h < q.H;
    const Heads& x = isq ? q : k;
    const int hh = isq ? h : h - q.H;
    rope_unit<T>(static_cast<const T*>(x.in) + n * x.ld_in + int64_t(hh) * d,
                 static_cast<T*>(x.out) + n * x.ld_out + int64_t(hh) * d, lane_unit, rot, inter != 0, cs);
  }
}

// ------------------------------------------------------------------ append
// As in quarot_kv_write, d / 32 lanes own one (token, head) vector, 32
// elements each.  A CTA takes 64 (d = 128) or 128 neighbouring vectors of the
// keys, the values or the queries, heads fastest, so that the angles of its
// few tokens are made once, in shared memory.
constexpr int AT = 256;       // threads
constexpr int ATOK = 64;      // most tokens of a CTA
constexpr int AHALF = 64;     // most pairs of a head

template <typename T, int D>
__global__ void __launch_bounds__(AT)
append_kernel(Heads k, Heads v, Heads q, int64_t N, const double* __restrict__ inv_freq, int rot, int inter, float scale,
              uint8_t* __restrict__ k_q, __half* __restrict__ k_s, uint8_t* __restrict__ v_q, __half* __restrict__ v_s,
              Batch t, int blocks_kv) {
  constexpr int TPV = D / 32;
  __shared__ float2 cs[ATOK][AHALF];
  __shared__ uint64_t step[AHALF];
  __shared__ int row[ATOK], posn[ATOK];
  const int which = int(blockIdx.x) < blocks_kv ? 0 : int(blockIdx.x) < 2 * blocks_kv ? 1 : 2;
  const Heads x = which == 0 ? k : which == 1 ? v : q;
  const int64_t blk = int64_t(blockIdx.x) - which * int64_t(blocks_kv);
  // tokens [n0, n0 + nt): whole tokens, as many as fit
  const int per = AT / TPV;                              // vectors at a time
  const int nt_max = min(ATOK, max(1, per / x.H));
  const int64_t n0 = blk * nt_max;
  const int nt = int(min(int64_t(nt_max), N - n0));
  const bool turned = which != 1 && rot > 0;
  const int half = rot >> 1;
  if (int(threadIdx.x) < nt) {
    const Place p = place_of(t, int(n0) + threadIdx.x);
    int r = -2;  // nothing to store, and nothing wrong
    if (p.b >= 0 && p.pos >= 0) {
      const int page = page_at(t, p.b, p.pos / t.ps);
      r = page < 0 ? -1 : p.pos % t.ps;
      posn[threadIdx.x] = p.pos;
      row[threadIdx.x] = page < 0 ? -1 : page;
    } else {
      posn[threadIdx.x] = p.b < 0 ? -2 : -1;
      row[threadIdx.x] = r;
    }
  }
  if (turned && int(threadIdx.x) < half) step[threadIdx.x] = turn_step(inv_freq[threadIdx.x]);
  __syncthreads();
  if (turned) {
    for (int i = threadIdx.x; i < nt * half; i += AT) cs[i / half][i % half] = turn_of(posn[i / half], step[i % half], scale);
    __syncthreads();
  }
  const int total = nt * x.H;
  for (int base = 0; base < total; base += per) {
    const int vi = base + int(threadIdx.x) / TPV, part = int(threadIdx.x) % TPV;
    const bool valid = vi < total;
    const int ti = valid ? vi / x.H : 0, h = valid ? vi % x.H : 0;
    const T* src = static_cast<const T*>(x.in) + (n0 + ti) * x.ld_in + int64_t(h) * D;
    float e[32];
    if (valid) {
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack8<T>(*reinterpret_cast<const uint4*>(src + 32 * part + 8 * i), e + 8 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) e[i] = 0.f;
    }
    if (turned && valid) {
      if (inter) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * part + 2 * i < rot) turn(e[2 * i], e[2 * i + 1], cs[ti][16 * part + i]);
      } else {
        // the partners of 8 elements are 8 neighbouring ones, all on one side
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e0 = 32 * part + 8 * i;
          if (e0 < rot) {
            const bool low = e0 < half;
            const int f = low ? e0 : e0 - half;
            float o[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(src + (low ? e0 + half : f)), o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 c = cs[ti][f + j];
              e[8 * i + j] = low ? e[8 * i + j] * c.x - o[j] * c.y : e[8 * i + j] * c.x + o[j] * c.y;
            }
          }
        }
      }
    }
    if (which == 2) {
      __syncwarp();  // q_out may be q: partners are read before they are written
      if (valid && posn[ti] != -2) {
        T* dst = static_cast<T*>(x.out) + (n0 + ti) * x.ld_out + int64_t(h) * D;
        const bool none = posn[ti] < 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(dst + 32 * part + 8 * i) = none ? make_uint4(0u, 0u, 0u, 0u) : pack8<T>(e + 8 * i);
      }
      continue;
    }
    hadamard32<TPV>(e, part);
    const float inv_sqrt_d = 1.0f / sqrtf(float(D));
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      e[i] *= inv_sqrt_d;
      amax = fmaxf(amax, fabsf(e[i]));
    }
#pragma unroll
    for (int o = 1; o < TPV; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const __half S = quant_scale_fp16(amax, 1.0f);
    const float inv = 1.0f / __half2float(S);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i >> 3] |= nibble_rne(fminf(fmaxf(e[i] * inv, -8.0f), 7.0f)) << (4 * (i & 7));
    if (valid && row[ti] >= 0) {
      const int64_t at = (int64_t(row[ti]) * x.H + h) * t.ps + posn[ti] % t.ps;
      *reinterpret_cast<uint4*>((which == 0 ? k_q : v_q) + at * (D / 2) + part * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      if (part == 0) (which == 0 ? k_s : v_s)[at] = S;
    }
  }
}

// ------------------------------------------------------------------ read
// One (token, head) vector of the keys and of the values by d / 32 lanes each.
template <typename T, int D, bool BACK>
__global__ void __launch_bounds__(256)
read_kernel(const uint8_t* __restrict__ k_q, const __half* __restrict__ k_s, const uint8_t* __restrict__ v_q,
            const __half* __restrict__ v_s, int64_t N, int Hkv, Batch t, T* __restrict__ k_out, T* __restrict__ v_out) {
  constexpr int TPV = D / 32;
  const int64_t gt = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t vi = gt / TPV;
  const int part = int(gt % TPV);
  const bool valid = vi < N * Hkv;
  const int n = valid ? int(vi / Hkv) : 0, h = valid ? int(vi % Hkv) : 0;
  Place p = {-1, -1};
  if (valid) p = place_of(t, n);
  int page = -1;
  if (p.b >= 0 && p.pos >= 0) page = page_at(t, p.b, p.pos / t.ps);
  const int64_t at = page < 0 ? 0 : (int64_t(page) * Hkv + h) * t.ps + p.pos % t.ps;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    float s = 0.f;
    if (page >= 0) {
      r = *reinterpret_cast<const uint4*>((which ? v_q : k_q) + at * (D / 2) + part * 16);
      s = __half2float((which ? v_s : k_s)[at]);
    }
    float e[32];
    codes8(r.x, e);
    codes8(r.y, e + 8);
    codes8(r.z, e + 16);
    codes8(r.w, e + 24);
    if constexpr (BACK) {
      hadamard32<TPV>(e, part);  // sums of codes are whole numbers: exact
      s *= 1.0f / sqrtf(float(D));
    }
    if (p.b >= 0) {
      T* dst = (which ? v_out : k_out) + (int64_t(n) * Hkv + h) * D + 32 * part;
#pragma unroll
      for (int i = 0; i < 32; ++i) e[i] *= s;
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(dst + 8 * i) = pack8<T>(e + 8 * i);
    }
  }
}

}  // namespace paged
}  // namespace quarot

using namespace quarot;
using namespace quarot::paged;

extern "C" int quarot_rope(const void* q, int64_t Hq, int64_t ld_q, void* q_out, int64_t ld_qo, const void* k, int64_t Hk,
                           int64_t ld_k, void* k_out, int64_t ld_ko, int dtype, int64_t N, int64_t d,
                           const int32_t* positions, const double* inv_freq, int64_t rot, int interleaved, float scale,
                           void* stream) {
  if (dtype != QUAROT_FP16 && dtype != QUAROT_BF16) return QUAROT_ERR_INVALID_ARG;
  if (N < 0 || Hq <= 0 || Hk < 0 || d <= 0 || !isfinite(scale)) return QUAROT_ERR_INVALID_ARG;
  if (d % 16 != 0 || d > 1024 || N > kMaxTokens || Hq + Hk > 2 * kMaxHeads) return QUAROT_ERR_UNSUPPORTED;
  int rc = check_rotation(inv_freq, rot, d, interleaved);
  if (rc != QUAROT_OK) return rc;
  if (N == 0) return QUAROT_OK;
  if ((rc = check_heads(q, ld_q, Hq, d)) != QUAROT_OK || (rc = check_heads(q_out, ld_qo, Hq, d)) != QUAROT_OK) return rc;
  if (Hk > 0 && ((rc = check_heads(k, ld_k, Hk, d)) != QUAROT_OK || (rc = check_heads(k_out, ld_ko, Hk, d)) != QUAROT_OK))
    return rc;
  if (!positions) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(positions, 4)) return QUAROT_ERR_ALIGNMENT;
  int sms = 0;
  if (!sm_count(&sms)) return QUAROT_ERR_CUDA;
  const int U = int(d >> 4), H = int(Hq + Hk);
  const int HS = H;
  const int64_t threads = N * HS * U;
  const int64_t blocks = (threads + 255) / 256;
  const Heads hq = {q, q_out, ld_q, ld_qo, int(Hq)}, hk = {k, k_out, ld_k, ld_ko, int(Hk)};
  auto kern = dtype == QUAROT_FP16 ? rope_kernel<__half> : rope_kernel<__nv_bfloat16>;
  kern<<<unsigned(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(hq, hk, N, int(d), positions, inv_freq, int(rot),
                                                                       interleaved, scale, HS);
  return cuda_ok(cudaGetLastError()) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}

extern "C" int quarot_paged_append(const void* k, int64_t ld_k, const void* v, int64_t ld_v, const void* q, int64_t Hq,
                                   int64_t ld_q, void* q_out, int64_t ld_qo, int dtype, int64_t N, int64_t Hkv, int64_t d,
                                   const double* inv_freq, int64_t rot, int interleaved, float scale, uint8_t* k_q,
                                   void* k_s, uint8_t* v_q, void* v_s, int64_t n_pages, int64_t page_size,
                                   const int32_t* page_table, int64_t B, int64_t max_pages, const int32_t* lengths,
                                   const int32_t* cu_q, void* stream) {
  int rc = check_sizes(dtype, N, Hkv, d, n_pages, page_size, B, max_pages, cu_q);
  if (rc != QUAROT_OK) return rc;
  if (!isfinite(scale) || Hq < 0 || (Hq == 0 && q != nullptr)) return QUAROT_ERR_INVALID_ARG;
  if (Hq > kMaxHeads) return QUAROT_ERR_UNSUPPORTED;
  if ((rc = check_rotation(inv_freq, rot, d, interleaved)) != QUAROT_OK) return rc;
  if (N == 0 || B == 0) return QUAROT_OK;
  if ((rc = check_heads(k, ld_k, Hkv, d)) != QUAROT_OK || (rc = check_heads(v, ld_v, Hkv, d)) != QUAROT_OK) return rc;
  if (Hq > 0 && ((rc = check_heads(q, ld_q, Hq, d)) != QUAROT_OK || (rc = check_heads(q_out, ld_qo, Hq, d)) != QUAROT_OK))
    return rc;
  if ((rc = check_cache(k_q, k_s, v_q, v_s, page_table, lengths, cu_q, max_pages)) != QUAROT_OK) return rc;
  const Batch t = {page_table, lengths, cu_q, int(B), int(max_pages), int(n_pages), int(page_size)};
  const Heads hk = {k, nullptr, ld_k, 0, int(Hkv)}, hv = {v, nullptr, ld_v, 0, int(Hkv)}, hq = {q, q_out, ld_q, ld_qo, int(Hq)};
  const int64_t per = AT / (d / 32);
  auto blocks_of = [&](int64_t H) {
    int64_t nt = per / H;
    nt = nt < 1 ? 1 : nt > ATOK ? ATOK : nt;
    return (N + nt - 1) / nt;
  };
  const int64_t bkv = blocks_of(Hkv), bq = Hq > 0 ? blocks_of(Hq) : 0;
  auto go = [&](auto kern) {
    kern<<<unsigned(2 * bkv + bq), AT, 0, static_cast<cudaStream_t>(stream)>>>(
        hk, hv, hq, N, inv_freq, int(rot), interleaved, scale, k_q, static_cast<__half*>(k_s), v_q,
        static_cast<__half*>(v_s), t, int(bkv));
  };
  if (dtype == QUAROT_FP16) d == 64 ? go(append_kernel<__half, 64>) : go(append_kernel<__half, 128>);
  else d == 64 ? go(append_kernel<__nv_bfloat16, 64>) : go(append_kernel<__nv_bfloat16, 128>);
  return cuda_ok(cudaGetLastError()) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}

extern "C" int quarot_paged_read(const uint8_t* k_q, const void* k_s, const uint8_t* v_q, const void* v_s, int64_t n_pages,
                                 int64_t page_size, int64_t Hkv, int64_t d, const int32_t* page_table, int64_t B,
                                 int64_t max_pages, const int32_t* lengths, const int32_t* cu_q, int64_t N, int unrotate,
                                 void* k_out, void* v_out, int dtype, void* stream) {
  int rc = check_sizes(dtype, N, Hkv, d, n_pages, page_size, B, max_pages, cu_q);
  if (rc != QUAROT_OK) return rc;
  if (unrotate != 0 && unrotate != 1) return QUAROT_ERR_INVALID_ARG;
  if (N == 0 || B == 0) return QUAROT_OK;
  if ((rc = check_heads(k_out, Hkv * d, Hkv, d)) != QUAROT_OK || (rc = check_heads(v_out, Hkv * d, Hkv, d)) != QUAROT_OK)
    return rc;
  if ((rc = check_cache(k_q, k_s, v_q, v_s, page_table, lengths, cu_q, max_pages)) != QUAROT_OK) return rc;
  const Batch t = {page_table, lengths, cu_q, int(B), int(max_pages), int(n_pages), int(page_size)};
  const int64_t blocks = (N * Hkv * (d / 32) + 255) / 256;
  if (blocks > 0x7fffffff) return QUAROT_ERR_UNSUPPORTED;
  auto go = [&](auto kern, auto* ko, auto* vo) {
    kern<<<unsigned(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        k_q, static_cast<const __half*>(k_s), v_q, static_cast<const __half*>(v_s), N, int(Hkv), t, ko, vo);
  };
  auto typed = [&](auto* ko, auto* vo) {
    using T = std::remove_pointer_t<decltype(ko)>;
    if (d == 64) unrotate ? go(read_kernel<T, 64, true>, ko, vo) : go(read_kernel<T, 64, false>, ko, vo);
    else unrotate ? go(read_kernel<T, 128, true>, ko, vo) : go(read_kernel<T, 128, false>, ko, vo);
  };
  if (dtype == QUAROT_FP16) typed(static_cast<__half*>(k_out), static_cast<__half*>(v_out));
  else typed(static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out));
  return cuda_ok(cudaGetLastError()) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}
