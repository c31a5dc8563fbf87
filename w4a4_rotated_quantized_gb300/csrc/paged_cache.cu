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
// rot / 2 further of the half layout), or 16 elements that stay: either way two
// 16-byte loads and stores that no other unit touches, so the outputs may be
// the inputs.  A CTA makes the cosines and sines of its few tokens once, in
// shared memory, one or a few a thread; its threads then walk over the units of
// all their heads, three loaded ahead of the arithmetic.
struct Heads {
  const void* in;
  void* out;
  int64_t ld_in, ld_out;
  int H;
};
constexpr int RT = 256;  // threads

// Units of `nt` tokens from n0 on.  A thread has unit u = tid % U of every
// (RT / U * parts)-th head; cs [token][pair].  skip: for each token 0 to turn
// it, 1 to write zeros, 2 to leave its output.
template <typename T>
__device__ __forceinline__ void turn_heads(const Heads& x, int64_t n0, int nt, int d, int rot, bool inter, const float2* cs,
                                           const int* skip, int part, int parts) {
  constexpr int AHEAD = 3;
  const int U = d >> 4, u = int(threadIdx.x) % U, per = RT / U * parts;
  if (int(threadIdx.x) >= RT / U * U) return;
  const bool turned = 16 * u < rot;
  const int e0 = turned && !inter ? 8 * u : 16 * u, e1 = turned && !inter ? e0 + (rot >> 1) : e0 + 8;
  const float2* c = cs + 8 * u;
  const int half = rot >> 1;
  int v = int(threadIdx.x) / U + RT / U * part;  // (token, head)
  int ti = v / x.H, h = v - ti * x.H;
  while (ti < nt) {
    uint4 r[AHEAD][2];
    int tk[AHEAD], hk[AHEAD], cnt = 0;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      tk[i] = ti;
      hk[i] = h;
      if (ti < nt) {
        const T* src = static_cast<const T*>(x.in) + (n0 + ti) * x.ld_in + int64_t(h) * d;
        r[i][0] = *reinterpret_cast<const uint4*>(src + e0);
        r[i][1] = *reinterpret_cast<const uint4*>(src + e1);
        cnt = i + 1;
        h += per;
        if (h >= x.H) {
          const int k = h / x.H;
          ti += k;
          h -= k * x.H;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (i >= cnt) continue;
      const int what = skip == nullptr ? 0 : skip[tk[i]];
      if (what == 2) continue;
      if (turned) {
        float a[8], b[8];
        unpack8<T>(r[i][0], a);
        unpack8<T>(r[i][1], b);
        float2 t[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 f = *reinterpret_cast<const float4*>(c + tk[i] * half + 2 * k);
          t[2 * k] = make_float2(f.x, f.y);
          t[2 * k + 1] = make_float2(f.z, f.w);
        }
        if (inter) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            turn(a[2 * k], a[2 * k + 1], t[k]);
            turn(b[2 * k], b[2 * k + 1], t[4 + k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) turn(a[k], b[k], t[k]);
        }
        r[i][0] = pack8<T>(a);
        r[i][1] = pack8<T>(b);
      }
      if (what == 1) r[i][0] = r[i][1] = make_uint4(0u, 0u, 0u, 0u);
      T* dst = static_cast<T*>(x.out) + (n0 + tk[i]) * x.ld_out + int64_t(hk[i]) * d;
      *reinterpret_cast<uint4*>(dst + e0) = r[i][0];
      *reinterpret_cast<uint4*>(dst + e1) = r[i][1];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(RT)
rope_kernel(Heads q, Heads k, int64_t N, int d, const int32_t* __restrict__ positions,
            const double* __restrict__ inv_freq, int rot, int inter, float scale, int tokens) {
  extern __shared__ __align__(16) unsigned char rsm[];
  float2* cs = reinterpret_cast<float2*>(rsm);  // [tokens][half]
  const int half = rot >> 1;
  const int64_t n0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), N - n0));
  // a thread's pair is the same for every token that it makes an angle of, where half is a power of two
  for (int i = threadIdx.x; i < nt * half; i += RT)
    cs[i] = turn_of(positions[n0 + i / half], turn_step(inv_freq[i % half]), scale);
  __syncthreads();
  turn_heads<T>(q, n0, nt, d, rot, inter != 0, cs, nullptr, blockIdx.y, gridDim.y);
  if (k.H > 0) turn_heads<T>(k, n0, nt, d, rot, inter != 0, cs, nullptr, blockIdx.y, gridDim.y);
}

// ------------------------------------------------------------------ append
// As in quarot_kv_write, d / 32 lanes own one (token, head) vector, 32
// elements each.  A CTA takes some neighbouring tokens' keys, values or
// queries, so that places are looked up and angles made once for all heads.
constexpr int ATOK = 32;      // most tokens of a CTA
constexpr int AHALF = 64;     // most pairs of a head

template <typename T, int D>
__global__ void __launch_bounds__(RT)
append_kernel(Heads k, Heads v, Heads q, int64_t N, const double* __restrict__ inv_freq, int rot, int inter, float scale,
              uint8_t* __restrict__ k_q, __half* __restrict__ k_s, uint8_t* __restrict__ v_q, __half* __restrict__ v_s,
              Batch t, int kv_tokens, int kv_blocks, int q_tokens, int q_parts) {
  constexpr int TPV = D / 32;
  __shared__ __align__(16) float2 cs[ATOK * AHALF];
  __shared__ uint64_t step[AHALF];
  __shared__ int row[ATOK], posn[ATOK], skip[ATOK];
  // the queries' CTAs first: theirs is most of the memory's work
  const int which = int(blockIdx.x) >= int(gridDim.x) - kv_blocks ? 1 : int(blockIdx.x) >= int(gridDim.x) - 2 * kv_blocks ? 0 : 2;
  const Heads x = which == 0 ? k : which == 1 ? v : q;
  const int64_t blk = which == 2 ? blockIdx.x / q_parts : which == 0 ? blockIdx.x - (gridDim.x - 2 * kv_blocks) : blockIdx.x - (gridDim.x - kv_blocks);
  const int nt_max = which == 2 ? q_tokens : kv_tokens;
  const int64_t n0 = blk * nt_max;
  const int nt = int(min(int64_t(nt_max), N - n0));
  const int half = rot >> 1;
  const bool turned = which != 1 && half > 0;
  if (int(threadIdx.x) < nt) {
    const Place p = place_of(t, int(n0) + threadIdx.x);
    posn[threadIdx.x] = p.pos;
    skip[threadIdx.x] = p.b < 0 ? 2 : p.pos < 0 ? 1 : 0;
    if (which != 2) row[threadIdx.x] = p.b >= 0 && p.pos >= 0 ? page_at(t, p.b, p.pos / t.ps) : -1;
  }
  if (turned && int(threadIdx.x) < half) step[threadIdx.x] = turn_step(inv_freq[threadIdx.x]);
  __syncthreads();
  if (turned) {
    for (int i = threadIdx.x; i < nt * half; i += RT) cs[i] = turn_of(posn[i / half], step[i % half], scale);
    __syncthreads();
  }
  if (which == 2) {
    turn_heads<T>(x, n0, nt, D, rot, inter != 0, cs, skip, int(blockIdx.x) % q_parts, q_parts);
    return;
  }
  constexpr int per = RT / TPV;  // vectors at a time
  const int total = nt * x.H, part = int(threadIdx.x) % TPV;
  // The next vector's 64 bytes are loaded before this one is worked on.
  auto source = [&](int vi) {
    const int ti = vi / x.H;
    return static_cast<const T*>(x.in) + (n0 + ti) * x.ld_in + int64_t(vi - ti * x.H) * D;
  };
  const int first = int(threadIdx.x) / TPV;
  uint4 nx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    nx[i] = first < total ? __ldcs(reinterpret_cast<const uint4*>(source(first) + 32 * part) + i) : make_uint4(0u, 0u, 0u, 0u);
  for (int base = 0; base < total; base += per) {
    const int vi = base + first;
    const bool valid = vi < total;
    const int ti = valid ? vi / x.H : 0, h = valid ? vi - ti * x.H : 0;
    const T* src = static_cast<const T*>(x.in) + (n0 + ti) * x.ld_in + int64_t(h) * D;
    float e[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack8<T>(nx[i], e + 8 * i);
    if (vi + per < total) {
      const uint4* p = reinterpret_cast<const uint4*>(source(vi + per) + 32 * part);
#pragma unroll
      for (int i = 0; i < 4; ++i) nx[i] = __ldcs(p + i);
    }
    if (turned && valid) {
      const float2* c = cs + ti * half;
      if (inter) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * part + 2 * i < rot) turn(e[2 * i], e[2 * i + 1], c[16 * part + i]);
      } else {
        // the partners of 8 elements are 8 neighbouring ones, all on one side
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e0 = 32 * part + 8 * i;
          if (e0 < rot) {
            const bool low = e0 < half;
            const int f = low ? e0 : e0 - half;
            const float sign = low ? -1.f : 1.f;
            float o[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(src + (low ? e0 + half : f)), o);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const float4 w = *reinterpret_cast<const float4*>(c + f + j);
              e[8 * i + j] = e[8 * i + j] * w.x + o[j] * (w.y * sign);
              e[8 * i + j + 1] = e[8 * i + j + 1] * w.z + o[j + 1] * (w.w * sign);
            }
          }
        }
      }
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
// One (token, head) vector of the keys and of the values by d / 32 lanes; a CTA
// looks its tokens' places up once.
template <typename T, int D, bool BACK>
__global__ void __launch_bounds__(RT)
read_kernel(const uint8_t* __restrict__ k_q, const __half* __restrict__ k_s, const uint8_t* __restrict__ v_q,
            const __half* __restrict__ v_s, int64_t N, int Hkv, Batch t, T* __restrict__ k_out, T* __restrict__ v_out, int tokens) {
  constexpr int TPV = D / 32;
  __shared__ int row[ATOK], slot[ATOK];  // page (-1: zeros, -2: left as it is) and slot
  const int64_t n0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), N - n0));
  if (int(threadIdx.x) < nt) {
    const Place p = place_of(t, int(n0) + threadIdx.x);
    int r = p.b < 0 ? -2 : -1, sl = 0;
    if (p.b >= 0 && p.pos >= 0) {
      const int index = p.pos / t.ps;
      r = page_at(t, p.b, index);
      sl = p.pos - index * t.ps;
    }
    row[threadIdx.x] = r;
    slot[threadIdx.x] = sl;
  }
  __syncthreads();
  const int total = nt * Hkv, part = int(threadIdx.x) % TPV;
  constexpr int per = RT / TPV;
  for (int base = 0; base < total; base += per) {  // the whole warp takes part in the transform
    const int vi = base + int(threadIdx.x) / TPV;
    const bool valid = vi < total;
    const int ti = valid ? vi / Hkv : 0, h = valid ? vi - ti * Hkv : 0;
    const int page = valid ? row[ti] : -2;
    uint4 r[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    __half sc[2] = {__half(0.f), __half(0.f)};
    if (page >= 0) {
      const int64_t at = (int64_t(page) * Hkv + h) * t.ps + slot[ti];
      r[0] = __ldcs(reinterpret_cast<const uint4*>(k_q + at * (D / 2) + part * 16));
      r[1] = __ldcs(reinterpret_cast<const uint4*>(v_q + at * (D / 2) + part * 16));
      sc[0] = k_s[at];
      sc[1] = v_s[at];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float s = __half2float(sc[which]);
      float e[32];
      codes8(r[which].x, e);
      codes8(r[which].y, e + 8);
      codes8(r[which].z, e + 16);
      codes8(r[which].w, e + 24);
      if constexpr (BACK) {
        hadamard32<TPV>(e, part);  // sums of codes are whole numbers: exact
        s *= 1.0f / sqrtf(float(D));
      }
      if (page != -2) {
        T* dst = (which ? v_out : k_out) + ((n0 + ti) * Hkv + h) * D + 32 * part;
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i] *= s;
#pragma unroll
        for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<uint4*>(dst + 8 * i), pack8<T>(e + 8 * i));
      }
    }
  }
}

// Tokens of a CTA, and CTAs that share a group of tokens: some 12 units a
// thread where there are enough tokens for four CTAs on every SM; else fewer
// tokens, down to one whose heads are shared out.
inline void rope_split(int64_t N, int64_t H, int64_t d, int sms, int* tokens, int* parts) {
  const int64_t units = H * (d >> 4);
  int64_t t = (12 * RT + units - 1) / units;
  const int64_t enough = N / (int64_t(4) * sms);
  t = t > enough ? enough : t;
  t = t < 1 ? 1 : t > ATOK ? ATOK : t;
  while (t > 1 && t * (d / 2) * int64_t(sizeof(float2)) > 16 * 1024) --t;
  int64_t p = 1;
  if (t == 1 && N * units < int64_t(4) * sms * RT) p = (units + RT - 1) / RT;
  *tokens = int(t);
  *parts = int(p);
}
// Tokens of a CTA whose vectors are worked on by d / 32 lanes each: four rounds of them, fewer where CTAs are few.
inline int vector_tokens(int64_t N, int64_t H, int64_t d, int sms) {
  const int64_t per = RT / (d / 32);
  int64_t t = 4 * per / H;
  const int64_t enough = N / (int64_t(4) * sms);
  t = t > enough ? enough : t;
  return int(t < 1 ? 1 : t > ATOK ? ATOK : t);
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
  int tokens, parts;
  rope_split(N, Hq > Hk ? Hq : Hk, d, sms, &tokens, &parts);
  const Heads hq = {q, q_out, ld_q, ld_qo, int(Hq)}, hk = {k, k_out, ld_k, ld_ko, int(Hk)};
  auto kern = dtype == QUAROT_FP16 ? rope_kernel<__half> : rope_kernel<__nv_bfloat16>;
  kern<<<dim3(unsigned((N + tokens - 1) / tokens), unsigned(parts)), RT, size_t(tokens) * (rot / 2) * sizeof(float2),
         static_cast<cudaStream_t>(stream)>>>(hq, hk, N, int(d), positions, inv_freq, int(rot), interleaved, scale, tokens);
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
  int sms = 0;
  if (!sm_count(&sms)) return QUAROT_ERR_CUDA;
  int q_tokens = 1, q_parts = 1;
  if (Hq > 0) rope_split(N, Hq, d, sms, &q_tokens, &q_parts);
  const int kt = vector_tokens(N, Hkv, d, sms);
  const int64_t bkv = (N + kt - 1) / kt, bq = Hq > 0 ? (N + q_tokens - 1) / q_tokens * q_parts : 0;
  if (2 * bkv + bq > 0x7fffffff) return QUAROT_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    kern<<<unsigned(2 * bkv + bq), RT, 0, static_cast<cudaStream_t>(stream)>>>(
        hk, hv, hq, N, inv_freq, int(rot), interleaved, scale, k_q, static_cast<__half*>(k_s), v_q,
        static_cast<__half*>(v_s), t, kt, int(bkv), q_tokens, q_parts);
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
  int sms = 0;
  if (!sm_count(&sms)) return QUAROT_ERR_CUDA;
  const int tokens = vector_tokens(N, Hkv, d, sms);
  auto go = [&](auto kern, auto* ko, auto* vo) {
    kern<<<unsigned((N + tokens - 1) / tokens), RT, 0, static_cast<cudaStream_t>(stream)>>>(
        k_q, static_cast<const __half*>(k_s), v_q, static_cast<const __half*>(v_s), N, int(Hkv), t, ko, vo, tokens);
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
