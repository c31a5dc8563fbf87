// Rotary positions and the paged INT4 cache's writing and reading:
// quarot_rope, quarot_paged_append, quarot_paged_read.
//
// The cache holds what quarot_kv_write stores (the head-wise rotation of
// [S] Stages 1c and 1d, the symmetric quantizer of Stage 2c's procedure), in
// pages: codes [n_pages, Hkv, page_size, d / 2], scales [n_pages, Hkv,
// page_size].  Token p of sequence b is slot p % page_size of page
// table[b][p / page_size].
#include <type_traits>

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
// all their heads, three loaded ahead of the arithmetic.  Bound by HBM: 8192
// tokens of 40 heads of 128 32 us, 5.3 TB/s.
struct Heads {
  const void* in;
  void* out;
  int64_t ld_in, ld_out;
  int H;
};
constexpr int RT = 256;  // threads

// A decode step makes these calls one after another, each hardly longer than
// its launch: they are programmatic dependents, like the 8-bit calls.
__device__ __forceinline__ void begin() {
  fp8::wait_for_previous();
  fp8::next_may_start();
}

// Units of `nt` tokens from n0 on.  A thread has unit u = tid % U of every
// (RT / U * parts)-th head; cs holds a token's cosines, then its sines.  skip: for each token 0 to turn
// it, 1 to write zeros, 2 to leave its output.
template <typename T>
__device__ __forceinline__ void turn_heads(const Heads& x, int64_t n0, int nt, int d, int rot, bool inter, const float* cs,
                                           const int* skip, int part, int parts) {
  constexpr int AHEAD = 3;
  const int U = d >> 4, u = int(threadIdx.x) % U, per = RT / U * parts;
  if (int(threadIdx.x) >= RT / U * U) return;
  const bool turned = 16 * u < rot;
  const int e0 = turned && !inter ? 8 * u : 16 * u, e1 = turned && !inter ? e0 + (rot >> 1) : e0 + 8;
  const int half = rot >> 1;
  const float* c = cs + 8 * u;
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
        r[i][0] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
        r[i][1] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
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
        float2 a[4], b[4];
        unpack8<T>(r[i][0], a);
        unpack8<T>(r[i][1], b);
        const float4* cf = reinterpret_cast<const float4*>(c + tk[i] * rot);
        const float4* sf = reinterpret_cast<const float4*>(c + tk[i] * rot + half);
        const float4 c0 = cf[0], c1 = cf[1], s0 = sf[0], s1 = sf[1];
        if (inter) {
          a[0] = turn1(a[0], c0.x, s0.x), a[1] = turn1(a[1], c0.y, s0.y);
          a[2] = turn1(a[2], c0.z, s0.z), a[3] = turn1(a[3], c0.w, s0.w);
          b[0] = turn1(b[0], c1.x, s1.x), b[1] = turn1(b[1], c1.y, s1.y);
          b[2] = turn1(b[2], c1.z, s1.z), b[3] = turn1(b[3], c1.w, s1.w);
        } else {
          turn2(a[0], b[0], make_float2(c0.x, c0.y), make_float2(s0.x, s0.y));
          turn2(a[1], b[1], make_float2(c0.z, c0.w), make_float2(s0.z, s0.w));
          turn2(a[2], b[2], make_float2(c1.x, c1.y), make_float2(s1.x, s1.y));
          turn2(a[3], b[3], make_float2(c1.z, c1.w), make_float2(s1.z, s1.w));
        }
        r[i][0] = pack8<T>(a);
        r[i][1] = pack8<T>(b);
      }
      if (what == 1) r[i][0] = r[i][1] = make_uint4(0u, 0u, 0u, 0u);
      T* dst = static_cast<T*>(x.out) + (n0 + tk[i]) * x.ld_out + int64_t(hk[i]) * d;
      __stcs(reinterpret_cast<uint4*>(dst + e0), r[i][0]);
      __stcs(reinterpret_cast<uint4*>(dst + e1), r[i][1]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(RT)
rope_kernel(Heads q, Heads k, int64_t N, int d, const int32_t* __restrict__ positions,
            const double* __restrict__ inv_freq, int rot, int inter, float scale, int tokens) {
  extern __shared__ __align__(16) unsigned char rsm[];
  float* cs = reinterpret_cast<float*>(rsm);  // [tokens][cosines, sines]
  const int half = rot >> 1;
  const int64_t n0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), N - n0));
  begin();
  for (int i = threadIdx.x; i < nt * half; i += RT) {
    const int n = i / half, f = i - n * half;
    const float2 v = turn_of(positions[n0 + n], turn_step(inv_freq[f]), scale);
    cs[n * rot + f] = v.x;
    cs[n * rot + half + f] = v.y;
  }
  __syncthreads();
  turn_heads<T>(q, n0, nt, d, rot, inter != 0, cs, nullptr, blockIdx.y, gridDim.y);
  if (k.H > 0) turn_heads<T>(k, n0, nt, d, rot, inter != 0, cs, nullptr, blockIdx.y, gridDim.y);
}

// ------------------------------------------------------------------ append
// As in quarot_kv_write, d / 32 lanes own one (token, head) vector, 32
// elements each.  A CTA takes some neighbouring tokens' keys, values or
// queries, so that places are looked up and angles made once for all heads.
// Bound by latency: with 80 registers a thread a third of the warps are there to
// cover loads, shuffles and the quantizer's chain, and neither issue (55 % of the
// clocks) nor HBM (31 %) is full.  4 x 2048 tokens of 32 + 8 + 8 heads of 128 44 us;
// 16 x 1 4.1 us, a launch and its look-ups.
constexpr int ATOK = 32;      // most tokens of a CTA
constexpr int AHALF = 64;     // most pairs of a head
constexpr int CU = 257;       // entries of cu that a CTA keeps at hand

// The batch with cu in shared memory, where it fits: a search in it is then a
// few steps of some clocks each.  The whole CTA takes part.
__device__ __forceinline__ Batch near(Batch t, int* cu) {
  if (t.cu != nullptr && t.B < CU) {
    for (int i = threadIdx.x; i <= t.B; i += RT) cu[i] = t.cu[i];
    __syncthreads();
    t.cu = cu;
  }
  return t;
}

template <typename T, int D>
__global__ void __launch_bounds__(RT, 3)
append_kernel(Heads k, Heads v, Heads q, int64_t N, const double* __restrict__ inv_freq, int rot, int inter, float scale,
              uint8_t* __restrict__ k_q, __half* __restrict__ k_s, uint8_t* __restrict__ v_q, __half* __restrict__ v_s,
              Batch t, int kv_tokens, int kv_blocks, int q_tokens, int q_parts) {
  constexpr int TPV = D / 32;
  __shared__ __align__(16) float cs[ATOK * AHALF * 2];  // a token's cosines, then its sines
  __shared__ uint64_t step[AHALF];
  __shared__ int row[ATOK], posn[ATOK], skip[ATOK];
  __shared__ int cu[CU];
  // CTAs of keys, values and queries in turn, as long as there are all of them: the former mostly compute, the
  // latter mostly move memory (4 x 2048 tokens, with reading back: queries first 59.9 us, in turn 52.4 us)
  const int m = min(kv_blocks, int(gridDim.x) - 2 * kv_blocks), b = int(blockIdx.x);
  const int which = b < 3 * m ? b % 3 : m < kv_blocks ? (b - 3 * m) & 1 : 2;
  int64_t blk = b < 3 * m ? b / 3 : m < kv_blocks ? m + ((b - 3 * m) >> 1) : b - 2 * m;
  const int q_part = which == 2 ? int(blk % q_parts) : 0;
  if (which == 2) blk /= q_parts;
  const Heads x = which == 0 ? k : which == 1 ? v : q;
  const int nt_max = which == 2 ? q_tokens : kv_tokens;
  const int64_t n0 = blk * nt_max;
  const int nt = int(min(int64_t(nt_max), N - n0));
  const int half = rot >> 1;
  const bool turned = which != 1 && half > 0;
  begin();
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
    nx[i] = which != 2 && first < total ? __ldcs(reinterpret_cast<const uint4*>(source(first) + 32 * part) + i) : make_uint4(0u, 0u, 0u, 0u);
  t = near(t, cu);
  if (int(threadIdx.x) < nt) {
    const Place p = place_of(t, int(n0) + threadIdx.x);
    posn[threadIdx.x] = p.pos;
    skip[threadIdx.x] = p.b < 0 ? 2 : p.pos < 0 ? 1 : 0;
    if (which != 2) row[threadIdx.x] = p.b >= 0 && p.pos >= 0 ? page_at(t, p.b, p.pos / t.ps) : -1;
  }
  if (turned && int(threadIdx.x) < half) step[threadIdx.x] = turn_step(inv_freq[threadIdx.x]);
  __syncthreads();
  if (turned) {
    for (int i = threadIdx.x; i < nt * half; i += RT) {
      const int n = i / half, f = i - n * half;
      const float2 w = turn_of(posn[n], step[f], scale);
      cs[n * rot + f] = w.x;
      cs[n * rot + half + f] = w.y;
    }
    __syncthreads();
  }
  if (which == 2) {
    turn_heads<T>(x, n0, nt, D, rot, inter != 0, cs, skip, q_part, q_parts);
    return;
  }
  for (int base = 0; base < total; base += per) {
    const int vi = base + first;
    const bool valid = vi < total;
    const int ti = valid ? vi / x.H : 0, h = valid ? vi - ti * x.H : 0;
    const T* src = static_cast<const T*>(x.in) + (n0 + ti) * x.ld_in + int64_t(h) * D;
    float2 e[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack8<T>(nx[i], e + 4 * i);
    if (vi + per < total) {
      const uint4* p = reinterpret_cast<const uint4*>(source(vi + per) + 32 * part);
#pragma unroll
      for (int i = 0; i < 4; ++i) nx[i] = __ldcs(p + i);
    }
    if (turned && valid) {
      const float* c = cs + ti * rot;
      if (inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (32 * part + 8 * i < rot) {
            const float4 cf = *reinterpret_cast<const float4*>(c + 16 * part + 4 * i);
            const float4 sf = *reinterpret_cast<const float4*>(c + half + 16 * part + 4 * i);
            e[4 * i] = turn1(e[4 * i], cf.x, sf.x), e[4 * i + 1] = turn1(e[4 * i + 1], cf.y, sf.y);
            e[4 * i + 2] = turn1(e[4 * i + 2], cf.z, sf.z), e[4 * i + 3] = turn1(e[4 * i + 3], cf.w, sf.w);
          }
      } else {
        // the partners of 8 elements are 8 neighbouring ones, all on one side
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e0 = 32 * part + 8 * i;
          if (e0 < rot) {
            const bool low = e0 < half;
            const int f = low ? e0 : e0 - half;
            const float2 sign = make_float2(low ? -1.f : 1.f, low ? -1.f : 1.f);
            float2 o[4];
            unpack8<T>(*reinterpret_cast<const uint4*>(src + (low ? e0 + half : f)), o);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float4 cf = *reinterpret_cast<const float4*>(c + f + 2 * j), sf = *reinterpret_cast<const float4*>(c + half + f + 2 * j);
              e[4 * i + j] = __ffma2_rn(__fmul2_rn(o[j], sign), make_float2(sf.x, sf.y), __fmul2_rn(e[4 * i + j], make_float2(cf.x, cf.y)));
              e[4 * i + j + 1] = __ffma2_rn(__fmul2_rn(o[j + 1], sign), make_float2(sf.z, sf.w), __fmul2_rn(e[4 * i + j + 1], make_float2(cf.z, cf.w)));
            }
          }
        }
      }
    }
    hadamard<32, TPV>(e, part);
    const float inv_sqrt_d = 1.0f / sqrtf(float(D));
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      e[i] = __fmul2_rn(e[i], make_float2(inv_sqrt_d, inv_sqrt_d));
      amax = fmaxf(amax, fmaxf(fabsf(e[i].x), fabsf(e[i].y)));
    }
#pragma unroll
    for (int o = 1; o < TPV; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const __half S = quant_scale_fp16(amax, 1.0f);
    const float s32 = __half2float(S), inv = 1.0f / s32;
    // v / S is v * inv and, to put its two roundings right, the rest of that quotient over S: a quotient of a half then is
    // one, and goes to the even code (2.1 million codes of bf16 values, heads of 64: 20 others without).  fp16 vectors that
    // are not turned keep quarot_kv_write's rounded product, and so its codes (where the compiler fused it with the
    // addition that follows, 34 of 17 million bytes of heads of 64 were others).  4 x 2048 tokens 46.7 us, 45.7 us without.
    const float rest = turned || !std::is_same<T, __half>::value ? inv : 0.f;
    // Only where the scale is at its largest can a quotient round past 7 or -8
    // (else S >= amax / 7 within 2^-11, or 3 % among the subnormals).
    if (__any_sync(0xffffffffu, !(amax < 7.0f * 65504.0f))) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        e[i] = make_float2(fminf(fmaxf(e[i].x, -8.0f * s32), 7.0f * s32), fminf(fmaxf(e[i].y, -8.0f * s32), 7.0f * s32));
      }
    }
    // round(v / S) + 8 as a whole number (adding 1.5 * 2^23 rounds to even), and eight of them to a word in base 16,
    // four at a time: exact in fp32, and no integer instruction for each
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 acc[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 u = __fmul2_rn(e[4 * i + j], make_float2(inv, inv));
        u = __ffma2_rn(__ffma2_rn(u, make_float2(-s32, -s32), e[4 * i + j]), make_float2(rest, rest), u);
        u = __fadd2_rn(u, make_float2(12582912.0f, 12582912.0f));
        u = __fadd2_rn(u, make_float2(-12582904.0f, -12582904.0f));
        acc[j >> 1] = (j & 1) ? __ffma2_rn(u, make_float2(256.0f, 4096.0f), acc[j >> 1]) : __fmul2_rn(u, make_float2(1.0f, 16.0f));
      }
      w[i] = (uint32_t(__float2int_rn(acc[0].x + acc[0].y)) | (uint32_t(__float2int_rn(acc[1].x + acc[1].y)) << 16)) ^ 0x88888888u;
    }
    if (valid && row[ti] >= 0) {
      const int64_t at = (int64_t(row[ti]) * x.H + h) * t.ps + posn[ti] % t.ps;
      *reinterpret_cast<uint4*>((which == 0 ? k_q : v_q) + at * (D / 2) + part * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      if (part == 0) (which == 0 ? k_s : v_s)[at] = S;
    }
  }
}

// ------------------------------------------------------------------ read
// d / 8 lanes own one (token, head) vector of the keys and of the values, one
// packed word each, so that neighbouring lanes write neighbouring 16 bytes (32
// elements a lane, as in append, wrote half sectors: 16 x 4096 tokens 77 us,
// now 60 us, 5.6 TB/s: bound by HBM).  A CTA looks its tokens' places up once;
// four vectors' words are loaded before the first is worked on.
template <typename T, int D, bool BACK>
__global__ void __launch_bounds__(RT)
read_kernel(const uint8_t* __restrict__ k_q, const __half* __restrict__ k_s, const uint8_t* __restrict__ v_q,
            const __half* __restrict__ v_s, int64_t N, int Hkv, Batch t, T* __restrict__ k_out, T* __restrict__ v_out, int tokens) {
  constexpr int TPV = D / 8, AHEAD = 4, per = RT / TPV;
  __shared__ int row[ATOK], slot[ATOK];  // page (-1: zeros, -2: left as it is) and slot
  __shared__ int cu[CU];
  const int64_t n0 = int64_t(blockIdx.x) * tokens;
  const int nt = int(min(int64_t(tokens), N - n0));
  begin();
  t = near(t, cu);
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
  for (int base = 0; base < total; base += per * AHEAD) {  // whole warps take part in the transform
    uint32_t w[AHEAD][2];
    __half sc[AHEAD][2];
    int page[AHEAD], vi[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      vi[i] = base + i * per + int(threadIdx.x) / TPV;
      const bool valid = vi[i] < total;
      const int ti = valid ? vi[i] / Hkv : 0, h = valid ? vi[i] - ti * Hkv : 0;
      page[i] = valid ? row[ti] : -2;
      w[i][0] = w[i][1] = 0u;
      sc[i][0] = sc[i][1] = __half(0.f);
      if (page[i] >= 0) {
        const int64_t at = (int64_t(page[i]) * Hkv + h) * t.ps + slot[ti];
        w[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(k_q + at * (D / 2)) + part);
        w[i][1] = __ldcs(reinterpret_cast<const uint32_t*>(v_q + at * (D / 2)) + part);
        sc[i][0] = k_s[at];
        sc[i][1] = v_s[at];
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (base + i * per >= total) break;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float s = __half2float(sc[i][which]);
        float2 e[4];
        codes8(w[i][which], e);
        if constexpr (BACK) {  // sums of codes are whole numbers: exact
          hadamard<8, TPV>(e, part);
          s *= 1.0f / sqrtf(float(D));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = __fmul2_rn(e[j], make_float2(s, s));
        if (page[i] != -2) __stcs(reinterpret_cast<uint4*>((which ? v_out : k_out) + (n0 * Hkv + vi[i]) * D + 8 * part), pack8<T>(e));
      }
    }
  }
}

// Tokens of a CTA, and CTAs that share a group of tokens: some 6 units a
// thread where there are enough tokens for two CTAs on every SM; else fewer
// tokens, down to one whose heads are shared out.
inline void rope_split(int64_t N, int64_t H, int64_t d, int sms, int* tokens, int* parts) {
  const int64_t units = H * (d >> 4);
  int64_t t = (6 * RT + units - 1) / units;
  const int64_t enough = N / (int64_t(2) * sms);
  t = t > enough ? enough : t;
  t = t < 1 ? 1 : t > ATOK ? ATOK : t;
  while (t > 1 && t * (d / 2) * int64_t(sizeof(float2)) > 16 * 1024) --t;
  int64_t p = 1;
  if (t == 1 && N * units < int64_t(4) * sms * RT) p = (units + RT - 1) / RT;
  *tokens = int(t);
  *parts = int(p);
}
// Tokens of a CTA that works on `per` of their H vectors at a time: four rounds of them, fewer where
// that leaves SMs without one (its look-ups take as long as several rounds: 5 x 700 tokens of 16 heads of 64, 5 tokens a CTA
// 20 us, 23 tokens 14 us; two or eight rounds: 4 x 2048 tokens 55.9 and 54.6 us against 52.4 us).
inline int vector_tokens(int64_t N, int64_t H, int64_t per, int sms) {
  int64_t t = 4 * per / H;
  const int64_t enough = N / sms;
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
  return fp8::launch_dependent(kern, dim3(unsigned((N + tokens - 1) / tokens), unsigned(parts)), RT,
                               size_t(tokens) * rot * sizeof(float), 1, static_cast<cudaStream_t>(stream), hq, hk, N, int(d),
                               positions, inv_freq, int(rot), interleaved, scale, tokens);
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
  const int kt = vector_tokens(N, Hkv, RT / (d / 32), sms);
  const int64_t bkv = (N + kt - 1) / kt, bq = Hq > 0 ? (N + q_tokens - 1) / q_tokens * q_parts : 0;
  if (2 * bkv + bq > 0x7fffffff) return QUAROT_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return fp8::launch_dependent(kern, dim3(unsigned(2 * bkv + bq)), RT, 0, 1, static_cast<cudaStream_t>(stream), hk, hv, hq, N,
                                 inv_freq, int(rot), interleaved, scale, k_q, static_cast<__half*>(k_s), v_q,
                                 static_cast<__half*>(v_s), t, kt, int(bkv), q_tokens, q_parts);
  };
  if (dtype == QUAROT_FP16) return d == 64 ? go(append_kernel<__half, 64>) : go(append_kernel<__half, 128>);
  return d == 64 ? go(append_kernel<__nv_bfloat16, 64>) : go(append_kernel<__nv_bfloat16, 128>);
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
  const int tokens = vector_tokens(N, Hkv, RT / (d / 8), sms);
  auto go = [&](auto kern, auto* ko, auto* vo) {
    return fp8::launch_dependent(kern, dim3(unsigned((N + tokens - 1) / tokens)), RT, 0, 1, static_cast<cudaStream_t>(stream), k_q,
                                 static_cast<const __half*>(k_s), v_q, static_cast<const __half*>(v_s), N, int(Hkv), t, ko, vo,
                                 tokens);
  };
  auto typed = [&](auto* ko, auto* vo) {
    using T = std::remove_pointer_t<decltype(ko)>;
    if (d == 64) return unrotate ? go(read_kernel<T, 64, true>, ko, vo) : go(read_kernel<T, 64, false>, ko, vo);
    return unrotate ? go(read_kernel<T, 128, true>, ko, vo) : go(read_kernel<T, 128, false>, ko, vo);
  };
  if (dtype == QUAROT_FP16) return typed(static_cast<__half*>(k_out), static_cast<__half*>(v_out));
  return typed(static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out));
}
