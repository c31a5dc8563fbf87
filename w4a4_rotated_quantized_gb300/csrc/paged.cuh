// Shared pieces of the paged INT4 cache: where a batch's tokens lie, the
// turning of position pairs, and the head-wise Hadamard transform in registers.
#pragma once

#include <math.h>

#include "fp8.cuh"

namespace quarot {
namespace paged {

// A batch of sequences whose tokens lie in pages.  cu (int32 [B + 1], or null:
// one new token a sequence) says which of the batch's N new tokens belong to
// which sequence; lengths count the new ones.
struct Batch {
  const int32_t* table;    // [B, max_pages]
  const int32_t* lengths;  // [B]
  const int32_t* cu;
  int B, max_pages, n_pages, ps;
};

// Sequence and position of new token n.  b < 0: the token is behind the last
// sequence.  pos < 0: its sequence is shorter than its new tokens.
struct Place {
  int b, pos;
};
__device__ __forceinline__ Place place_of(const Batch& t, int n) {
  Place p;
  if (t.cu == nullptr) {
    p.b = n < t.B ? n : -1;
    p.pos = p.b < 0 ? -1 : t.lengths[p.b] - 1;
    return p;
  }
  if (n < t.cu[0] || n >= t.cu[t.B]) return {-1, -1};
  int lo = 0, hi = t.B;  // cu[lo] <= n < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.cu[mid] <= n) lo = mid;
    else hi = mid;
  }
  p.b = lo;
  p.pos = t.lengths[lo] - (t.cu[lo + 1] - n);
  return p;
}

// The index-th page of sequence b; -1 (and an error for quarot_check_error)
// where the table has none.
__device__ __forceinline__ int page_at(const Batch& t, int b, int index) {
  const int page = index < t.max_pages ? t.table[int64_t(b) * t.max_pages + index] : -1;
  if (page >= 0 && page < t.n_pages) return page;
  record_error(QUAROT_ERR_INVALID_ARG);
  return -1;
}

// ------------------------------------------------------------------ positions
// Pair i of a head at position p is turned by p * inv_freq[i].  Far positions
// leave nothing of an angle's fraction in fp32 (2^20 rad has steps of 1/8), so
// the angle is counted in turns of 2^64: one double product per frequency,
// then position times step is an exact integer product that wraps as the angle
// does.  An error of half a unit in the double's last place moves the angle
// at position p by p * 2^-54 turns.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  double f = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  f -= floor(f);
  return __double2ull_rz(f * 18446744073709551616.0);
}
// cos and sin of position * step, times scale.
__device__ __forceinline__ float2 turn_of(int pos, uint64_t step, float scale) {
  const uint64_t a = uint64_t(int64_t(pos)) * step;
  float s, c;
  sincospif(float(int32_t(a >> 32)) * (1.0f / 2147483648.0f), &s, &c);
  return make_float2(c * scale, s * scale);
}
__device__ __forceinline__ float2 negated(float2 v) { return make_float2(-v.x, -v.y); }
// Two pairs (a, b), each element of both in one register pair.
__device__ __forceinline__ void turn2(float2& a, float2& b, float2 c, float2 s) {
  const float2 u = __ffma2_rn(b, negated(s), __fmul2_rn(a, c));
  b = __ffma2_rn(a, s, __fmul2_rn(b, c));
  a = u;
}
// A pair of neighbours.
__device__ __forceinline__ float2 turn1(float2 v, float c, float s) {
  return make_float2(v.x * c - v.y * s, v.y * c + v.x * s);
}

// ------------------------------------------------------------------ vectors
// 8 elements of 16 bits from or to one 16-byte access.
template <typename T>
__device__ __forceinline__ void unpack8(uint4 r, float2* v) {
  v[0] = fp8::to_f2<T>(r.x);
  v[1] = fp8::to_f2<T>(r.y);
  v[2] = fp8::to_f2<T>(r.z);
  v[3] = fp8::to_f2<T>(r.w);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float2* v) {
  return make_uint4(fp8::from_f2<T>(v[0]), fp8::from_f2<T>(v[1]), fp8::from_f2<T>(v[2]), fp8::from_f2<T>(v[3]));
}
// x H of a vector of E * TPV elements, E consecutive ones in each of TPV
// neighbouring lanes (the whole warp takes part), two to a register pair.  Not
// divided by the root.
template <int E, int TPV>
__device__ __forceinline__ void hadamard(float2* v, int part) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) v[i] = make_float2(v[i].x + v[i].y, v[i].x - v[i].y);
#pragma unroll
  for (int h = 1; h < E / 2; h <<= 1)
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      if ((i & h) == 0) {
        const float2 a = v[i], b = v[i + h];
        v[i] = __fadd2_rn(a, b);
        v[i + h] = __fadd2_rn(a, negated(b));
      }
#pragma unroll
  for (int o = 1; o < TPV; o <<= 1) {
    const float sign = (part & o) != 0 ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      v[i] = __ffma2_rn(v[i], make_float2(sign, sign),
                        make_float2(__shfl_xor_sync(0xffffffffu, v[i].x, o), __shfl_xor_sync(0xffffffffu, v[i].y, o)));
  }
}

// Codes of one 32-bit word, the even dim in the low nibble.
__device__ __forceinline__ void codes8(uint32_t w, float2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_float2(float(int32_t(w << (28 - 8 * i)) >> 28), float(int32_t(w << (24 - 8 * i)) >> 28));
}

// ------------------------------------------------------------------ checks
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // tokens of a batch, and sequences
constexpr int64_t kMaxHeads = 1024;

// Sizes that every paged entry point checks alike.
inline int check_sizes(int dtype, int64_t N, int64_t Hkv, int64_t d, int64_t n_pages, int64_t ps, int64_t B,
                       int64_t max_pages, const void* cu) {
  if (dtype != QUAROT_FP16 && dtype != QUAROT_BF16) return QUAROT_ERR_INVALID_ARG;
  if (N < 0 || B < 0 || Hkv <= 0 || d <= 0 || n_pages < 0 || ps <= 0 || max_pages < 0) return QUAROT_ERR_INVALID_ARG;
  if (cu == nullptr && N != B) return QUAROT_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return QUAROT_ERR_UNSUPPORTED;
  if (ps % 16 != 0 || ps > 65536 || n_pages > 0x7fffffff || max_pages > 0x7fff0000 / ps) return QUAROT_ERR_UNSUPPORTED;
  if (N > kMaxTokens || B > kMaxTokens || Hkv > kMaxHeads || n_pages > (int64_t(1) << 35) / (Hkv * ps))
    return QUAROT_ERR_UNSUPPORTED;
  return QUAROT_OK;
}
// The cache's tensors and the batch's, once sizes are right and there is work.
inline int check_cache(const void* k_q, const void* k_s, const void* v_q, const void* v_s, const void* table,
                       const void* lengths, const void* cu, int64_t max_pages) {
  if (!k_q || !k_s || !v_q || !v_s || !lengths || (!table && max_pages > 0)) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(k_q, 16) || misaligned(v_q, 16) || misaligned(k_s, 16) || misaligned(v_s, 16) || misaligned(table, 4) ||
      misaligned(lengths, 4) || misaligned(cu, 4))
    return QUAROT_ERR_ALIGNMENT;
  return QUAROT_OK;
}
// A [N, H, d] tensor of 16-bit elements whose tokens are ld elements apart.
inline int check_heads(const void* p, int64_t ld, int64_t H, int64_t d) {
  if (p == nullptr || ld < H * d) return QUAROT_ERR_INVALID_ARG;
  return (misaligned(p, 16) || ld % 8 != 0) ? QUAROT_ERR_ALIGNMENT : QUAROT_OK;
}
inline int check_rotation(const void* inv_freq, int64_t rot, int64_t d, int interleaved) {
  if (interleaved != 0 && interleaved != 1) return QUAROT_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || (rot > 0 && inv_freq == nullptr)) return QUAROT_ERR_INVALID_ARG;
  if (rot % 16 != 0) return QUAROT_ERR_UNSUPPORTED;
  return misaligned(inv_freq, 8) ? QUAROT_ERR_ALIGNMENT : QUAROT_OK;
}
inline bool sm_count(int* sms) {
  int dev = 0;
  return cuda_ok(cudaGetDevice(&dev)) && cuda_ok(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
}

}  // namespace paged
}  // namespace quarot
