// quarot_paged_attn: attention over the paged INT4 cache.
//
// For new token i at position p of sequence b, and query head h of group
// g = h / (Hq / Hkv):
//   q~ = q H_d / sqrt(d),  s_t = sm_scale * q~ . (k_s[t] kcode_t)  for t <= p
//   out = sum_t softmax(s)_t v_s[t] vcode_t
//
// Rows (a token's heads of one group, R = Hq / Hkv a token) that attend to the
// same keys are worked on together.  With a shared prefix there are two parts:
// all rows of the batch against the shared tokens, once, and each sequence's
// rows against its own tokens; without one there is the second alone.  A part
// is a list of units, a unit being up to RP rows of one KV head and the tiles
// of 128 tokens that they see.  The tiles of all units lie in one row, which
// is cut into equal pieces, one a CTA, whatever the sequences' lengths: a CTA
// works on the end of one unit, whole ones, and the start of another, and
// leaves a partial softmax state (o, m, l) of each in the workspace, which the
// last kernel joins.  The cut depends on the lengths and the number of CTAs
// alone, so results are the same every time.
#include "paged.cuh"

namespace quarot {
namespace paged {

// ------------------------------------------------------------------ tcgen05
// Shared-memory descriptors (addresses and offsets in 16-byte units, version 1):
// 128-byte swizzle, 8-row groups `sbo` bytes apart; no swizzle, with both offsets.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t sbo) {
  return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t(1) << 16) | (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46);
}
// Instruction descriptor of kind::f8f6f4, e4m3 x e4m3 to fp32: M = 128, N = n;
// a_mn, b_mn: the operand is stored with M (N) running fastest.
__host__ __device__ constexpr uint32_t idesc8(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)));
}
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)));
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void tmem_ld8(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 8 N columns: lane l holds columns 8 i + 2 (l % 4) and + 1 of row
// l / 4 in r[4 i], r[4 i + 1], of row l / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_st_rows4(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_rows2(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// One lane of a converged warp, in the form in which the compiler sees that it is one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Bytes (a multiple of 16, like both addresses) from global to this CTA's shared memory.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 8 offset codes u = v + 8 of a packed word as e4m3 bytes with that bit
// pattern, whose value is u 2^-9: even dims in lo, odd ones in hi.  (w & mask)
// ^ flip is one instruction when both constants are in registers; as literals
// they make it two, so they come as values that the compiler does not know.
struct Masks {
  uint32_t mask, flip;  // 0x0F0F0F0F, 0x08080808
};
__device__ __forceinline__ void bytes_of(uint32_t w, Masks m, uint32_t& lo, uint32_t& hi) {
  lo = (w & m.mask) ^ m.flip;
  hi = ((w >> 4) & m.mask) ^ m.flip;
}
__device__ __forceinline__ uint32_t e4m3x2_of_h2(uint32_t h) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h));
  return d;
}
__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint32_t c) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(uint16_t(c)));
  return d;
}
__device__ __forceinline__ uint32_t h2_of_f2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// (a - b) * 16 of fp16 pairs, exact where b is a rounded to fewer bits.
__device__ __forceinline__ uint32_t rest16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}" : "=r"(d) : "r"(a), "r"(b), "r"(0x4C004C00u));
  return d;
}
// An fp16 pair as three e4m3 pairs, a = c0 + c1 / 16 + c2 / 256 + what is
// returned / 256: 4 bits of fraction each hold all 11 of an fp16 down to 2^-6,
// fewer below, and nothing below 2^-18.
__device__ __forceinline__ uint32_t pieces_of(uint32_t a, uint32_t* c) {
  c[0] = e4m3x2_of_h2(a);
  a = rest16(a, h2_of_e4m3x2(c[0]));
  c[1] = e4m3x2_of_h2(a);
  a = rest16(a, h2_of_e4m3x2(c[1]));
  c[2] = e4m3x2_of_h2(a);
  uint32_t left;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(left) : "r"(a), "r"(h2_of_e4m3x2(c[2])));
  return left;
}

// ------------------------------------------------------------------ units
constexpr int TILE = 128;  // tokens
constexpr int kTries = 1 << 18;
constexpr float kLeast = 0x1p-112f;  // a query's largest element counts as this much at least: 256 over it stays finite, and its scores are 0
constexpr float kNone = -1e30f;  // reference of a row that has seen nothing: 2^(kNone - s) is 0

// One part of a call: the shared prefix (rows of all N tokens as one list,
// tokens [0, shared)), the sequences' own tokens [shared, length), or (whole)
// all tokens of each sequence, the shared ones from the first one's pages.
struct Part {
  Batch t;
  int N, G, Hkv, shared, prefix, whole;
  int RP;  // rows of a unit
};

__device__ __forceinline__ int cu_at(const Part& p, int b) {
  return p.t.cu == nullptr ? b : min(max(__ldcg(p.t.cu + b), 0), p.N);
}
// A sequence as a part sees it.
struct Seq {
  int tok0, rows;      // first token, rows (tokens * G)
  int first, len;      // position of token tok0, tokens in the cache
  int tile0;           // first tile
};
__device__ __forceinline__ Seq seq_of(const Part& p, int b, bool tell) {
  Seq s;
  if (p.prefix) return {0, p.N * p.G, 0, p.shared, 0};
  s.tok0 = cu_at(p, b);
  const int n = max(cu_at(p, b + 1) - s.tok0, 0);
  const int cap = p.t.max_pages * p.t.ps;
  const int len = max(__ldcg(p.t.lengths + b), 0);
  if (len > cap && tell) record_error(QUAROT_ERR_INVALID_ARG);
  s.rows = n * p.G;
  s.first = len - n;
  s.len = min(len, cap);
  s.tile0 = p.shared / TILE;
  return s;
}
// Tiles of row tile j.
__device__ __forceinline__ int tiles_of(const Part& p, const Seq& s, int j) {
  int end = s.len;
  if (!p.prefix) {
    const int last = min(p.RP * (j + 1), s.rows) - 1;
    end = min(end, s.first + last / p.G + 1);
  }
  if (end <= 0) return 0;
  const int own = (end + TILE - 1) / TILE - s.tile0;
  if (!p.whole) return max(own, 0);
  return (min(end, p.shared) + TILE - 1) / TILE + (end > p.shared ? own : 0);
}
// Tiles of one KV head of a sequence.
__device__ __forceinline__ int64_t steps_of(const Part& p, const Seq& s) {
  const int J = (s.rows + p.RP - 1) / p.RP;
  if (p.prefix) return int64_t(J) * tiles_of(p, s, 0);
  int64_t n = 0;
  for (int j = 0; j < J; ++j) n += tiles_of(p, s, j);
  return n;
}
// Number of a sequence's first unit: ceilings of what lies between two
// multiples never pass the next number.
__host__ __device__ inline int64_t unit_base(int64_t tok0, int64_t b, int64_t G, int64_t Hkv, int64_t RP) {
  return Hkv * (tok0 * G / RP + b);
}
__host__ __device__ inline int64_t unit_count(int64_t N, int64_t B, int64_t G, int64_t Hkv, int64_t RP) {
  return unit_base(N, B, G, Hkv, RP);
}

// Where a part's states lie in the workspace: unit u's first and last CTA, and
// for CTA w its state of unit u in slot u + w (one more of either is one more
// slot), o [slots, RP, d] and (m, l) [slots, RP, 2].
struct Space {
  int* span;  // [units, 2]
  float* ml;
  float* o;
  int ctas;
};
constexpr size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
inline size_t space_bytes(int64_t units, int64_t ctas, int64_t RP, int64_t d) {
  const size_t slots = size_t(units + ctas);
  return round256(size_t(units) * 8) + round256(slots * RP * 8) + round256(slots * RP * d * 4);
}
inline Space space_at(unsigned char* p, int64_t units, int64_t ctas, int64_t RP) {
  Space s;
  s.span = reinterpret_cast<int*>(p);
  p += round256(size_t(units) * 8);
  s.ml = reinterpret_cast<float*>(p);
  p += round256(size_t(units + ctas) * RP * 8);
  s.o = reinterpret_cast<float*>(p);
  s.ctas = int(ctas);
  return s;
}

// A CTA's place in the row of all tiles: found once by all its threads.
struct Cursor {
  int b, g, j, tile, tiles;  // unit (b, g, j), next of its tiles, all of them
  Seq s;
};
// Sums over the block: of the threads up to this one, and (returned) of all.  sh: a word a warp, at most 24.
__device__ __forceinline__ int64_t block_scan(int64_t& v, int64_t* sh) {
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (int(threadIdx.x & 31) >= o) v += y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 31) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < int(blockDim.x >> 5); ++w) {
    if (w < int(threadIdx.x >> 5)) v += sh[w];
    all += sh[w];
  }
  return all;
}
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // both positive
  return (a | b) >> 32 ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}
// A cursor from thread 0 to all, through 16 ints of shared memory: whatever the
// batch's arrays do meanwhile, the threads of a CTA agree on its tiles.
__device__ __forceinline__ void tell_cursor(const Cursor& c, int* sh) {
  const int v[10] = {c.b, c.g, c.j, c.tile, c.tiles, c.s.tok0, c.s.rows, c.s.first, c.s.len, c.s.tile0};
#pragma unroll
  for (int i = 0; i < 10; ++i) sh[i] = v[i];
}
__device__ __forceinline__ Cursor told_cursor(const int* sh) {
  return {sh[0], sh[1], sh[2], sh[3], sh[4], {sh[5], sh[6], sh[7], sh[8], sh[9]}};
}
// Sets the cursor to this CTA's first tile (the row of all tiles is cut into
// equal parts, the last ones maybe none) and returns how many it has.  sh: 34 words of shared memory.
// per: the tiles of each but the last CTAs.
__device__ __forceinline__ int64_t find_start(const Part& p, Cursor& c, int64_t& per, int64_t* sh) {
  const int n = blockDim.x, nseq = p.prefix ? 1 : p.t.B, tid = threadIdx.x;
  const bool tell = blockIdx.x == 0;
  // sequences in blocks of n, this thread's within the first one kept
  Seq mine = {0, 0, 0, 0, 0};
  int64_t head = 0;  // its tiles of one KV head
  if (tid < nseq) {
    mine = seq_of(p, tid, tell);
    head = steps_of(p, mine);
  }
  const int64_t own = head * p.Hkv;
  int64_t first = own, sum = own;
  for (int b = tid + n; b < nseq; b += n) sum += steps_of(p, seq_of(p, b, tell)) * p.Hkv;
  if (tid == 0) sh[24] = 0;  // whether some thread found the tile
  int64_t all = block_scan(first, sh), total = all;
  if (nseq > n) total = block_scan(sum, sh);
  if (total == 0) return 0;
  per = quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t at = per * blockIdx.x;
  if (at >= total) return 0;
  int64_t v = own, x = first, done = 0;
  for (int b0 = 0;;) {
    if (v > 0 && at >= done + x - v && at < done + x) {
      int64_t rest = at - (done + x - v);
      c.b = b0 + tid;
      c.s = mine;
      c.g = int(quotient(rest, head));
      rest -= c.g * head;
      c.j = 0;
      if (p.prefix) {
        c.tiles = tiles_of(p, c.s, 0);
        c.j = int(quotient(rest, c.tiles));
        rest -= int64_t(c.j) * c.tiles;
      } else {
        while (rest >= (c.tiles = tiles_of(p, c.s, c.j))) {
          rest -= c.tiles;
          ++c.j;
        }
      }
      c.tile = int(rest);
      tell_cursor(c, reinterpret_cast<int*>(sh + 26));
      sh[24] = 1;
    }
    __syncthreads();
    if (sh[24] != 0) break;
    done += all;
    b0 += n;
    if (b0 >= nseq) return 0;  // the batch changed under the call
    head = v = 0;
    if (b0 + tid < nseq) {
      mine = seq_of(p, b0 + tid, false);
      head = steps_of(p, mine);
      v = head * p.Hkv;
    }
    x = v;
    all = block_scan(x, sh);
  }
  c = told_cursor(reinterpret_cast<int*>(sh + 26));
  __syncthreads();
  return min(per, total - at);
}
// The next unit that has tiles; without one (the batch changed under the call) c.tiles is 0.
__device__ __forceinline__ void next_unit(const Part& p, Cursor& c) {
  c.tile = 0;
  for (;;) {
    if (++c.j * p.RP >= c.s.rows) {
      c.j = 0;
      if (++c.g == p.Hkv) {
        c.g = 0;
        do {
          if (++c.b >= (p.prefix ? 1 : p.t.B)) {
            c.tiles = 0;
            return;
          }
          c.s = seq_of(p, c.b, false);
        } while (c.s.rows == 0);
      }
    }
    c.tiles = tiles_of(p, c.s, c.j);
    if (c.tiles > 0) return;
  }
}

// A row: its token, its query head within the group, and how many tokens it sees.
struct Row {
  int tok, hh, end;
};
__device__ __forceinline__ Row row_of(const Part& p, const Seq& s, int rr) {
  Row r = {-1, 0, 0};
  if (rr >= s.rows) return r;
  const int i = rr / p.G;
  r.hh = rr - i * p.G;
  r.tok = s.tok0 + i;
  int pos = s.first + i;
  if (p.prefix) {
    const Place w = place_of(p.t, r.tok);
    pos = w.b < 0 ? -1 : w.pos;
  }
  r.end = min(max(pos + 1, 0), s.len);
  return r;
}

// ===================================================================== few
// Up to 16 rows.  Everything that would be multiplied is small against the
// cache's bytes, so the kernel is made to read them at the memory's rate:
//   - a packed word becomes 8 operand bytes in 3 instructions (bytes_of), 8 bits
//     being what the tensor cores take: queries and probabilities, which need
//     more, are three e4m3 pieces each, in columns of their own;
//   - S^T [tokens, 3 RP] = K Q^T with the tokens as the MMA's M: the keys go
//     from registers to tensor memory (the A operand), never through shared
//     memory; a thread then holds one token's scores, so the token's scales are
//     its own registers;
//   - O^T [dims, 3 RP] += V^T P^T: values lie in shared memory as they come,
//     token after token (the A operand, M running fastest), and a thread writes
//     its token's 3 RP probability bytes with one or a few 16-byte stores.
// The offset of the codes (u = v + 8) is taken out of the results: 8 sum q~ of
// each score, 8 sum p' of each output.
//
// Softmax: p' = 2^(s - m) v_s, with m raised only when some s + log2 v_s
// exceeds it by 8, and then to 5 below that, so p' <= 2^8 and the largest is at
// least 2^5: fp16, then its pieces, hold it to 2^-12, and a small one to 2^-18.
// (With one token that outweighs the others by far, 16 x 4096 tokens, their
// rounding left 9e-4 of an output where the largest was 1; now 2.4e-4, of which
// the output's own rounding is 2.1e-4.)  Sums of 2^(s - m) and of p' stay in fp32,
// those of p' over what the products take, which is the pieces' sum, so that a
// rounding weighs a code and not code + 8 (35 tokens: error 4.2e-4 without; over the
// fp16 values, whose small ones lose bits in the pieces, 32768 tokens of which one
// outweighs the others 2^24 times: 4.5e-3, now 3.9e-4).
//
// A CTA is four warps that unpack and do the softmax, and a fifth that feeds
// them: it looks up the pages, has the packed tiles copied to shared memory two
// ahead (contiguous pages, or parts of one, in one copy), and issues the MMAs.
// There is one barrier a tile: behind it the fifth warp issues the scores'
// products of the next tile and the outputs' of this one, and copies over what
// was read.  The barrier also tells whether some thread's score passed its
// reference; then the references are raised and the probabilities made again
// (a unit's first tile sets them before).  Several CTAs on an SM fill each other's waits.
//
// What bounds it: a tile's chain of hand-overs, and with few tiles a CTA the
// launches and the join.  32 query and 8 key heads of 128, with the join: 16 x 4096
// tokens 26 us (2.7 TB/s of pages), 64 x 4096 66 us (4.2 TB/s), 1 x 4097 10 us.
namespace few {

constexpr int NT = 160;
constexpr int FEED = 4;  // the feeding warp

template <int RP, int D>
struct Cfg {
  static constexpr int NC = RP == 4 ? 16 : RP == 8 ? 32 : 48;  // columns: piece * RP + row
  static constexpr int KC = D / 4;                             // tensor-memory columns of a key
  static constexpr uint32_t COLS = KC + 2 * NC <= 64 ? 64 : 128;
  static constexpr int WPT = D / 32;                           // packed words a thread has of a token
  static constexpr int CODES = TILE * D / 2;                   // packed codes of a tile
  static constexpr int STAGE_V = CODES + 2 * TILE * 2;         // with key scales and value scales
  static constexpr int OFF_V = 0;                              // [128 tokens][128 bytes], swizzled
  static constexpr int OFF_Q = OFF_V + TILE * 128;             // [NC][128 bytes], swizzled
  static constexpr int OFF_P = (OFF_Q + NC * 128 + 1023) / 1024 * 1024;  // [NC / 16][128 tokens][16 bytes]
  static constexpr int OFF_RK = OFF_P + NC * TILE;             // packed keys, two tiles
  static constexpr int OFF_RV = OFF_RK + 2 * CODES;            // packed values and scales, two tiles
  static constexpr int OFF_ROW = OFF_RV + 2 * STAGE_V;         // four numbers a row
  static constexpr int OFF_X = OFF_ROW + RP * 16;              // float [4][2 RP] exchange
  static constexpr int OFF_CUR = OFF_X + 4 * 2 * RP * 4;       // the next cursor; find_start's words begin 208 bytes before
  static constexpr int OFF_BAR = OFF_CUR + 64;
  static constexpr int SMEM = OFF_BAR + 80;
};
template <int RP>
constexpr int ctas_per_sm() {
  return RP == 4 ? 4 : RP == 8 ? 3 : 2;
}

template <typename T, int RP, int D>
__global__ void __launch_bounds__(NT, ctas_per_sm<RP>())
few_kernel(const T* __restrict__ q, int64_t ld_q, const uint8_t* __restrict__ k_q, const __half* __restrict__ k_s,
           const uint8_t* __restrict__ v_q, const __half* __restrict__ v_s, Part part, float qscale, Space ws, int behind,
           Masks masks) {
  using C = Cfg<RP, D>;
  constexpr int NC = C::NC, WPT = C::WPT;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sma = smem_u32(sm);
  // of the rows, two at a time: factor and offset of the scores, the tokens they see, reference m + 8
  float2* rowf = reinterpret_cast<float2*>(sm + C::OFF_ROW);
  float2* rowo = rowf + RP / 2;
  int2* rowe = reinterpret_cast<int2*>(rowo + RP / 2);
  float2* mtop = reinterpret_cast<float2*>(rowe + RP / 2);
  float* xch = reinterpret_cast<float*>(sm + C::OFF_X);
  int* next = reinterpret_cast<int*>(sm + C::OFF_CUR);
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* bar_o = bar_s + 1;
  uint64_t* bar_k = bar_s + 2;  // [2]
  uint64_t* bar_v = bar_s + 4;  // [2]
  volatile int* there = reinterpret_cast<volatile int*>(bar_s + 6);  // [2]: which groups of 16 tokens a tile has
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(bar_s + 7);
  volatile int* gave_up = reinterpret_cast<volatile int*>(bar_s + 8);

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) mbar_init(bar_s + i, 1);
    *gave_up = 0;
    fence_barrier_init();
  }
  if (warp == FEED) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(const_cast<uint32_t*>(slot))),
                 "r"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  // behind the prefix part of the same call, what this part reads was there
  // before that part's CTAs let it start
  if (!behind) fp8::wait_for_previous();
  fp8::next_may_start();

  const uint32_t tm_k = tmem, tm_s = tmem + C::KC, tm_o = tm_s + NC;
  const Batch& bt = part.t;
  Cursor cur;
  int64_t per;
  int64_t left = find_start(part, cur, per, reinterpret_cast<int64_t*>(sm + C::OFF_CUR - 208));
  // A wait ends after about a second (each try sleeps some microseconds) and is
  // recorded.  Once one gave up, waits for MMAs end at once; copies are waited
  // for all the same, so that none is in flight when the CTA ends.
  auto wait = [&](uint64_t* bar, uint32_t phase, bool copy) {
    bool ok = mbar_try_wait(bar, phase);
    for (int n = 0; !ok && n < kTries && (copy || !*gave_up); ++n) ok = mbar_try_wait(bar, phase);
    if (!ok) {
      *gave_up = 1;
      record_error(QUAROT_ERR_TIMEOUT);
    }
    __syncwarp();
  };

  if (warp == FEED) {
    // ================================================================ feeder
    const int shift = (bt.ps & (bt.ps - 1)) == 0 ? __ffs(bt.ps) - 1 : -1;
    const int lo = part.prefix ? 0 : part.shared;
    const int rows_of_page = part.Hkv * (bt.ps >> 4);
    Cursor f = cur;
    int64_t ahead = left;  // tiles not looked up yet
    int page = -2, off = 0;
    // lane l < 8: page of the next tile's group l of 16 tokens, and the group's place in it in units of 16 rows
    auto look = [&]() {
      page = -2;
      if (ahead <= 0) return;
      --ahead;
      if (f.tiles == 0) return;
      const int tb = (f.s.tile0 + f.tile) * TILE + 16 * (lane & 7);
      const int index = shift >= 0 ? tb >> shift : tb / bt.ps;
      off = f.g * (bt.ps >> 4) + ((tb - index * bt.ps) >> 4);
      if (lane < 8 && tb < f.s.len && tb + 16 > lo)
        page = index < bt.max_pages ? __ldcg(bt.table + int64_t(part.prefix ? 0 : f.b) * bt.max_pages + index) : -1;
      if (++f.tile == f.tiles && ahead > 0) next_unit(part, f);
    };
    auto take = [&]() -> int {  // that group's first row, -1: none
      int row = -1;
      if (unsigned(page) < unsigned(bt.n_pages)) row = page * rows_of_page + off;
      else if (page != -2) record_error(QUAROT_ERR_INVALID_ARG);
      look();
      return row;
    };
    int rows[2] = {-1, -1};  // of the latest two tiles
    uint32_t nk = 0, nv = 0;
    const int64_t total = left;
    auto copy = [&](bool keys, int row) {
      const uint32_t n = keys ? nk : nv, st = n & 1;
      const unsigned valid = __ballot_sync(0xffffffffu, row >= 0) & 0xFF;
      const int before = __shfl_up_sync(0xffffffffu, row, 1);
      unsigned starts = __ballot_sync(0xffffffffu, row >= 0 && (lane == 0 || before < 0 || row != before + 1)) & 0xFF;
      const unsigned ends = (starts | ~valid) & 0x1FF;
      uint64_t* bar = (keys ? bar_k : bar_v) + st;
      const uint32_t to = sma + (keys ? C::OFF_RK + st * C::CODES : C::OFF_RV + st * C::STAGE_V);
      constexpr uint32_t GROUP = 16 * D / 2;
      if (elect_one()) {
        if (!keys) there[st] = int(valid);
        mbar_arrive_expect_tx(bar, __popc(valid) * (GROUP + (keys ? 0 : 64)));
      }
      while (starts) {
        const int a = __ffs(starts) - 1;
        starts &= starts - 1;
        const int len = __ffs(ends >> (a + 1));
        const int64_t r = __shfl_sync(0xffffffffu, row, a);
        if (elect_one()) {
          bulk_copy(to + a * GROUP, (keys ? k_q : v_q) + r * GROUP, len * GROUP, bar);
          if (!keys) {
            bulk_copy(to + C::CODES + a * 32, k_s + r * 16, len * 32, bar);
            bulk_copy(to + C::CODES + 2 * TILE + a * 32, v_s + r * 16, len * 32, bar);
          }
        }
      }
      __syncwarp();
    };
    auto feed_keys = [&]() {
      if (nk >= total) return;
      const int row = take();
      rows[0] = rows[1];
      rows[1] = row;
      copy(true, row);
      ++nk;
    };
    auto feed_values = [&]() {
      if (nv >= total) return;
      copy(false, nk == nv + 1 ? rows[1] : rows[0]);
      ++nv;
    };
    auto issue_scores = [&]() {
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk)
        mma8_ts(tm_s, tm_k + 8 * kk, desc_sw128(sma + C::OFF_Q + 32 * kk, 1024), idesc8(NC, false, false), kk > 0);
      mma_commit(bar_s);
    };
    look();
    feed_keys();
    feed_values();
    feed_keys();
    feed_values();
    while (left > 0) {
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      __syncthreads();  // the queries and the first keys are there
      tc_after();
      if (elect_one()) issue_scores();
      __syncwarp();
      to_async_proxy();
      feed_keys();
      for (int it = 0; it < nt; ++it) {
        if (it == 0 || __syncthreads_or(0))
          for (int i = 0; i < 4; ++i) __syncthreads();
        tc_after();
        if (elect_one()) {
          if (it + 1 < nt) issue_scores();
#pragma unroll
          for (int kk = 0; kk < TILE / 32; ++kk)
            mma8_ss(tm_o, desc_sw128(sma + C::OFF_V + 4096 * kk, 1024), desc_plain(sma + C::OFF_P + 512 * kk, 128, 16 * TILE),
                    idesc8(NC, true, true), it > 0 || kk > 0);
          mma_commit(bar_o);
        }
        __syncwarp();
        to_async_proxy();
        if (it + 1 < nt) feed_keys();
        feed_values();
      }
      left -= nt;
      cur.tile += nt;
      if (left > 0) {
        next_unit(part, cur);
        if (lane == 0) tell_cursor(cur, next);
      }
      __syncthreads();
      if (left > 0) cur = told_cursor(next);
      __syncthreads();
      if (cur.tiles == 0) break;
    }
    for (uint32_t n = nk < 2 ? 0 : nk - 2; n < nk; ++n) wait(bar_k + (n & 1), (n >> 1) & 1, true);
    for (uint32_t n = nv < 2 ? 0 : nv - 2; n < nv; ++n) wait(bar_v + (n & 1), (n >> 1) & 1, true);
  } else {
    // ================================================================ unpacking and softmax
    const uint32_t quad = uint32_t(32 * warp) << 16;
    const int r4 = lane >> 2, c4 = lane & 3;
    const uint32_t frag = (32 * warp + r4) * (D / 2) + c4 * (4 * WPT);  // this lane's words of token 32 warp + r4
    uint32_t v_dst[2];  // and its 16-byte chunks of that token's row of values
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v_dst[h] = sma + C::OFF_V + (32 * warp + r4) * 128 + ((((WPT / 2) * c4 + h % (WPT / 2)) ^ r4) << 4);
    const uint32_t p_dst = sma + C::OFF_P + tid * 16;
    auto words = [&](uint32_t from, uint32_t (*w)[WPT]) {  // of tokens 32 warp + r4 + 8 i
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = from + frag + 8 * (D / 2) * i;
        if constexpr (WPT == 4)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]) : "r"(at));
        else
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(at));
      }
    };
    // keys of the CTA's tile n, unpacked, to tensor memory
    auto put_keys = [&](uint32_t n) {
      uint32_t kw[4][WPT];
      wait(bar_k + (n & 1), (n >> 1) & 1, true);
      words(sma + C::OFF_RK + (n & 1) * C::CODES, kw);
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
        uint32_t a[4 * WPT];
#pragma unroll
        for (int j = 0; j < WPT; ++j) {
          bytes_of(kw[2 * gi][j], masks, a[4 * j], a[4 * j + 1]);
          bytes_of(kw[2 * gi + 1][j], masks, a[4 * j + 2], a[4 * j + 3]);
        }
        if constexpr (WPT == 4) tmem_st_rows4(tm_k + quad + (uint32_t(16 * gi) << 16), a);
        else tmem_st_rows2(tm_k + quad + (uint32_t(16 * gi) << 16), a);
      }
    };
    uint32_t n = 0;  // tiles done
    while (left > 0) {
      // -------------------------------------------------------------- a unit's tiles
      const int t_lo = cur.s.tile0 + cur.tile;
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      const int lo = part.prefix ? 0 : part.shared, hi = cur.s.len;  // tokens of this part
      // ---- the rows' queries: a warp takes rows warp, warp + 4, ...; lane l
      // holds dims E l .. E l + E - 1, E = d / 32
      {
        constexpr int E = D / 32;
        for (int r = warp; r < RP; r += 4) {
          const Row row = row_of(part, cur.s, cur.j * RP + r);
          float x[E];
          if (row.tok >= 0) {
            const T* src = q + row.tok * ld_q + int64_t(cur.g * part.G + row.hh) * D + E * lane;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float2 f = fp8::to_f2<T>(__ldcg(reinterpret_cast<const unsigned int*>(src + e)));
              x[e] = f.x;
              x[e + 1] = f.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
          }
#pragma unroll
          for (int s = 1; s < E; s <<= 1)
#pragma unroll
            for (int e = 0; e < E; ++e)
              if ((e & s) == 0) {
                const float a = x[e], b = x[e + s];
                x[e] = a + b;
                x[e + s] = a - b;
              }
          float amax = 0.f;
#pragma unroll
          for (int s = 1; s < 32; s <<= 1)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float other = __shfl_xor_sync(0xffffffffu, x[e], s);
              x[e] = (lane & s) ? other - x[e] : x[e] + other;
            }
#pragma unroll
          for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
          // pieces of x * 256 / amax: the first of up to 256, the others' sixteenths
          amax = fmaxf(amax, kLeast);
          const float up = 256.0f / amax;
          uint32_t c[E / 2][3];
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            float a = x[e] * up, b = x[e + 1] * up;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              c[e / 2][k] = fp8::cvt_e4m3x2(make_float2(a, b));
              const float2 f = h2_to_f2(h2_of_e4m3x2(c[e / 2][k]));
              const float w = k == 0 ? 1.f : k == 1 ? 0.0625f : 0.00390625f;
              sum += (f.x + f.y) * w;
              a = (a - f.x) * 16.f;
              b = (b - f.y) * 16.f;
            }
          }
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          // dim 8 w + 2 byte + h lies in byte 4 (8 (w % WPT) + 2 (w / WPT) + h) + byte
          const int w = E * lane / 8;
          const uint32_t col = 8u * (w % WPT) + 2u * (w / WPT);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t n = k * RP + r;
            auto put = [&](uint32_t pos) { return sma + C::OFF_Q + n * 128 + ((((pos >> 4) ^ n) & 7) << 4) + (pos & 15); };
            if constexpr (E == 4) {
              const uint32_t v = c[0][k] | (c[1][k] << 16);  // dims 0 1 2 3 of this lane
              const uint32_t ev = (v & 0xFF) | ((v >> 8) & 0xFF00), od = ((v >> 8) & 0xFF) | ((v >> 16) & 0xFF00);
              const uint32_t pos = 4 * col + 2 * (lane & 1);
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(put(pos)), "h"(uint16_t(ev)) : "memory");
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(put(pos + 4)), "h"(uint16_t(od)) : "memory");
            } else {
              const uint32_t pos = 4 * col + (lane & 3);
              asm volatile("st.shared.b8 [%0], %1;" ::"r"(put(pos)), "r"(c[0][k] & 0xFF) : "memory");
              asm volatile("st.shared.b8 [%0], %1;" ::"r"(put(pos + 4)), "r"(c[0][k] >> 8) : "memory");
            }
          }
          if (lane == 0) {
            reinterpret_cast<float*>(rowf)[r] = 2.0f * amax * qscale;  // 2^9 of the codes, 1 / 256 of the pieces
            reinterpret_cast<float*>(rowo)[r] = sum * (-8.0f / 512.0f);
            reinterpret_cast<int*>(rowe)[r] = row.end;
            reinterpret_cast<float*>(mtop)[r] = kNone;
          }
        }
      }
      to_async_proxy();
      put_keys(n);
      tc_wait_st();
      tc_before();
      __syncthreads();  // the fifth warp issues the products of the first scores

      float2 l[RP / 2], z[RP / 2];
#pragma unroll
      for (int r = 0; r < RP / 2; ++r) l[r] = z[r] = make_float2(0.f, 0.f);

      for (int it = 0; it < nt; ++it, ++n) {
        // ---- the next tile's keys, once this one's scores are there
        wait(bar_s, n & 1, false);
        tc_after();
        if (it + 1 < nt) put_keys(n + 1);
        // ---- values, once the products of the tile before have read theirs
        uint32_t vw[4][WPT];
        const uint32_t raw = sma + C::OFF_RV + (n & 1) * C::STAGE_V;
        wait(bar_v + (n & 1), (n >> 1) & 1, true);
        words(raw, vw);
        uint32_t k_half, v_half;
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(k_half) : "r"(raw + C::CODES + 2 * tid));
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v_half) : "r"(raw + C::CODES + 2 * TILE + 2 * tid));
        v_half = min(v_half & 0x7FFFu, 0x7BFFu) | (v_half & 0x8000u);  // what is not finite counts as 65504: times a probability of 0 it is 0
        int tok = (t_lo + it) * TILE + tid;
        const bool absent = !((there[n & 1] >> (tid >> 4)) & 1) || tok < lo || tok >= hi;
        if (it > 0) wait(bar_o, (n - 1) & 1, false);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b[2 * WPT];
#pragma unroll
          for (int j = 0; j < WPT; ++j) bytes_of(vw[i][j], masks, b[2 * j], b[2 * j + 1]);
#pragma unroll
          for (int h = 0; h < WPT / 2; ++h)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(v_dst[h] + 1024u * i), "r"(b[4 * h]), "r"(b[4 * h + 1]),
                         "r"(b[4 * h + 2]), "r"(b[4 * h + 3])
                         : "memory");
        }
        // ---- scores of this thread's token, two rows at a time
        uint32_t v[NC];
#pragma unroll
        for (int c = 0; c < NC; c += 16) tmem_ld16(tm_s + quad + c, v + c);
        const float2 scales = make_float2(__half2float(__ushort_as_half(uint16_t(k_half))),
                                          absent ? 0.f : __half2float(__ushort_as_half(uint16_t(v_half))));
        const float lv = lg2(fmaxf(scales.y, 5.9604645e-8f));
        if (absent) tok = 0x7fffffff;
        tc_wait_ld();
        float2 s[RP / 2];
        bool above = false;
#pragma unroll
        for (int r = 0; r < RP / 2; ++r) {
          auto two = [&](int c) { return make_float2(__uint_as_float(v[c + 2 * r]), __uint_as_float(v[c + 2 * r + 1])); };
          const float2 f = rowf[r], o = rowo[r];
          const float2 x = __fadd2_rn(__ffma2_rn(two(RP), make_float2(0.0625f, 0.0625f), two(0)),
                                      __ffma2_rn(two(2 * RP), make_float2(0.00390625f, 0.00390625f), o));
          s[r] = __fmul2_rn(x, __fmul2_rn(f, make_float2(scales.x, scales.x)));
          const int2 end = rowe[r];
          if (tok >= end.x) s[r].x = -INFINITY;
          if (tok >= end.y) s[r].y = -INFINITY;
          const float2 y = __fadd2_rn(s[r], make_float2(lv, lv)), m = mtop[r];  // mtop = mref + 8
          above |= y.x > m.x || y.y > m.y;
        }
        float2 p[RP / 2], w[RP / 2];
        auto probabilities = [&]() {
          uint32_t pw[3][RP / 4];
#pragma unroll
          for (int r = 0; r < RP / 2; r += 2) {
            uint32_t c[2][3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 m = mtop[r + h], y = __fadd2_rn(s[r + h], make_float2(8.0f - m.x, 8.0f - m.y));
              w[r + h] = make_float2(ex2(y.x), ex2(y.y));
              const float2 x = __fmul2_rn(w[r + h], make_float2(scales.y, scales.y));
              const uint32_t rounded = h2_of_f2(x.x, x.y);
              // what the products take: the pieces' sum, exact in fp32
              p[r + h] = __ffma2_rn(h2_to_f2(pieces_of(rounded, c[h])), make_float2(-0.00390625f, -0.00390625f), h2_to_f2(rounded));
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) pw[k][r / 2] = c[0][k] | (c[1][k] << 16);
          }
          uint32_t words[NC / 4];
#pragma unroll
          for (int i = 0; i < NC / 4; ++i) words[i] = i < 3 * RP / 4 ? pw[i / (RP / 4)][i % (RP / 4)] : 0u;
#pragma unroll
          for (int i = 0; i < NC / 16; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p_dst + 16u * TILE * i), "r"(words[4 * i]),
                         "r"(words[4 * i + 1]), "r"(words[4 * i + 2]), "r"(words[4 * i + 3])
                         : "memory");
          to_async_proxy();
        };
        bool raise = it == 0;  // a unit's first tile always raises
        if (!raise) {
          probabilities();
          if (it + 1 < nt) tc_wait_st();
          tc_before();
          raise = __syncthreads_or(above);
        }
        if (raise) {
          // ---- raise the references that some score exceeds; sums and outputs so far follow
          float* mt = reinterpret_cast<float*>(mtop);
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            float x = (r & 1 ? s[r / 2].y : s[r / 2].x) + lv;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (lane == 0) xch[warp * RP + r] = x;
          }
          __syncthreads();
          float al[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float mo = mt[r], x = fmaxf(fmaxf(xch[r], xch[RP + r]), fmaxf(xch[2 * RP + r], xch[3 * RP + r]));
            al[r] = x > mo ? ex2(mo - 3.0f - x) : 1.0f;
            (r & 1 ? l[r / 2].y : l[r / 2].x) *= al[r];
            (r & 1 ? z[r / 2].y : z[r / 2].x) *= al[r];
          }
          if (it > 0) {
            uint32_t o[NC];
            tc_after();
#pragma unroll
            for (int c = 0; c < NC; c += 16) tmem_ld16(tm_o + quad + c, o + c);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
              for (int r = 0; r < RP; ++r) o[k * RP + r] = __float_as_uint(__uint_as_float(o[k * RP + r]) * al[r]);
#pragma unroll
            for (int c = 0; c < NC; c += 16) tmem_st16(tm_o + quad + c, o + c);
            tc_wait_st();
          }
          __syncthreads();
          if (tid < RP) {
            const float x = fmaxf(fmaxf(xch[tid], xch[RP + tid]), fmaxf(xch[2 * RP + tid], xch[3 * RP + tid]));
            if (x > mt[tid]) mt[tid] = x + 3.0f;
          }
          __syncthreads();
          probabilities();
          if (it + 1 < nt) tc_wait_st();
          tc_before();
          __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < RP / 2; ++r) {
          l[r] = __fadd2_rn(l[r], w[r]);
          z[r] = __fadd2_rn(z[r], p[r]);
        }
      }

      // ---------------------------------------------------------------- the unit's state
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        float lr = r & 1 ? l[r / 2].y : l[r / 2].x, zr = r & 1 ? z[r / 2].y : z[r / 2].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          lr += __shfl_xor_sync(0xffffffffu, lr, o);
          zr += __shfl_xor_sync(0xffffffffu, zr, o);
        }
        if (lane == 0) {
          xch[warp * 2 * RP + r] = lr;
          xch[warp * 2 * RP + RP + r] = zr;
        }
      }
      __syncthreads();
      wait(bar_o, (n - 1) & 1, false);
      tc_after();
      uint32_t v[NC];
#pragma unroll
      for (int c = 0; c < NC; c += 16) tmem_ld16(tm_o + quad + c, v + c);
      tc_wait_ld();
      const int J = (cur.s.rows + RP - 1) / RP;
      const int64_t unit = unit_base(cur.s.tok0, part.prefix ? 0 : cur.b, part.G, part.Hkv, RP) + int64_t(cur.g) * J + cur.j;
      const int64_t dst = (unit + blockIdx.x) * RP;
      const int dim = (tid & ~7) + 2 * (tid & 3) + ((tid >> 2) & 1);  // of byte tid of a token's row
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float zz = (xch[RP + r] + xch[3 * RP + r]) + (xch[5 * RP + r] + xch[7 * RP + r]);
        const float o = fmaf(__uint_as_float(v[2 * RP + r]), 0.00390625f,
                             fmaf(__uint_as_float(v[RP + r]), 0.0625f, __uint_as_float(v[r])));
        if (tid < D) ws.o[(dst + r) * D + dim] = fmaf(o, 512.0f, -8.0f * zz);
      }
      if (tid < RP) {
        const float ll = (xch[tid] + xch[2 * RP + tid]) + (xch[4 * RP + tid] + xch[6 * RP + tid]);
        *reinterpret_cast<float2*>(ws.ml + (dst + tid) * 2) = make_float2(reinterpret_cast<float*>(mtop)[tid] - 8.0f, ll);
      }
      if (tid == 0) {
        if (cur.tile == 0) ws.span[2 * unit] = blockIdx.x;
        if (cur.tile + nt == cur.tiles) ws.span[2 * unit + 1] = blockIdx.x;
      }
      tc_before();
      left -= nt;
      __syncthreads();  // the exchange, the rows and the references are read
      if (left > 0) cur = told_cursor(next);
      if (left > 0 && cur.tiles == 0) break;
    }
  }
  if (behind) fp8::wait_for_previous();  // the prefix part is over before this part is
  __syncthreads();
  if (warp == FEED) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::COLS) : "memory");
  }
}

}  // namespace few

// ===================================================================== many
// Up to 128 rows of a unit, rows as the MMA's M: a row's scores are one
// thread pair's, its probabilities go back to tensor memory as the A operand
// of O += P V without a word between lanes.  The warps of a CTA (one on an SM):
//   warp 0      feeder: pages, copies of packed tiles, three ahead
//   warp 1      MMA issuer
//   warps 2-5   converters: key codes to e4m3 bytes (bytes_of, rows of a
//               swizzled K-major operand); values to fp16 code * scale, token
//               after token (the B operand with N running fastest: no transpose)
//   warps 6-21  softmax, four to a lane quadrant, each a quarter of its rows:
//               queries rotated and split into e4m3 pieces at a unit's start,
//               scores to probabilities, outputs at its end
//   warp 22     the next unit: which it is, and its queries
//   warp 23     key scales
// Tensor memory: the three pieces of the queries (A operand of S), two score
// buffers, in which fp16 probabilities take the place of the scores that they
// were made from, and O.  S(n + 1) runs while the softmax works on S(n).
//
// A score is (S - off) ks f with off = 8 sum q~ (the codes' offset) and f the
// row's factor; the references are raised as in `few`, without the value
// scales, which the values carry here.
//
// What bounds it: the hand-overs between these roles.  A tile takes some 2800
// clocks.  The MMAs need 1350 of them (12 of 128 x 128 x 32 for S and 8 of
// 128 x 128 x 16 for P V, each of the two after what it waits for), the
// converters 1600 busy and four waits, the softmax 2100 busy and two waits.  256
// sequences sharing 32768 tokens take 19 % less without the softmax, 9 % without
// the conversion, and nothing less without the exponentials or a third of the MMAs.
// Two score buffers are what tensor memory has room for.  A unit's start and end
// cost some 14000 clocks more, of which the tensor cores wait for 8000: queries
// rotated and split (e4m3 conversions run at a few lanes a clock), outputs
// rotated back.  256 sharing 32768: 198 us, 697 TFLOP/s of the formula's
// products; 4 x 2048 tokens: 344 us, 400 TFLOP/s.
namespace many {

constexpr uint32_t kLoud = 0x6FFF;  // 8188 in fp16
constexpr int NT = 768, ROWS = 128, NCW = 4, NSW = 16, SP = 3, UNIT_READERS = 3 + NCW + NSW;
constexpr uint32_t COL_Q = 0, COL_S = 128, COL_O = 384;  // S buffer b at COL_S + 128 b

template <int D>
struct Cfg {
  static constexpr int WPT = D / 32;
  static constexpr int CODES = TILE * D / 2;
  static constexpr int STAGE = 2 * CODES + 4 * TILE;   // packed keys, values, key scales, value scales
  static constexpr int ATOM = TILE * 128;              // 128 bytes of every token
  static constexpr int VBYTES = ATOM * (D / 64);       // a converted value tile
  static constexpr int OFF_K = 0;                      // converted keys, two tiles
  static constexpr int OFF_V = OFF_K + 2 * ATOM;       // converted values, two tiles
  static constexpr int OFF_Q = OFF_V + 2 * VBYTES;     // the unit's queries, 16-byte chunks swizzled
  static constexpr int OFF_RAW = OFF_Q + ROWS * D * 2;
  static constexpr int OFF_KS = OFF_RAW + SP * STAGE;  // float [2][TILE] key scales of the score buffers
  static constexpr int OFF_X = OFF_KS + 2 * TILE * 4;  // float [4][ROWS] exchange of a row's quarters, three times; at first find_start's words
  static constexpr int OFF_CUR = OFF_X + 12 * ROWS * 4; // cursors of four units
  static constexpr int OFF_BAR = OFF_CUR + 256;
  static constexpr int NBAR = 2 * SP + 4 + 4 + 3 + 8 + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 64;  // 48 of them used
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Instruction descriptor of kind::f16, fp16 x fp16 to fp32, M = 128, B with N running fastest.
__host__ __device__ constexpr uint32_t idesc16(int n) { return (1u << 4) | (1u << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24); }
__device__ __forceinline__ void mma16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)));
}
// 128-byte swizzle, N (or M) running fastest: 64 fp16 of 8 tokens are 1024
// bytes, further tokens `sbo`, further columns `lbo` bytes on.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
__device__ __forceinline__ void tmem_st4(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Sequence-row, tokens and range of a unit's k-th tile: the tiles of the
// prefix come first where a part has both.
struct Span {
  int row, t0, lo, hi;
};
__device__ __forceinline__ Span tile_at(const Part& p, const Cursor& c, int k) {
  if (p.prefix) return {0, k * TILE, 0, c.s.len};
  if (p.whole) {
    const int np = (min(c.s.len, p.shared) + TILE - 1) / TILE;
    if (k < np) return {0, k * TILE, 0, min(c.s.len, p.shared)};
    k -= np;
  }
  return {c.b, (c.s.tile0 + k) * TILE, p.shared, c.s.len};
}
// Sums and differences over spans 1 .. N / 2 of N registers.
template <int N>
__device__ __forceinline__ void hadamard_regs(float2* x) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) x[i] = make_float2(x[i].x + x[i].y, x[i].x - x[i].y);
#pragma unroll
  for (int s = 1; s < N / 2; s <<= 1)
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      if ((i & s) == 0) {
        const float2 a = x[i], b = x[i + s];
        x[i] = __fadd2_rn(a, b);
        x[i + s] = __ffma2_rn(b, make_float2(-1.f, -1.f), a);
      }
}

struct Values {  // constants of the values' conversion, like Masks
  uint32_t mask, flip;      // 0x000F000F, 0x64086408: 1024 + u of the lowest nibble
  uint32_t mask16, flip16;  // 0x00F000F0, 0x64806480: 1024 + 16 u of the next
};

// direct: units that a CTA works on alone are written to out; of the others
// (the start of one and the end of another, two a CTA) slot 2 w + 0 holds the
// state of one that an earlier CTA began, 2 w + 1 of one that this CTA began,
// and todo [w] names the unit of another CTA's that CTA w ended.
template <typename T, int D>
__global__ void __launch_bounds__(NT, 1)
many_kernel(const T* __restrict__ q, int64_t ld_q, const uint8_t* __restrict__ k_q, const __half* __restrict__ k_s,
            const uint8_t* __restrict__ v_q, const __half* __restrict__ v_s, Part part, float qscale, Space ws, int4* todo,
            int unrotate, T* __restrict__ out, int64_t ld_out, Masks masks, Values vals) {
  using C = Cfg<D>;
  constexpr int WPT = C::WPT, E = D / 4;  // E: elements of a thread's quarter of a row
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t sma = smem_u32(sm);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* raw_empty = raw_full + SP;
  uint64_t* k_full = raw_empty + SP;  // [2] each
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* unit_full = v_empty + 2;   // cursor and queries
  uint64_t* unit_empty = unit_full + 1;
  uint64_t* q_full = unit_empty + 1;
  uint64_t* s_full = q_full + 1;  // [2] each
  uint64_t* p_full = s_full + 2;
  uint64_t* ks_full = p_full + 2;
  uint64_t* ks_empty = ks_full + 2;
  uint64_t* o_done = ks_empty + 2;     // one phase a tile
  uint64_t* unit_done = o_done + 1;    // and a unit
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MISC);
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  volatile int* there = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 8);      // [SP] groups of 16 tokens that a packed tile has
  volatile int* there_s = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 24);   // [2] of the score buffers; 0x100: all tokens are there
  volatile int64_t* each = reinterpret_cast<volatile int64_t*>(sm + C::OFF_MISC + 32);  // tiles of a CTA
  volatile uint8_t* eighth = sm + C::OFF_MISC + 40;  // [2 value tiles][4] whether values of 32 tokens are an eighth
  float* ksf = reinterpret_cast<float*>(sm + C::OFF_KS);
  float* xch = reinterpret_cast<float*>(sm + C::OFF_X);
  int* cursors = reinterpret_cast<int*>(sm + C::OFF_CUR);  // [4][16]

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < SP; ++i) {
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, NCW + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, NCW);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, NCW);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, NSW);
      mbar_init(ks_full + i, 1);
      mbar_init(ks_empty + i, NSW);
    }
    mbar_init(unit_full, 33);  // each lane's copies, and the cursor
    mbar_init(unit_empty, UNIT_READERS);
    mbar_init(q_full, NSW);
    mbar_init(o_done, 1);
    mbar_init(unit_done, 1);
    *gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(const_cast<uint32_t*>(slot))),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  fp8::wait_for_previous();
  fp8::next_may_start();
  Cursor cur;
  int64_t per;
  int64_t left = find_start(part, cur, per, reinterpret_cast<int64_t*>(sm + C::OFF_X));
  if (tid == 0) {
    *each = per;  // (the softmax reads it behind barriers that follow this warp's copies)
    if (todo != nullptr) todo[blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  auto wait = [&](uint64_t* bar, uint32_t phase, bool copy = false) {
    bool ok = mbar_try_wait(bar, phase);
    for (int n = 0; !ok && n < kTries && (copy || !*gave_up); ++n) ok = mbar_try_wait(bar, phase);
    if (!ok) {
      *gave_up = 1;
      record_error(QUAROT_ERR_TIMEOUT);
    }
    __syncwarp();
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // the unit that the feeder published: waits for it and reads its cursor
  auto unit_at = [&](uint32_t u) {
    wait(unit_full, u & 1, true);
    return told_cursor(cursors + 16 * (u & 3));
  };

  if (warp == 0) {
    // ================================================================ feeder
    const int shift = (part.t.ps & (part.t.ps - 1)) == 0 ? __ffs(part.t.ps) - 1 : -1;
    uint32_t n = 0;
    for (uint32_t u = 0; left > 0; ++u) {
      cur = unit_at(u);
      arrive(unit_empty);
      if (cur.tiles == 0) break;
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      left -= nt;
      for (int k = 0; k < nt; ++k, ++n) {
        const Span sp = tile_at(part, cur, cur.tile + k);
        const int tb = sp.t0 + 16 * (lane & 7);
        const int index = shift >= 0 ? tb >> shift : tb / part.t.ps;
        int row = -1;
        if (lane < 8 && tb < sp.hi && tb + 16 > sp.lo) {
          const int page = index < part.t.max_pages ? __ldcg(part.t.table + int64_t(sp.row) * part.t.max_pages + index) : -1;
          if (unsigned(page) < unsigned(part.t.n_pages))
            row = (page * part.Hkv + cur.g) * (part.t.ps >> 4) + ((tb - index * part.t.ps) >> 4);
          else
            record_error(QUAROT_ERR_INVALID_ARG);
        }
        const uint32_t st = n % SP;
        if (n >= SP) wait(raw_empty + st, (n / SP - 1) & 1);
        const unsigned valid = __ballot_sync(0xffffffffu, row >= 0) & 0xFF;
        const int before = __shfl_up_sync(0xffffffffu, row, 1);
        unsigned starts = __ballot_sync(0xffffffffu, row >= 0 && (lane == 0 || before < 0 || row != before + 1)) & 0xFF;
        const unsigned ends = (starts | ~valid) & 0x1FF;
        const uint32_t to = sma + C::OFF_RAW + st * C::STAGE;
        constexpr uint32_t GROUP = 16 * D / 2;
        if (elect_one()) {
          to_async_proxy();
          there[st] = int(valid);
          mbar_arrive_expect_tx(raw_full + st, __popc(valid) * (2 * GROUP + 64));
        }
        while (starts) {
          const int a = __ffs(starts) - 1;
          starts &= starts - 1;
          const int len = __ffs(ends >> (a + 1));
          const int64_t r = __shfl_sync(0xffffffffu, row, a);
          if (elect_one()) {
            bulk_copy(to + a * GROUP, k_q + r * GROUP, len * GROUP, raw_full + st);
            bulk_copy(to + C::CODES + a * GROUP, v_q + r * GROUP, len * GROUP, raw_full + st);
            bulk_copy(to + 2 * C::CODES + a * 32, k_s + r * 16, len * 32, raw_full + st);
            bulk_copy(to + 2 * C::CODES + 2 * TILE + a * 32, v_s + r * 16, len * 32, raw_full + st);
          }
        }
        __syncwarp();
      }
    }
    for (uint32_t m = n < SP ? 0 : n - SP; m < n; ++m) wait(raw_full + m % SP, (m / SP) & 1, true);
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    uint32_t n = 0, units = 0;
    for (uint32_t u = 0; left > 0; ++u) {
      cur = unit_at(u);
      arrive(unit_empty);
      if (cur.tiles == 0) break;
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      left -= nt;
      ++units;
      auto issue_scores = [&](uint32_t m) {
        const uint32_t d = tmem + COL_S + 128 * (m & 1);
        const uint64_t kd = desc_sw128(sma + C::OFF_K + (m & 1) * C::ATOM, 1024);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma8_ts(d, tmem + COL_Q + p * (D / 4) + 8 * kk, kd + 2 * kk, idesc8(TILE, false, false), p + kk > 0);
        mma_commit(s_full + (m & 1));
        mma_commit(k_empty + (m & 1));
      };
      // the queries are there while the unit before may still be at its last products: these read the buffer's place
      wait(q_full, u & 1);
      if (u > 0) wait(unit_done, (u - 1) & 1);
      wait(k_full + (n & 1), (n >> 1) & 1);
      tc_after();
      if (elect_one()) issue_scores(n);
      __syncwarp();
      for (int k = 0; k < nt; ++k, ++n) {
        if (k + 1 < nt) {
          // buffer (n + 1) % 2 holds P(n - 1), which O += P(n - 1) V has to have read
          wait(k_full + ((n + 1) & 1), ((n + 1) >> 1) & 1);
          if (n > 0) wait(o_done, (n - 1) & 1);
          tc_after();
          if (elect_one()) issue_scores(n + 1);
          __syncwarp();
        }
        wait(v_full + (n & 1), (n >> 1) & 1);
        wait(p_full + (n & 1), (n >> 1) & 1);
        tc_after();
        if (elect_one()) {
          const uint64_t vd = desc_sw128_mn(sma + C::OFF_V + (n & 1) * C::VBYTES, C::ATOM, 1024);
          auto products = [&](int kk, bool acc) {
            mma16_ts(tmem + COL_O, tmem + COL_S + 128 * (n & 1) + 32 * (kk >> 1) + 8 * (kk & 1), vd + 128 * kk, idesc16(D), acc);
          };
#pragma unroll
          for (int kk = 0; kk < TILE / 16; ++kk) products(kk, k > 0 || kk > 0);
          const uint32_t again = *reinterpret_cast<volatile uint32_t*>(const_cast<uint8_t*>(eighth) + 4 * (n & 1));
          if (again != 0) {  // values of an eighth eight times
#pragma unroll 1
            for (int kk = 0; kk < 7 * TILE / 16; ++kk)
              if ((again >> (8 * ((kk & 7) >> 1))) & 1) products(kk & 7, true);
          }
          mma_commit(o_done);
          mma_commit(v_empty + (n & 1));
          if (k + 1 == nt) mma_commit(unit_done);
        }
        __syncwarp();
      }
    }
    if (units > 0) wait(unit_done, (units - 1) & 1);
  } else if (warp < 2 + NCW) {
    // ================================================================ converters
    const int cw = warp - 2, r4 = lane >> 2, c4 = lane & 3;
    uint32_t n = 0;
    for (uint32_t u = 0; left > 0; ++u) {
      cur = unit_at(u);
      arrive(unit_empty);
      if (cur.tiles == 0) break;
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      left -= nt;
      for (int k = 0; k < nt; ++k, ++n) {
        const Span sp = tile_at(part, cur, cur.tile + k);
        const uint32_t st = n % SP, b = n & 1;
        wait(raw_full + st, (n / SP) & 1, true);
        const uint32_t raw = sma + C::OFF_RAW + st * C::STAGE + (32 * cw + r4) * (D / 2) + c4 * (4 * WPT);
        const int have = there[st];
        // words c4 WPT .. of tokens 32 cw + 8 i + r4
        uint32_t w[4][WPT];
        auto words = [&](uint32_t from) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = from + 8 * (D / 2) * i;
            if constexpr (WPT == 4)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]) : "r"(at));
            else
              asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(at));
          }
        };
        // ---- keys
        words(raw);
        if (n > 1) wait(k_empty + b, ((n >> 1) - 1) & 1);
        const uint32_t k_row = sma + C::OFF_K + b * C::ATOM + (32 * cw + r4) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[2 * WPT];
#pragma unroll
          for (int j = 0; j < WPT; ++j) bytes_of(w[i][j], masks, o[2 * j], o[2 * j + 1]);
#pragma unroll
          for (int h = 0; h < WPT / 2; ++h)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(k_row + 1024 * i + ((((WPT / 2) * c4 + h) ^ r4) << 4)),
                         "r"(o[4 * h]), "r"(o[4 * h + 1]), "r"(o[4 * h + 2]), "r"(o[4 * h + 3])
                         : "memory");
        }
        to_async_proxy();
        arrive(k_full + b);
        uint32_t half;
        const uint32_t scales = sma + C::OFF_RAW + st * C::STAGE + 2 * C::CODES;
        // ---- values: fp16 code * scale, pairs (k, k + 4) of a word's dims; 0 where the part has no token
        // (4 words: lanes of the two halves of a token change their pairs, to store different chunks at a time)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = raw + C::CODES + 8 * (D / 2) * i, first = WPT == 4 ? 4 * (c4 & 2) : 0;
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(at + first));
          if constexpr (WPT == 4) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][2]), "=r"(w[i][3]) : "r"(at + (first ^ 8)));
        }
        uint32_t vs2[4];
        bool loud = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 32 * cw + 8 * i + r4;
          asm volatile("ld.shared.u16 %0, [%1];" : "=r"(half) : "r"(scales + 2 * TILE + 2 * t));
          const bool in = sp.t0 + t >= sp.lo && sp.t0 + t < sp.hi && ((have >> (t >> 4)) & 1);
          half = in ? min(half & 0x7FFFu, 0x7BFFu) | (half & 0x8000u) : 0u;  // what is not finite counts as 65504
          loud |= (half & 0x7FFFu) > kLoud;
          vs2[i] = half | (half << 16);
        }
        // With a scale above 8188 a code times it could pass fp16's largest, and products have to stay finite for rows that
        // do not see the token too: these 32 tokens' values are an eighth then (to 2^-25), and their products are added eight
        // times.  (Eight times the probabilities instead: the flag comes too late, or holds the keys up; 4 x 2048 tokens 353 us
        // and more, this way 345, scales cut off at 8188 340.)
        const bool any = __any_sync(0xffffffffu, loud);
        if (any) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vs2[i] = hmul2(vs2[i], 0x30003000u);
        }
        arrive(raw_empty + st);
        if (n > 1) wait(v_empty + b, ((n >> 1) - 1) & 1);
        if (lane == 0) eighth[4 * b + cw] = any;
        const uint32_t v_row = sma + C::OFF_V + b * C::VBYTES + (32 * cw + r4) * 128 + (WPT == 4 ? (c4 >> 1) * C::ATOM : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int j = 0; j < WPT; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = hmul2(e & 1 ? hfma2(((w[i][j] >> (4 * (e & 2))) & vals.mask16) ^ vals.flip16, 0x2C002C00u, 0xD480D480u)  // (1024 + 16 u) / 16 - 72
                                 : hadd2(((w[i][j] >> (4 * e)) & vals.mask) ^ vals.flip, 0xE408E408u),  // (1024 + u) - 1032
                           vs2[i]);
            const uint32_t chunk = WPT == 4 ? uint32_t(4 * (c4 & 1) + (j ^ (c4 & 2))) : uint32_t(2 * c4 + j);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(v_row + 1024 * i + ((chunk ^ r4) << 4)), "r"(o[0]),
                         "r"(o[1]), "r"(o[2]), "r"(o[3])
                         : "memory");
          }
        }
        to_async_proxy();
        arrive(v_full + b);
      }
    }
  } else if (warp == 3 + NCW + NSW) {
    // ================================================================ key scales
    uint32_t n = 0;
    for (uint32_t u = 0; left > 0; ++u) {
      cur = unit_at(u);
      arrive(unit_empty);
      if (cur.tiles == 0) break;
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      left -= nt;
      for (int k = 0; k < nt; ++k, ++n) {
        const Span sp = tile_at(part, cur, cur.tile + k);
        const uint32_t st = n % SP, b = n & 1;
        wait(raw_full + st, (n / SP) & 1, true);
        const int have = there[st], tok = sp.t0 + 4 * lane;
        uint2 h;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(h.x), "=r"(h.y) : "r"(sma + C::OFF_RAW + st * C::STAGE + 2 * C::CODES + 8 * lane));
        arrive(raw_empty + st);
        const float2 lo = h2_to_f2(h.x), hi = h2_to_f2(h.y);
        const float f[4] = {lo.x, lo.y, hi.x, hi.y};
        float e[4];  // 0 where the part has no token
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = tok + i >= sp.lo && tok + i < sp.hi && ((have >> (lane >> 2)) & 1) ? f[i] : 0.f;
        if (n > 1) wait(ks_empty + b, ((n >> 1) - 1) & 1);
        reinterpret_cast<float4*>(ksf + b * TILE)[lane] = make_float4(e[0], e[1], e[2], e[3]);
        if (lane == 0) there_s[b] = have | (have == 0xFF && sp.t0 >= sp.lo && sp.t0 + TILE <= sp.hi ? 0x100 : 0);
        arrive(ks_full + b);
      }
    }
  } else if (warp == 2 + NCW + NSW) {
    // ================================================================ units
    for (uint32_t u = 0; left > 0; ++u) {
      if (u > 0) wait(unit_empty, (u - 1) & 1);
      if (lane == 0) tell_cursor(cur, cursors + 16 * (u & 3));
#pragma unroll 1
      for (int r = lane; r < ROWS; r += 32) {
        const int rr = cur.j * ROWS + r, i = rr / part.G;
        const bool in = rr < cur.s.rows && cur.tiles > 0;
        const T* src = q + (in ? (cur.s.tok0 + i) * ld_q + int64_t(cur.g * part.G + rr - i * part.G) * D : 0);
        const uint32_t dst = sma + C::OFF_Q + r * (2 * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + ((c ^ (r & 7)) << 4)), "l"(src + 8 * c),
                       "r"(in ? 16 : 0)
                       : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(unit_full)) : "memory");
      if (lane == 0) mbar_arrive(unit_full);
      if (cur.tiles == 0) break;  // the batch changed under the call: an empty unit ends every role
      const int nt = int(min(left, int64_t(cur.tiles - cur.tile)));
      left -= nt;
      cur.tile += nt;
      if (left > 0) next_unit(part, cur);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ================================================================ softmax
    const int qd = warp & 3, qq = (warp - 2 - NCW) >> 2;  // lane quadrant; quarter of the row's columns
    const int r = 32 * qd + lane;                         // row
    const uint32_t quad = tmem + (uint32_t(32 * qd) << 16);
    const int group = 1 + qd;  // named barrier of the four warps that share the rows
    auto group_any = [&](bool v) {
      uint32_t o;
      asm volatile(
          "{\n\t.reg .pred p, o;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred o, %2, 128, p;\n\tselp.u32 %0, 1, 0, o;\n\t}"
          : "=r"(o)
          : "r"(uint32_t(v)), "r"(group)
          : "memory");
      return o != 0;
    };
    // the values of the row's quarters, to all of them
    auto all_four = [&](float v, int which) {
      float* x = xch + 4 * ROWS * which + r;
      x[ROWS * qq] = v;
      asm volatile("bar.sync %0, 128;" ::"r"(group) : "memory");
      return make_float4(x[0], x[ROWS], x[2 * ROWS], x[3 * ROWS]);
    };
    // of the row's quarters a .. d what spans E and 2 E leave in this one
    auto spans = [&](float2 a, float2 b, float2 c, float2 d) {
      const float2 s1 = make_float2(qq & 1 ? -1.f : 1.f, qq & 1 ? -1.f : 1.f), s2 = make_float2(qq & 2 ? -1.f : 1.f, qq & 2 ? -1.f : 1.f);
      return __ffma2_rn(__ffma2_rn(d, s1, c), s2, __ffma2_rn(b, s1, a));
    };
    int rem = int(left);  // of this CTA's tiles
    uint32_t n = 0;
    float f = 0.f, off = 0.f;
    int tile = 0, end = 0, clear = 0, nt = 0;  // of the unit at work: what the row sees, tiles before one that not all rows of the warp see whole, tiles
    // The next unit: false where there is none.
    auto begin = [&](uint32_t u) -> bool {
      if (rem <= 0) return false;
      const Cursor cur = unit_at(u);
      tile = cur.tile;
      if (cur.tiles == 0) {
        arrive(unit_empty);
        rem = 0;
        return false;
      }
      nt = min(rem, cur.tiles - cur.tile);
      rem -= nt;
      end = row_of(part, cur.s, cur.j * ROWS + r).end;
      const int all_see = __reduce_min_sync(0xffffffffu, end);
      clear = all_see / TILE;
      if (!part.prefix) {
        const int np = part.whole ? (min(cur.s.len, part.shared) + TILE - 1) / TILE : 0;
        if (clear >= np) clear = np + max(clear - cur.s.tile0, 0);
      }
      // ---- the query: spans over the whole row, then this quarter's own
      {
        float2 x[E / 2];
        const uint32_t qr = sma + C::OFF_Q + r * (2 * D);
#pragma unroll
        for (int c = 0; c < E / 8; ++c) {
          uint32_t w[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[k][0]), "=r"(w[k][1]), "=r"(w[k][2]), "=r"(w[k][3])
                         : "r"(qr + (((c + k * (E / 8)) ^ (r & 7)) << 4)));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[4 * c + i] = spans(fp8::to_f2<T>(w[0][i]), fp8::to_f2<T>(w[1][i]), fp8::to_f2<T>(w[2][i]), fp8::to_f2<T>(w[3][i]));
        }
        arrive(unit_empty);
        hadamard_regs<E>(x);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) amax = max3(amax, fabsf(x[i].x), fabsf(x[i].y));
        float4 all = all_four(amax, 0);
        amax = fmaxf(fmaxf(all.x, all.y), fmaxf(all.z, all.w));
        // pieces of x * 256 / amax that add up to it: each of 4 bits, off by 2^-15 of the largest in the end
        amax = fmaxf(amax, kLeast);
        const float up = 256.0f / amax;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) x[i] = __fmul2_rn(x[i], make_float2(up, up));
        // their sum is what they were made from less what is left in the end
        float2 sums = make_float2(0.f, 0.f);
        uint32_t rest[E / 2];  // of pairs of even, pairs of odd dims; after the first piece at most 8, in fp16 off by 2^-17 of the largest
        uint32_t o[E / 4];
        const uint32_t to = quad + COL_Q + qq * (D / 16);
        auto put = [&](int p) {
          if constexpr (E == 32) tmem_st8(to + p * (D / 4), o);
          else tmem_st4(to + p * (D / 4), o);
        };
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {  // dims 4 i, 4 i + 1 and 4 i + 2, 4 i + 3: bytes of a word's dims are the even ones, then the odd ones
          const float2 a = x[2 * i], c = x[2 * i + 1];
          sums = __fadd2_rn(sums, __fadd2_rn(a, c));
          const uint32_t e0 = fp8::cvt_e4m3x2(make_float2(a.x, c.x)), e1 = fp8::cvt_e4m3x2(make_float2(a.y, c.y));
          const float2 ev = h2_to_f2(h2_of_e4m3x2(e0)), od = h2_to_f2(h2_of_e4m3x2(e1));
          rest[2 * i] = h2_of_f2(a.x - ev.x, c.x - ev.y);
          rest[2 * i + 1] = h2_of_f2(a.y - od.x, c.y - od.y);
          const int w = 2 * (i / 2);
          o[w] = i & 1 ? o[w] | (e0 << 16) : e0;
          o[w + 1] = i & 1 ? o[w + 1] | (e1 << 16) : e1;
        }
        put(0);
#pragma unroll
        for (int p = 1; p < 3; ++p) {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const uint32_t e = e4m3x2_of_h2(rest[i]);
            rest[i] = hsub2(rest[i], h2_of_e4m3x2(e));
            const int w = 2 * (i / 4) + (i & 1);
            o[w] = i & 2 ? o[w] | (e << 16) : e;
          }
          put(p);
        }
#pragma unroll
        for (int i = 1; i < E / 2; ++i) rest[0] = hadd2(rest[0], rest[i]);
        const float2 left_over = h2_to_f2(rest[0]);
        float sum = (sums.x + sums.y) - (left_over.x + left_over.y);
        tc_wait_st();
        tc_before();
        all = all_four(sum, 1);
        sum = (all.x + all.y) + (all.z + all.w);
        arrive(q_full);
        // of 2^9 of the codes and 1 / 256 of the pieces; never 0, so that a hidden score stays -inf
        f = fmaxf(2.0f * amax * qscale, 1e-37f);
        off = sum * (-8.0f / 512.0f);
      }
      return true;
    };
    bool more = begin(0);
    for (uint32_t u = 0; more; ++u) {
      // ---- tiles
      float m = kNone, l = 0.f;
      for (int k = 0; k < nt; ++k, ++n) {
        const uint32_t b = n & 1;
        wait(s_full + b, (n >> 1) & 1);
        wait(ks_full + b, (n >> 1) & 1);
        tc_after();
        const uint32_t s_t = quad + COL_S + 128 * b + 32 * qq;
        uint32_t v[32];
        tmem_ld16(s_t, v);
        tmem_ld16(s_t + 16, v + 16);
        const int have = there_s[b];
        const uint32_t kf = smem_u32(ksf + b * TILE + 32 * qq);
        tc_wait_ld();
        const float2 o2 = make_float2(off, off);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4 s4;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(s4.x), "=f"(s4.y), "=f"(s4.z), "=f"(s4.w) : "r"(kf + 4 * e));
          const float2 a = __fmul2_rn(__fadd2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), o2), make_float2(s4.x, s4.y));
          const float2 c = __fmul2_rn(__fadd2_rn(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), o2), make_float2(s4.z, s4.w));
          v[e] = __float_as_uint(a.x), v[e + 1] = __float_as_uint(a.y), v[e + 2] = __float_as_uint(c.x), v[e + 3] = __float_as_uint(c.y);
        }
        arrive(ks_empty + b);
        if (!(have & 0x100) || tile + k >= clear) {  // columns that this row does not see
          const Span sp = tile_at(part, told_cursor(cursors + 16 * (u & 3)), tile + k);
          const int lo = sp.lo - sp.t0 - 32 * qq, hi = min(end, sp.hi) - sp.t0 - 32 * qq, h2 = have >> (2 * qq);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < lo || e >= hi || !((h2 >> (e >> 4)) & 1)) v[e] = __float_as_uint(-INFINITY);
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(v[i]);
#pragma unroll
        for (int e = 4; e < 28; e += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], __uint_as_float(v[e + i]), __uint_as_float(v[e + 4 + i]));
        float top = fmaxf(max3(max3(mx[0], mx[1], mx[2]), mx[3], __uint_as_float(v[28])),
                          max3(__uint_as_float(v[29]), __uint_as_float(v[30]), __uint_as_float(v[31]))) * f;
        if (group_any(top > m + 8.0f)) {
          const float4 all = all_four(top, int(b));
          top = fmaxf(fmaxf(all.x, all.y), fmaxf(all.z, all.w));
          const bool raise = top > m + 8.0f;
          const float al = raise ? ex2(m - top) : 1.0f;
          if (raise) m = top;
          l *= al;
          if (k > 0) {  // outputs so far follow, once O += P(n - 1) V is over
            wait(o_done, (n - 1) & 1);
            tc_after();
            const uint32_t o_t = quad + COL_O + E * qq;
#pragma unroll 1
            for (int c = 0; c < E / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(o_t + 16 * c, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tmem_st16(o_t + 16 * c, o);
            }
          }
        }
        const float2 f2 = make_float2(f, f), m2 = make_float2(-m, -m);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 d = __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f2, m2);
          const float2 p = make_float2(ex2(d.x), ex2(d.y));
          ls[(e >> 1) & 1] = __fadd2_rn(ls[(e >> 1) & 1], p);
          v[e >> 1] = h2_of_f2(p.x, p.y);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tmem_st16(s_t, v);
        tc_wait_st();
        tc_before();
        arrive(p_full + b);
      }
      {
        const float4 all = all_four(l, 2);
        l = (all.x + all.y) + (all.z + all.w);
      }
      // The next unit's queries first: its scores can be computed while this one's outputs are written.
      const int was_nt = nt;
      more = begin(u + 1);
      // ---- the unit's outputs: a state, or, where this CTA had all of its tiles, the result
      // (S of the last tile was issued before O += P V of the one before it, and a wait for a parity cannot tell a
      // phase from the one two earlier: the unit's end has a barrier of its own)
      wait(unit_done, u & 1);
      tc_after();
      const Cursor was = told_cursor(cursors + 16 * (u & 3));
      const bool starts = was.tile == 0, ends = was.tile + was_nt == was.tiles;
      const bool direct = todo != nullptr && starts && ends;
      const uint32_t o_t = quad + COL_O;
      float2 x[E / 2];
      // 8 columns are a word's dims: column 2 k + e is dim k + 4 e
      auto in_order = [&](const uint32_t* a, int i) {
        auto dim = [&](int d) { return __uint_as_float(a[2 * (d & 3) + (d >> 2)]); };
        return make_float2(dim(2 * i), dim(2 * i + 1));
      };
#pragma unroll
      for (int c = 0; c < E / 8; ++c) {
        uint32_t a[4][8];
        if (direct && unrotate) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld8(o_t + E * k + 8 * c, a[k]);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) x[4 * c + i] = spans(in_order(a[0], i), in_order(a[1], i), in_order(a[2], i), in_order(a[3], i));
        } else {
          tmem_ld8(o_t + E * qq + 8 * c, a[0]);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) x[4 * c + i] = in_order(a[0], i);
        }
      }
      if (direct) {
        float sc = l > 0.f ? 1.0f / l : 0.f;
        if (unrotate) {
          hadamard_regs<E>(x);
          sc *= 1.0f / sqrtf(float(D));
        }
        const Row row = row_of(part, was.s, was.j * ROWS + r);
        if (row.tok >= 0) {
          T* dst = out + row.tok * ld_out + int64_t(was.g * part.G + row.hh) * D + E * qq;
#pragma unroll
          for (int c = 0; c < E / 16; ++c) {
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fp8::from_f2<T>(make_float2(x[8 * c + i].x * sc, x[8 * c + i].y * sc));
            if (((reinterpret_cast<uintptr_t>(out) | uintptr_t(ld_out * 2)) & 31) == 0) {  // whole sectors (4 x 2048 tokens: 346 us, 352 us without)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * c), "r"(o[0]), "r"(o[1]),
                           "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      } else {
        const int J = (was.s.rows + ROWS - 1) / ROWS;
        const int64_t unit = unit_base(was.s.tok0, part.prefix ? 0 : was.b, part.G, part.Hkv, ROWS) + int64_t(was.g) * J + was.j;
        const int64_t at = ((todo != nullptr ? 2 * int64_t(blockIdx.x) + (starts ? 1 : 0) : unit + blockIdx.x) * ROWS + r);
        float4* dst = reinterpret_cast<float4*>(ws.o + at * D + E * qq);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) dst[i] = make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
        if (qq == 0) *reinterpret_cast<float2*>(ws.ml + at * 2) = make_float2(m, l);
        if (warp == 2 + NCW && lane == 0) {
          if (todo == nullptr) {
            if (starts) ws.span[2 * unit] = blockIdx.x;
            if (ends) ws.span[2 * unit + 1] = blockIdx.x;
          } else if (ends) {
            todo[blockIdx.x] = make_int4(int((was.tile + *each - 1) / *each), was.b, was.g, was.j);  // CTAs before this one that had tiles of it
          }
        }
      }
      tc_before();
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// The units that several CTAs had a part in, each joined by 16 CTAs of 8 rows:
// todo [w] says how many CTAs before w had tiles of the unit that CTA w ended
// (0: it ended none that it did not begin), and which unit.  Tokens that see
// nothing, whose units may have had no tile at all, get their zeros here.
template <typename T, int D>
__global__ void __launch_bounds__(256)
join_units_kernel(Part part, Space ws, const int4* __restrict__ todo, int unrotate, T* __restrict__ out, int64_t ld_out) {
  __shared__ float x[8][D];
  fp8::wait_for_previous();
  for (int n = 8 * (blockIdx.y * gridDim.x + blockIdx.x) + (threadIdx.x >> 5); n < part.N; n += 8 * gridDim.x * gridDim.y) {
    const Place p = place_of(part.t, n);
    if (p.b >= 0 && min(p.pos + 1, part.t.max_pages * part.t.ps) <= 0)
      for (int e = 8 * (threadIdx.x & 31); e < part.G * part.Hkv * D; e += 256)
        *reinterpret_cast<uint4*>(out + n * ld_out + e) = make_uint4(0u, 0u, 0u, 0u);
  }
  const int w = blockIdx.x;
  const int4 t = __ldcg(todo + w);
  if (t.x <= 0) return;
  const int before = min(t.x, w);
  const Seq s = seq_of(part, t.y, false);
  const int r = 8 * blockIdx.y + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Row row = row_of(part, s, t.w * ROWS + r);
  constexpr int E = D / 32;
  float m = kNone, den = 0.f, num[E];
#pragma unroll
  for (int e = 0; e < E; ++e) num[e] = 0.f;
  for (int c = w - before; c <= w; ++c) {
    const int64_t at = (2 * int64_t(c) + (c == w - before ? 1 : 0)) * ROWS + r;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(ws.ml + at * 2));
    const float mx = fmaxf(m, ml.x), a = ex2(m - mx), f = ex2(ml.x - mx);
    m = mx;
    den = den * a + ml.y * f;
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] = num[e] * a + f * __ldcg(ws.o + at * D + lane + 32 * e);
  }
  const float inv = den > 0.f ? 1.0f / den : 0.f;
  float* y = x[threadIdx.x >> 5];
#pragma unroll
  for (int e = 0; e < E; ++e) num[e] *= inv;
  if (unrotate) {
    for (int span = 1; span < D; span <<= 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) y[lane + 32 * e] = num[e];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float other = y[(lane + 32 * e) ^ span];
        num[e] = ((lane + 32 * e) & span) ? other - num[e] : num[e] + other;
      }
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] *= 1.0f / sqrtf(float(D));
  }
  if (row.tok >= 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) out[row.tok * ld_out + int64_t(t.z * part.G + row.hh) * D + lane + 32 * e] = T(num[e]);
  }
}

}  // namespace many

// ------------------------------------------------------------------ join
// o = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i over the states of a row's unit
// of each part.
struct States {
  const float *ml[2], *o[2];  // of slot 0, prefix and own part
  const int* span[2];         // null: no state
  bool none;                  // the token is behind the last sequence
  __device__ __forceinline__ States(const Part& own, const Space& so, const Part& pre, const Space& sp, int n, int h, int D) {
    const Place pl = place_of(own.t, n);
    none = pl.b < 0;
    const int g = h / own.G;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Part& p = k == 0 ? pre : own;
      const Space& s = k == 0 ? sp : so;
      span[k] = nullptr;
      if (none || pl.pos < 0 || (k == 0 && p.shared == 0)) continue;
      const Seq q = seq_of(p, pl.b, false);
      const int rr = (n - q.tok0) * p.G + h - g * p.G;
      if (rr < 0 || rr >= q.rows) continue;
      const int j = rr / p.RP, J = (q.rows + p.RP - 1) / p.RP;
      if (tiles_of(p, q, j) == 0) continue;
      const int64_t unit = unit_base(q.tok0, p.prefix ? 0 : pl.b, p.G, p.Hkv, p.RP) + int64_t(g) * J + j;
      span[k] = s.span + 2 * unit;
      const int64_t at = unit * p.RP + rr - j * p.RP;
      ml[k] = s.ml + at * 2;
      o[k] = s.o + at * D;
    }
  }
  // first and last slot; as they are, unless the batch changed under the call
  __device__ __forceinline__ int2 slots(int k, const Space& s) const {
    const int2 w = __ldcg(reinterpret_cast<const int2*>(span[k]));
    return make_int2(min(max(w.x, 0), s.ctas - 1), min(w.y, s.ctas - 1));
  }
};

// Many rows, few states each: a warp a (token, query head), E = d / 32 dims a lane.
template <typename T, int D>
__global__ void __launch_bounds__(256)
join_rows_kernel(Part own, Space so, Part pre, Space sp, int Hq, int unrotate, T* __restrict__ out, int64_t ld_out) {
  constexpr int E = D / 32;
  const int64_t row = 8 * int64_t(blockIdx.x) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int n = int(row / Hq), h = int(row - int64_t(n) * Hq);
  // the batch was there before the parts' CTAs let this kernel start
  const States t(own, so, pre, sp, n, h, D);
  fp8::wait_for_previous();
  if (t.none || n >= own.N) return;
  float m = kNone, den = 0.f, num[E];
#pragma unroll
  for (int e = 0; e < E; ++e) num[e] = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (t.span[k] == nullptr) continue;
    const int64_t step = k == 0 ? pre.RP : own.RP;
    const int2 w = t.slots(k, k == 0 ? sp : so);
    for (int i0 = w.x; i0 <= w.y; i0 += 32) {
      const int c = min(w.y - i0 + 1, 32);
      float2 s = make_float2(kNone, 0.f);
      if (lane < c) s = __ldcg(reinterpret_cast<const float2*>(t.ml[k] + (i0 + lane) * step * 2));
      float mx = fmaxf(m, s.x);
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
      const float a = ex2(m - mx), f = ex2(s.x - mx);
      m = mx;
      float lw = f * s.y;
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, b);
      den = den * a + lw;
#pragma unroll
      for (int e = 0; e < E; ++e) num[e] *= a;
      const float* src = t.o[k] + i0 * step * D + E * lane;
#pragma unroll 4
      for (int i = 0; i < c; ++i) {
        const float b = __shfl_sync(0xffffffffu, f, i);
        if constexpr (E == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i * step * D));
          num[0] = fmaf(b, v.x, num[0]), num[1] = fmaf(b, v.y, num[1]), num[2] = fmaf(b, v.z, num[2]), num[3] = fmaf(b, v.w, num[3]);
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(src + i * step * D));
          num[0] = fmaf(b, v.x, num[0]), num[1] = fmaf(b, v.y, num[1]);
        }
      }
    }
  }
  float sc = den > 0.f ? 1.0f / den : 0.f;
  if (unrotate) {
#pragma unroll
    for (int s = 1; s < E; s <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((e & s) == 0) {
          const float a = num[e], b = num[e + s];
          num[e] = a + b;
          num[e + s] = a - b;
        }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, num[e], s);
        num[e] = (lane & s) ? other - num[e] : num[e] + other;
      }
    sc *= 1.0f / sqrtf(float(D));
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + n * ld_out + int64_t(h) * D + E * lane);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = fp8::from_f2<T>(make_float2(num[e] * sc, num[e + 1] * sc));
}

// Few rows, many states each: a CTA a (token, query head).  A thread adds 4
// dims of every fourth state, eight loads at once: with one tile a CTA (33
// states of a row, 1 x 4097 tokens) the round trips to L2 are what counts.
template <typename T, int D>
__global__ void __launch_bounds__(D)
join_kernel(Part own, Space so, Part pre, Space sp, int Hq, int unrotate, T* __restrict__ out, int64_t ld_out) {
  __shared__ float x[D], top[D / 32], low[D / 32];
  __shared__ float4 part4[4][D / 4];
  const int n = blockIdx.x / Hq, h = blockIdx.x % Hq, e = threadIdx.x;
  // the batch was there before the parts' CTAs let this kernel start
  const States t(own, so, pre, sp, n, h, D);
  fp8::wait_for_previous();
  if (t.none) return;
  float m = kNone, den = 0.f;
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d4 = e % (D / 4), grp = e / (D / 4);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (t.span[k] == nullptr) continue;
    const int64_t step = k == 0 ? pre.RP : own.RP;
    const int2 w = t.slots(k, k == 0 ? sp : so);
    for (int i0 = w.x; i0 <= w.y; i0 += D) {
      const int c = min(w.y - i0 + 1, D);
      float2 s = make_float2(kNone, 0.f);
      if (e < c) s = __ldcg(reinterpret_cast<const float2*>(t.ml[k] + (i0 + e) * step * 2));
      const float* src = t.o[k] + (i0 + grp) * step * D + 4 * d4;
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (grp + 4 * i < c) v[i] = __ldcg(reinterpret_cast<const float4*>(src + 4 * i * step * D));
      float mx = s.x;
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
      __syncthreads();
      if ((e & 31) == 0) top[e >> 5] = mx;
      __syncthreads();
      mx = m;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) mx = fmaxf(mx, top[b]);
      const float a = ex2(m - mx), f = ex2(s.x - mx);
      m = mx;
      x[e] = f;
      float lw = f * s.y;
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, b);
      if ((e & 31) == 0) low[e >> 5] = lw;
      __syncthreads();
      den *= a;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) den += low[b];
      num = make_float4(num.x * a, num.y * a, num.z * a, num.w * a);
      for (int i1 = 0; i1 < c; i1 += 32) {
        if (i1 > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i1 + grp + 4 * i < c) v[i] = __ldcg(reinterpret_cast<const float4*>(src + (i1 + 4 * i) * step * D));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i1 + grp + 4 * i < c) {
            const float b = x[i1 + grp + 4 * i];
            num = make_float4(fmaf(b, v[i].x, num.x), fmaf(b, v[i].y, num.y), fmaf(b, v[i].z, num.z), fmaf(b, v[i].w, num.w));
          }
      }
    }
  }
  __syncthreads();
  part4[grp][d4] = num;
  __syncthreads();
  const float* pf = reinterpret_cast<const float*>(part4);
  const float all = (pf[e] + pf[D + e]) + (pf[2 * D + e] + pf[3 * D + e]);
  float y = den > 0.f ? all / den : 0.f;
  if (unrotate) {
    for (int span2 = 1; span2 < D; span2 <<= 1) {
      __syncthreads();
      x[e] = y;
      __syncthreads();
      const float other = x[e ^ span2];
      y = (e & span2) ? other - y : y + other;
    }
    y *= 1.0f / sqrtf(float(D));
  }
  out[n * ld_out + int64_t(h) * D + e] = T(y);
}

// ------------------------------------------------------------------ host
// Which kernel a part gets, by the rows that see the same keys: up to 16, the
// tokens as the MMA's M (each 4, 8 or 16 rows read the keys once); above, the
// rows (64 sequences sharing 8000 tokens, 256 rows: 96 us and 46 us; 256 sharing
// 32768: 728 and 202 us; 4 x 2048 new tokens: 2195 and 346 us).  For 16
// sequences of 4096 tokens and 8 key heads, whatever the group, and heads of 64 alike:
//   rows a sequence and key head    20    32    64   128
//   tokens as M, 16 rows a pass    59.3  63.2 113.3 212.9 us
//   rows as M                      79.0  79.1  79.4  62.9 us
// so from 17 to some 40 rows (drafts) the first would still be faster.
// Sequences of more than 16 new rows are worked on whole, the shared tokens with
// their own: from 128 rows on the keys are read for every 128 of them anyway;
// below, each sequence reads the prefix for itself.
struct Plan {
  bool many;
  int RP, ctas;
  int64_t units;
};
inline Plan plan(int64_t rows, int64_t N, int64_t B, int64_t G, int64_t Hkv, int sms) {
  Plan p;
  p.many = rows > 16;
  p.RP = p.many ? many::ROWS : rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  p.ctas = sms * (p.many ? 1 : p.RP == 4 ? few::ctas_per_sm<4>() : p.RP == 8 ? few::ctas_per_sm<8>() : few::ctas_per_sm<16>());
  p.units = unit_count(N, B, G, Hkv, p.RP);
  return p;
}
struct Call {
  Plan own, pre;
  bool prefix;  // there is a part of its own for the shared tokens
  size_t bytes;
};
inline size_t whole_bytes(int64_t ctas, int64_t d) { return round256(size_t(ctas) * 16) + space_bytes(0, 2 * ctas, many::ROWS, d); }
inline bool plan_call(int64_t N, int64_t B, int64_t G, int64_t Hkv, int64_t d, int64_t max_q, int64_t shared, Call* c) {
  int sms = 0;
  if (!sm_count(&sms)) return false;
  c->own = plan((max_q < N ? max_q : N) * G, N, B, G, Hkv, sms);
  c->pre = plan(N * G, N, 1, G, Hkv, sms);
  c->prefix = shared > 0 && !c->own.many;
  c->bytes = c->own.many ? whole_bytes(c->own.ctas, d) : space_bytes(c->own.units, c->own.ctas, c->own.RP, d);
  if (c->prefix) c->bytes += space_bytes(c->pre.units, c->pre.ctas, c->pre.RP, d);
  return true;
}

}  // namespace paged
}  // namespace quarot

using namespace quarot;
using namespace quarot::paged;

extern "C" size_t quarot_paged_workspace_bytes(int64_t N, int64_t B, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_q,
                                               int64_t shared_len) {
  if (N <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128) || max_q <= 0 || shared_len < 0 ||
      N > kMaxTokens || B > kMaxTokens || Hq > kMaxHeads)
    return 0;
  Call c;
  return plan_call(N, B, Hq / Hkv, Hkv, d, max_q, shared_len, &c) ? c.bytes : 0;
}

template <typename T, int D>
static int attn_impl(const T* q, int64_t ld_q, const uint8_t* k_q, const __half* k_s, const uint8_t* v_q, const __half* v_s,
                     Part own, const Call& call, unsigned char* work, int Hq, float qscale, int unrotate, T* out,
                     int64_t ld_out, cudaStream_t st) {
  const Masks masks = {0x0F0F0F0Fu, 0x08080808u};
  auto few_part = [&](const Part& part, const Plan& plan, const Space& ws, int behind) -> int {
    auto go = [&](auto kern, size_t smem, AttrCache& attr) {
      if (!smem_attr_once(kern, int(smem), attr)) return int(QUAROT_ERR_LAUNCH);
      return fp8::launch_dependent(kern, dim3(unsigned(plan.ctas)), few::NT, smem, 1, st, q, ld_q, k_q, k_s, v_q, v_s, part,
                                   qscale, ws, behind, masks);
    };
    static AttrCache attr[3];
    if (plan.RP == 4) return go(few::few_kernel<T, 4, D>, few::Cfg<4, D>::SMEM, attr[0]);
    if (plan.RP == 8) return go(few::few_kernel<T, 8, D>, few::Cfg<8, D>::SMEM, attr[1]);
    return go(few::few_kernel<T, 16, D>, few::Cfg<16, D>::SMEM, attr[2]);
  };
  auto many_part = [&](const Part& part, const Plan& plan, const Space& ws, int4* todo) -> int {
    static AttrCache attr;
    auto kern = many::many_kernel<T, D>;
    if (!smem_attr_once(kern, many::Cfg<D>::SMEM, attr)) return QUAROT_ERR_LAUNCH;
    return fp8::launch_dependent(kern, dim3(unsigned(plan.ctas)), many::NT, many::Cfg<D>::SMEM, 1, st, q, ld_q, k_q, k_s, v_q, v_s,
                                 part, qscale, ws, todo, unrotate, out, ld_out, masks, many::Values{0x000F000Fu, 0x64086408u, 0x00F000F0u, 0x64806480u});
  };
  const Plan &po = call.own, &pp = call.pre;
  own.RP = po.RP;
  int rc = QUAROT_OK;
  if (po.many) {
    own.whole = 1;
    int4* todo = reinterpret_cast<int4*>(work);
    const Space ws = space_at(work + round256(size_t(po.ctas) * 16), 0, 2 * po.ctas, po.RP);
    if ((rc = many_part(own, po, ws, todo)) != QUAROT_OK) return rc;
    return fp8::launch_dependent(many::join_units_kernel<T, D>, dim3(unsigned(po.ctas), 16), 256, 0, 1, st, own, ws,
                                 static_cast<const int4*>(todo), unrotate, out, ld_out);
  }
  const Space so = space_at(work, po.units, po.ctas, po.RP);
  const Space sp = space_at(work + space_bytes(po.units, po.ctas, po.RP, D), pp.units, pp.ctas, pp.RP);
  Part pre = own;
  pre.prefix = 1;
  pre.RP = pp.RP;
  if (call.prefix && (rc = pp.many ? many_part(pre, pp, sp, nullptr) : few_part(pre, pp, sp, 0)) != QUAROT_OK) return rc;
  if ((rc = few_part(own, po, so, call.prefix)) != QUAROT_OK) return rc;
  // a warp a row and a CTA a row: 256 sequences sharing 32768 tokens (8192 rows) 202 and 232 us, 64 sharing 8000 (2048
  // rows) 46 and 52 us, 16 x 4096 (512) 27.5 and 26.7 us, 1 x 4097 (32) 15.3 and 10.1 us
  const unsigned rows = unsigned(own.N) * unsigned(Hq);
  if (rows > 1024)
    return fp8::launch_dependent(join_rows_kernel<T, D>, dim3((rows + 7) / 8), 256, 0, 1, st, own, so, pre, sp, Hq, unrotate, out,
                                 ld_out);
  return fp8::launch_dependent(join_kernel<T, D>, dim3(rows), D, 0, 1, st, own, so, pre, sp, Hq, unrotate, out, ld_out);
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
  if (Hq > kMaxHeads || N * Hq > 0x7fffffff) return QUAROT_ERR_UNSUPPORTED;
  if (N == 0 || B == 0) return QUAROT_OK;
  if ((rc = check_heads(q, ld_q, Hq, d)) != QUAROT_OK || (rc = check_heads(out, ld_out, Hq, d)) != QUAROT_OK) return rc;
  if ((rc = check_cache(k_q, k_s, v_q, v_s, page_table, lengths, cu_q, max_pages)) != QUAROT_OK) return rc;
  if (!workspace) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(workspace, 256)) return QUAROT_ERR_ALIGNMENT;
  Call call;
  const int64_t G = Hq / Hkv;
  if (!plan_call(N, B, G, Hkv, d, max_q, shared_len, &call)) return QUAROT_ERR_CUDA;
  if (ws_bytes < call.bytes) return QUAROT_ERR_INVALID_ARG;
  const Batch t = {page_table, lengths, cu_q, int(B), int(max_pages), int(n_pages), int(page_size)};
  const Part own = {t, int(N), int(G), int(Hkv), int(shared_len), 0, 0, 0};
  const float qscale = (sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(float(d))) * 1.4426950408889634f / sqrtf(float(d));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto* ksh = static_cast<const __half*>(k_s);
  auto* vsh = static_cast<const __half*>(v_s);
  auto typed = [&](auto* qp, auto* op) {
    using T = std::remove_pointer_t<decltype(op)>;
    unsigned char* work = static_cast<unsigned char*>(workspace);
    return d == 64 ? attn_impl<T, 64>(qp, ld_q, k_q, ksh, v_q, vsh, own, call, work, int(Hq), qscale, unrotate_out, op, ld_out, st)
                   : attn_impl<T, 128>(qp, ld_q, k_q, ksh, v_q, vsh, own, call, work, int(Hq), qscale, unrotate_out, op, ld_out, st);
  };
  if (dtype == QUAROT_FP16) return typed(static_cast<const __half*>(q), static_cast<__half*>(out));
  return typed(static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(out));
}
