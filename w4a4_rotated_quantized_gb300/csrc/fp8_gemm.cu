// quarot_fp8_gemm and quarot_fp8_gated_gemm: products of e4m3 codes with block
// scales on both operands, on the sm_103a tensor cores.
//
//   P[i, j] = sum_b a_scale[b, i] w_scale[j / 128, b] sum_{k in block b} a[i, k] w[j, k]
//   gemm:  y = P rounded to fp16 / bf16
//   gated: z = silu(P_gate) P_up in fp32, quantized to e4m3 with a scale for
//          each token and 128 columns
//
// The scales change every 128 of the depth, so no product can run through: the
// MMAs of one k-block of 128 write a fresh accumulator in tensor memory, and
// epilogue warps read it, scale it and add it to fp32 sums in registers while
// the MMAs of the next k-blocks fill other tensor-memory columns.
//
//   namespace wide    many tokens: persistent CTAs, 128 tokens x 256 weight rows
//                     (gated: 128 gate and 128 up rows) at a time
//   namespace narrow  few tokens: the weight rows are the MMA's M and the
//                     tokens its N, the depth split over a thread-block cluster
//
// Every wait is bounded (QUAROT_ERR_TIMEOUT in the device error word).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

// setmaxnreg needs whole-program compilation: this file is compiled without
// relocatable device code and has an error word of its own.
#define QUAROT_OWN_ERROR_WORD
#include "fp8.cuh"

namespace quarot {
namespace fp8 {
namespace gemm {

constexpr int BK = BLK;  // bytes of depth in a k-block: one 128-byte swizzled row

// ------------------------------------------------------------------ PTX
// Shared-memory matrix descriptor of a K-major operand, 128B swizzle: rows of
// 128 bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFF) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc(int m, int n) { return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24); }

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
// Arrives on the barrier when all earlier MMAs of this thread are done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 (16) columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
// One box at (x, y) into this CTA's shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// One box from this CTA's shared memory to (x, y), parts past the tensor's end left out.
__device__ __forceinline__ void tma_store(const CUtensorMap* tm, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
               "r"(bytes)
               : "memory");
}
// Arrival of the lanes that `pred` names, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, uint32_t pred) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 st;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar), "r"(pred)
               : "memory");
}
// One lane of a converged warp, in the form in which the compiler sees that it is one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded waits: a try_wait that finds nothing sleeps for 3.8 us, and kTries of
// them are the wait limit, about a second.  They are on every k-block's path, so they
// are a handful of instructions: the caller records an expired one where its
// loop ends.  wait_one is for one thread, wait_warp for a converged warp, whose
// loop the vote keeps uniform.
constexpr int kTries = 1 << 18;
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int n = 0; n < kTries; ++n)
    if (try_wait(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_one(bar, parity));
}
// Four bytes from global to this CTA's shared memory, asynchronously; the
// arrival on the barrier follows this thread's copies so far.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory words by address: through a pointer made from an integer (the
// aligned base) the compiler falls back to generic loads, far slower here.
__device__ __forceinline__ float lds(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 lds128_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, float2 a, float2 b) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y) : "memory");
}
__device__ __forceinline__ float lds_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// silu(g) u = g u / (1 + exp(-g)) of two columns, to a few 2^-23.  exp(n) = 2^h 2^l
// with h = rn(n log2 e) and 2^l = 1 + l ln 2 for the rounding error l of h (exact by
// fma); 2^h and 1 / x by the hardware approximations, 1 / x improved by a Newton step.
// n = -g is held to [-88, 88.5], where 2^h is finite.  Below g = -87.4 (1 + exp(n) >
// 2^126) 1 / x is flushed to zero and silu(g), under 1.1e-36, with it.
__device__ __forceinline__ float2 silu_mul(float2 g, float2 u) {
  constexpr float kL2E = 1.44269502f, kL2ELow = 1.92596299e-8f;  // log2 e in two parts
  constexpr float kLn2 = 0.693147181f;
  const float2 n = make_float2(fminf(fmaxf(-g.x, -88.f), 88.5f), fminf(fmaxf(-g.y, -88.f), 88.5f));
  const float2 nh = __fmul2_rn(n, make_float2(-kL2E, -kL2E));
  const float2 l = __ffma2_rn(n, make_float2(kL2ELow, kL2ELow), __ffma2_rn(n, make_float2(kL2E, kL2E), nh));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-nh.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-nh.y));
  const float2 one = make_float2(1.f, 1.f), m1 = make_float2(-1.f, -1.f);
  const float2 nd = __ffma2_rn(e, __ffma2_rn(l, make_float2(-kLn2, -kLn2), m1), m1);  // -(1 + exp(n))
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-nd.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-nd.y));
  r = __ffma2_rn(r, __ffma2_rn(nd, r, one), r);
  return __fmul2_rn(__fmul2_rn(g, r), u);
}

// ===================================================================== wide
// Persistent CTAs, one on an SM; a tile is 128 tokens x 256 weight rows (gated:
// 128 gate and 128 up rows).  A stage holds a k-block of both (48 KB).
//
//   warp 0      TMA producer
//   warp 1      TMEM allocator, MMA issuer
//   warp 2      scales, CH k-blocks to a hand-over
//   warps 4-11  epilogue: warp w reads TMEM lane quadrant w % 4, column half (w - 4) / 4,
//               and holds the sums of 32 tokens x 128 columns (128 registers a thread)
//
// Two accumulators of 256 tensor-memory columns: one k-block is read, scaled
// and summed while the MMAs of the next fill the other.
//
// What bounds it: a k-block's MMAs take 512 clocks, reading and summing its
// accumulator 375 (256 of them the fp32 sums), but the two are tied by a chain
// of hand-overs (MMAs done -> read -> buffer free -> next MMAs) that is long on
// latency.  So everything on that chain is short: one elected thread runs the
// MMA loop, barriers are this CTA's own (CTA pairs, whose MMAs need less shared
// memory traffic, lose more to their remote barriers than they gain), and a
// k-block's scale is read from shared memory while the one before is summed.
//
// Every CTA loads its own weight rows, 48 KB a stage from L2, which holds the
// tensor cores up a little and costs power.  (A cluster of two that loads each
// row once for both was 2 to 5 % faster on the plain products below, 77.1 and 295
// us on a cool GPU, and no faster on the gated one.  It needs loads that write
// another CTA's shared memory, which a library that replicas on several GPUs load
// does without.)
//
// 2048 x 4096 x 12288: 86 us a call among others, at the power limit, 62 % of twice
// the bf16 rate, with 1.68 rounds of tiles; 8192 x 12288 x 4096: 336 us, 63 %; gated
// 4096 x 12288 x 4096: 338 us, 63 %, with silu and the quantizer between tiles.  On a
// cool GPU 78.8, 302 and 306 to 320 us.
//
// SPLIT: fewer tiles than SMs.  A cluster takes one tile, each CTA a share of
// the depth; the sums are joined through distributed shared memory in rank
// order (no workspace, no atomics, the same bits every time).
namespace wide {

constexpr int S = 4;  // stages
constexpr int A_BYTES = 128 * BK, B_BYTES = 256 * BK, STAGE = A_BYTES + B_BYTES;
constexpr int CH = 8;      // k-blocks whose scales are handed over together
constexpr int SLOT = 132;  // 128 token scales and the two weight blocks'
constexpr int OFF_BAR = S * STAGE;
constexpr int NBAR = 2 * S + 2 + 2 + 2 + 2 + 1 + 1;  // full empty acc_full[2] acc_empty[2] sc_full[2] sc_empty[2] exchange drain
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int OFF_AMAX = (OFF_MISC + 16 + 127) / 128 * 128;  // float [2][2][128]
constexpr int OFF_SCALE = OFF_AMAX + 2 * 2 * 128 * 4;         // float [2][CH][SLOT]
// staging of the output, 16-bit: [8 warps][2][32 rows][16] for TMA, [8 warps][32 rows][STG_LD] without it
constexpr int STG_LD = 34;
constexpr int OFF_STG = (OFF_SCALE + 2 * CH * SLOT * 4 + 127) / 128 * 128;
constexpr int SMEM = OFF_STG + 8 * 32 * STG_LD * 2 + 1024;
constexpr int EPI0 = 4, NT = 32 * (EPI0 + 8);
constexpr int REG_LO = 88, REG_HI = 208;  // of the 168 a thread that the block is launched with
constexpr int CW = 16;                    // columns of a tensor-memory read
constexpr uint32_t TMEM_COLS = 512;
static_assert(SMEM <= 227 * 1024, "shared memory");
static_assert(128 * REG_LO + 256 * REG_HI <= NT * 168, "register split");

// A k-block at depth x of 128 tokens from m0 and of the tile's weight rows.
template <bool GATED>
__device__ __forceinline__ void load_stage(const CUtensorMap* tmA, const CUtensorMap* tmW0, const CUtensorMap* tmW1,
                                           uint32_t bar, uint32_t st, int m0, int w0, int x) {
  mbar_arrive_expect_tx(bar, STAGE);
  tma_load(st, tmA, x, m0, bar);
  tma_load(st + A_BYTES, tmW0, x, w0, bar);
  tma_load(st + A_BYTES + B_BYTES / 2, GATED ? tmW1 : tmW0, x, GATED ? w0 : w0 + 128, bar);
}

// Tile number `tile` as (tile of tokens, tile of columns): GM tiles of tokens by all
// the columns, then the next GM, so that what the CTAs work on at one time needs
// little of either operand: gated 4096 x 12288 x 4096, whose weights are 100 MB,
// 351 us with GM = 4, 348 with 8, 343 with 16, 334 with 32, 333 with 64; 2048 x 4096 x
// 12288, hot, 91, 90, 90, 87, 87.
constexpr int GM = 32;
__device__ __forceinline__ int2 tile_at(int tile, int tiles_m, int tiles_n) {
  const int g = tile / (GM * tiles_n), rows = min(GM, tiles_m - g * GM), i = tile - g * GM * tiles_n;
  return make_int2(g * GM + i % rows, i / rows);
}

// A warp's 32 rows x 16 columns through one of its two buffers to a TMA store.
__device__ __forceinline__ void store16(const CUtensorMap* tm, int x, int y, uint32_t buf, int lane, const uint32_t* o,
                                        bool in) {
  bulk_wait_read<1>();  // of the lane that stores; the others have none
  __syncwarp();
  sts128(buf + 32u * lane, o);
  sts128(buf + 32u * lane + 16, o + 4);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    if (in) tma_store(tm, x, y, buf);
    bulk_commit();
  }
}

template <bool GATED, bool SPLIT, typename T>
__global__ void __launch_bounds__(NT, 1)
wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW0,
            const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmY, const float* __restrict__ as, const float* __restrict__ ws0,
            const float* __restrict__ ws1, int M, int N, int nkb, T* __restrict__ y, uint8_t* __restrict__ q,
            float* __restrict__ qs) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full = smem_u32(sm + OFF_BAR);
  const uint32_t empty = full + 8 * S;
  const uint32_t acc_full = empty + 8 * S;
  const uint32_t acc_empty = acc_full + 8 * 2;
  const uint32_t sc_full = acc_empty + 8 * 2;
  const uint32_t sc_empty = sc_full + 8 * 2;
  const uint32_t exch = sc_empty + 8 * 2;
  const uint32_t drain = exch + 8;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(sm + OFF_MISC);

  // the shuffles tell the compiler what is the same in all lanes: the roles'
  // branches, the barriers' and the tensor memory's addresses (20 % of the time)
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr int TM = 128, TN = GATED ? 128 : 256;  // tokens and output columns of a tile
  const int tiles_n = (N + TN - 1) / TN, nblk = (N + BLK - 1) / BLK;
  const int tiles_m = (M + TM - 1) / TM, n_tiles = tiles_m * tiles_n;
  // tiles of this CTA, and its k-blocks of each
  const int ranks = SPLIT ? int(cluster_size()) : 1, rank = SPLIT ? int(cluster_rank()) : 0;
  const int tile0 = int(blockIdx.x) / ranks, tstep = SPLIT ? n_tiles : int(gridDim.x);
  const int kb0 = SPLIT ? nkb * rank / ranks : 0, kb1 = SPLIT ? nkb * (rank + 1) / ranks : nkb;

  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmW0);
    if (GATED) prefetch_map(&tmW1);
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 8);
      mbar_init(sc_full + 8 * i, 32);
      mbar_init(sc_empty + 8 * i, 8);
    }
    mbar_init(exch, 8);
    mbar_init(drain, 1);
    fence_barrier_init();
    if constexpr (SPLIT) {  // a CTA is short-lived: its first loads do not wait for the set-up
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      wait_for_previous();
      for (int s = 0; s < min(S, kb1 - kb0); ++s)
        load_stage<GATED>(&tmA, &tmW0, &tmW1, full + 8 * s, smem_u32(sm + s * STAGE),
                          tile_at(tile0, tiles_m, tiles_n).x * TM, tile_at(tile0, tiles_m, tiles_n).y * TN,
                          (kb0 + s) * BK);
    }
  }
  if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t*>(slot)), TMEM_COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  wait_for_previous();

  bool ok = true;
  if (warp < EPI0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (elect_one()) {
        int s = 0;
        uint32_t par = 0, it = 0;
        for (int tile = tile0; ok && tile < n_tiles; tile += tstep) {
          const int2 at = tile_at(tile, tiles_m, tiles_n);
          const int m0 = at.x * TM, w0 = at.y * TN;
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            if (!SPLIT || it >= S) {
              ok = wait_one(empty + 8 * s, par ^ 1u);
              if (!ok) break;
              load_stage<GATED>(&tmA, &tmW0, &tmW1, full + 8 * s, smem_u32(sm + s * STAGE), m0, w0, kb * BK);
            }
            if (++s == S) { s = 0; par ^= 1u; }
          }
        }
        // whatever happens elsewhere, no copy is in flight when the CTA ends
        for (uint32_t j = it > S ? it - S : 0; j < it; ++j) ok = wait_one(full + 8 * (j % S), (j / S) & 1) && ok;
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        const uint64_t desc = sw128_desc(smem_u32(sm));
        int s = 0;
        uint32_t par = 0, it = 0;
        for (int tile = tile0; ok && tile < n_tiles; tile += tstep)
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t b = it & 1;
            ok = wait_one(full + 8 * s, par) && wait_one(acc_empty + 8 * b, ((it >> 1) & 1) ^ 1u);
            if (!ok) break;
            fence_after_sync();
            const uint64_t ad = desc + uint64_t(s * (STAGE >> 4)), bd = ad + (A_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk) mma(tmem + 256u * b, ad + 2 * kk, bd + 2 * kk, idesc(128, 256), kk != 0);
            commit(acc_full + 8 * b);
            commit(empty + 8 * s);
            if (++s == S) { s = 0; par ^= 1u; }
          }
        commit(drain);
        next_may_start();  // not earlier: its CTAs would hold the idle SMs for nothing
      }
      __syncwarp();
      ok = wait_warp(drain, 0) && ok;
    } else if (warp == 2) {
      // ---------------------------------------------------------- scales
      // Word by word with cp.async (rows of any alignment): each lane four
      // tokens' scales of a k-block, lanes 0 and 1 the weight blocks' (gated:
      // of gate and up).
      const uint32_t sc = smem_u32(sm + OFF_SCALE) + 4 * lane;
      uint32_t it = 0;
      for (int tile = tile0; ok && tile < n_tiles; tile += tstep) {
        const int2 at = tile_at(tile, tiles_m, tiles_n);
        const int nt = at.y, m = at.x * TM + lane;
        const float* pa = as + size_t(kb0) * M + m;
        const float* pw = kb0 + (lane == 0 ? ws0 + size_t(GATED ? nt : 2 * nt) * nkb
                                    : (GATED ? ws1 + size_t(nt) * nkb : ws0 + size_t(min(2 * nt + 1, nblk - 1)) * nkb));
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          if (it % CH == 0) ok = wait_warp(sc_empty + 8 * (it / CH & 1), (it / (2 * CH) & 1) ^ 1u);
          if (!ok) break;
          const uint32_t d = sc + it % (2 * CH) * (SLOT * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (m + 32 * i < M) cp_async4(d + 128 * i, pa + 32 * i);
          if (lane < 2) cp_async4(d + 512, pw);
          pa += M;
          ++pw;
          if (it % CH == CH - 1) cp_async_arrive(sc_full + 8 * (it / CH & 1));
        }
      }
      if (it % CH != 0) cp_async_arrive(sc_full + 8 * (it / CH & 1));
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HI));
    const int quad = warp & 3, h = (warp - EPI0) >> 2;
    const int r = 32 * quad + lane;
    // columns: plain 128 h + [0, 128); gated 64 h + [0, 64) of gate and of up, 128 apart
    const uint32_t tm_row = tmem + uint32_t((GATED ? 64 : 128) * h) + (uint32_t(32 * quad) << 16);
    auto col = [](int c) { return uint32_t(c + (GATED && c >= 64 ? 64 : 0)); };
    const uint32_t sc = smem_u32(sm + OFF_SCALE);
    uint32_t it = 0;
    int ti = 0;
    float sn0 = 0.f, sn1 = 0.f;  // of k-block `it`, read while the one before is summed
    auto next_scales = [&]() {
      if (it % CH == 0 && ok) ok = wait_warp(sc_full + 8 * (it / CH & 1), it / (2 * CH) & 1);
      const uint32_t sl = sc + it % (2 * CH) * (4 * SLOT);
      const float a = lds(sl + 4 * r);
      sn0 = a * lds(sl + 4 * (GATED ? 128 : 128 + h));
      if (GATED) sn1 = a * lds(sl + 4 * 129);
      if (it % CH == CH - 1) {
        __syncwarp();
        mbar_arrive_if(sc_empty + 8 * (it / CH & 1), lane == 0);
      }
    };
    const uint32_t last = uint32_t((n_tiles - tile0 + tstep - 1) / tstep) * uint32_t(kb1 - kb0);
    if (last > 0) next_scales();
    for (int tile = tile0; ok && tile < n_tiles; tile += tstep, ++ti) {
      const int2 at = tile_at(tile, tiles_m, tiles_n);
      const int gm = at.x * TM + r, nt = at.y;
      const bool in = gm < M;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t b = it & 1;
        ok = ok && wait_warp(acc_full + 8 * b, (it >> 1) & 1);
        if (!ok) break;
        fence_after_sync();
        const uint32_t t = tm_row + 256u * b;
        uint32_t v[2][CW];
        tmem_ld(t, v[0]);
        const float s0 = sn0, s1 = GATED ? sn1 : sn0;
#pragma unroll
        for (int c = 0; c < 128 / CW; ++c) {
          wait_ld();
          if (c < 128 / CW - 1) {
            tmem_ld(t + col(CW * (c + 1)), v[(c + 1) & 1]);
          } else {  // the last read is done: the buffer is free
            fence_before_sync();
            mbar_arrive_if(acc_empty + 8 * b, lane == 0);
            if (++it < last) next_scales();
          }
          const float s = GATED && c >= 64 / CW ? s1 : s0;
          const float2 s2 = make_float2(s, s);
#pragma unroll
          for (int j = 0; j < CW / 2; ++j)
            acc[CW / 2 * c + j] = __ffma2_rn(
                make_float2(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1])), s2, acc[CW / 2 * c + j]);
        }
      }
      if constexpr (SPLIT) {
        // partial sums to where the stages were (all read by now):
        // [column / 4][token][4], so that four columns are one 16-byte access
        if (ok) {
          const uint32_t part = smem_u32(sm) + 16 * r + 512 * ((GATED ? 64 : 128) * h);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            sts128(part + 2048 * (i + (GATED && i >= 16 ? 16 : 0)), acc[2 * i], acc[2 * i + 1]);
        }
        break;
      }
      if (!ok) break;
      if constexpr (!GATED) {
        const int n0 = nt * 256 + 128 * h;
        if ((N & 7) == 0) {
          // 16 columns at a time through one of the warp's two buffers to a TMA
          // store: the writes go out under the next tile's MMAs.  (Stores from
          // registers, 32 bytes to each of 32 rows, held the warps for 2.8 us a tile.)
          const int row0 = gm - lane;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t buf = smem_u32(sm + OFF_STG) + uint32_t(((warp - EPI0) * 2 + (c & 1)) * 1024);
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = from_f2<T>(acc[8 * c + j]);
            store16(&tmY, n0 + 16 * c, row0, buf, lane, o, row0 < M && n0 + 16 * c < N);
          }
        } else {
          // rows of any alignment: through shared memory, a row's 32 columns by the 32 lanes
          uint16_t* stg = reinterpret_cast<uint16_t*>(sm + OFF_STG) + (warp - EPI0) * 32 * STG_LD;
          uint16_t* y16 = reinterpret_cast<uint16_t*>(y);
          const int row0 = gm - lane, rows = min(32, M - row0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int gn = n0 + 32 * c;
            if (gn >= N) break;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) *reinterpret_cast<uint32_t*>(stg + lane * STG_LD + 2 * j) = from_f2<T>(acc[16 * c + j]);
            __syncwarp();
            if (gn + lane < N)
              for (int i = 0; i < rows; ++i) y16[size_t(row0 + i) * N + gn + lane] = stg[i * STG_LD + lane];
          }
        }
      } else {
        // acc[0 .. 31]: gate of columns 64 h + [0, 64), acc[32 .. 63]: up
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          acc[j] = silu_mul(acc[j], acc[32 + j]);
          m = max_nan(m, max_nan(fabsf(acc[j].x), fabsf(acc[j].y)));
        }
        // the block's other 64 columns are the other half's: exchange the abs-max
        const uint32_t am = smem_u32(sm + OFF_AMAX) + (ti & 1) * 1024 + 4 * r;
        sts(am + 512 * h, m);
        __syncwarp();
        if (lane == 0) mbar_arrive(exch);
        ok = wait_warp(exch, uint32_t(ti & 1));
        if (!ok) break;
        m = block_amax(max_nan(m, lds(am + 512 * (h ^ 1))));
        const Quotient quo(m);
        const int n0 = nt * 128 + 64 * h;
        if (in) {
          if (h == 0) qs[size_t(nt) * M + gm] = block_scale(m);
          uint8_t* qr = q + size_t(gm) * N + n0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (n0 + 16 * c < N) {
              uint4 o;
              o.x = cvt_e4m3x4(quo(acc[8 * c + 0]), quo(acc[8 * c + 1]));
              o.y = cvt_e4m3x4(quo(acc[8 * c + 2]), quo(acc[8 * c + 3]));
              o.z = cvt_e4m3x4(quo(acc[8 * c + 4]), quo(acc[8 * c + 5]));
              o.w = cvt_e4m3x4(quo(acc[8 * c + 6]), quo(acc[8 * c + 7]));
              *reinterpret_cast<uint4*>(qr + 16 * c) = o;
            }
        }
      }
    }
    if constexpr (SPLIT) {
      // ---- the ranks' sums, in rank order, through distributed shared memory:
      // 16 columns at a time, dealt out over the cluster's 2 * ranks warp sets
      cluster_sync();
      const int2 at = tile_at(tile0, tiles_m, tiles_n);
      const int gm = at.x * TM + r, row0 = gm - lane, nt = at.y;
      const uint32_t part = smem_u32(sm) + 16 * r;
      auto sum16 = [&](int col, float2 (&o)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < ranks; ++k) {
          const uint32_t src = mapa(part + 512 * col, uint32_t(k));
          float4 f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = lds128_cluster(src + 2048 * i);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[2 * i] = __fadd2_rn(o[2 * i], make_float2(f[i].x, f[i].y));
            o[2 * i + 1] = __fadd2_rn(o[2 * i + 1], make_float2(f[i].z, f[i].w));
          }
        }
      };
      const int w0 = 2 * rank + h;
      if constexpr (!GATED) {
        int n = 0;
        for (int c = w0; c < 16 && row0 < M; c += 2 * ranks, ++n) {
          const int gn = nt * 256 + 16 * c;
          if (gn >= N) break;
          float2 f[8];
          sum16(16 * c, f);
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = from_f2<T>(f[i]);
          if ((N & 7) == 0) {
            const uint32_t buf = smem_u32(sm + OFF_STG) + uint32_t(((warp - EPI0) * 2 + (n & 1)) * 1024);
            store16(&tmY, gn, row0, buf, lane, o, true);
          } else {
            uint16_t* stg = reinterpret_cast<uint16_t*>(sm + OFF_STG) + (warp - EPI0) * 32 * STG_LD;
            uint16_t* y16 = reinterpret_cast<uint16_t*>(y);
            const int cc = gn + (lane & 15), rows = min(32, M - row0);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint32_t*>(stg + lane * STG_LD + 2 * i) = o[i];
            __syncwarp();
            if (cc < N)
              for (int i = lane >> 4; i < rows; i += 2) y16[size_t(row0 + i) * N + cc] = stg[i * STG_LD + (lane & 15)];
          }
        }
      } else {
        float2 z[2][8];  // at most two of the eight chunks
        float m = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int c = w0 + 2 * ranks * n;
          if (c >= 8 || row0 >= M) break;
          float2 u[8];
          sum16(16 * c, z[n]);
          sum16(128 + 16 * c, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[n][i] = silu_mul(z[n][i], u[i]);
            m = max_nan(m, max_nan(fabsf(z[n][i].x), fabsf(z[n][i].y)));
          }
        }
        const uint32_t am = smem_u32(sm + OFF_AMAX) + 4 * r;
        sts(am + 512 * h, m);
        cluster_sync();
        if (row0 < M) {
          for (int k = 0; k < ranks; ++k) {
            const uint32_t src = mapa(am, uint32_t(k));
            m = max_nan(m, max_nan(lds_cluster(src), lds_cluster(src + 512)));
          }
          m = block_amax(m);
          const Quotient quo(m);
          if (gm < M && w0 == 0) qs[size_t(nt) * M + gm] = block_scale(m);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int c = w0 + 2 * ranks * n, gn = nt * 128 + 16 * c;
            if (c < 8 && gn < N && gm < M) {
              uint4 o;
              o.x = cvt_e4m3x4(quo(z[n][0]), quo(z[n][1]));
              o.y = cvt_e4m3x4(quo(z[n][2]), quo(z[n][3]));
              o.z = cvt_e4m3x4(quo(z[n][4]), quo(z[n][5]));
              o.w = cvt_e4m3x4(quo(z[n][6]), quo(z[n][7]));
              *reinterpret_cast<uint4*>(q + size_t(gm) * N + gn) = o;
            }
          }
        }
      }
      cluster_sync();  // this CTA's sums have been read
    }
  }
  if (SPLIT && warp < EPI0) {  // the barriers that the epilogue warps pass
    cluster_sync();
    if (GATED) cluster_sync();
    cluster_sync();
  }

  bulk_wait_read<0>();  // shared memory is read out
  if (!ok) record_error(QUAROT_ERR_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    fence_after_sync();
    tmem_free(tmem, TMEM_COLS);
  }
}

}  // namespace wide

// ===================================================================== narrow
// Few tokens: the time is that of reading the weights once: 1 x 4096 x 12288 in
// 11.3 us (4.5 TB/s), gated 4 x 12288 x 4096 in 18.7 us (5.4 TB/s), of which some
// 4 us are launch, set-up, first load and join.
//
// A CTA takes 128 weight rows (gated: 128 gate and 128 up rows) as the MMA's M,
// the tokens, up to TN, as its N, and 1 / cluster_size of the depth.  Its thread
// (lane quadrant, lane) holds one weight row's sums of the tokens.  At the end
// every CTA writes its sums to its shared memory, and the warps of all the
// cluster's CTAs take tokens in turn, adding the ranks' sums in rank order
// through distributed shared memory: no workspace, no atomics, the same bits
// every time.
//
//   warps 0-3  epilogue, one per TMEM lane quadrant
//   warp 4     TMA producer
//   warp 5     TMEM allocator, MMA issuer
namespace narrow {

constexpr int NT = 192;

template <bool GATED, int TN>
struct Cfg {
  static constexpr int NW = GATED ? 2 : 1;
  static constexpr int KC = GATED ? 2 : 4;  // k-blocks whose scales a warp stages at a time
  static constexpr int W_BYTES = 128 * BK, A_BYTES = TN * BK;
  static constexpr int STAGE = NW * W_BYTES + A_BYTES;
  static constexpr int S = GATED ? 3 : TN == 64 ? 4 : TN == 32 ? 5 : 6;
  static constexpr uint32_t COLS = 2 * NW * TN < 32 ? 32 : 2 * NW * TN;  // two accumulator buffers
  static constexpr int OFF_BAR = S * STAGE;
  static constexpr int NBAR = 2 * S + 5;  // full empty acc_full[2] acc_empty[2] drain
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_SC = (OFF_MISC + 16 + 127) / 128 * 128;  // float [4 warps][KC][NW][TN]
  static constexpr int SMEM_MIN = OFF_SC + 4 * KC * NW * TN * 4 + 1024;
  // at most two CTAs on an SM, whatever the tokens: their tensor memory always fits
  static constexpr int SMEM = SMEM_MIN < 80 * 1024 ? 80 * 1024 : SMEM_MIN;
  static_assert(2 * COLS <= 512 && SMEM <= 113 * 1024, "two CTAs per SM");
  static_assert(NW * TN * 128 * 4 <= S * STAGE, "the sums fit where the stages were");
};

template <bool GATED, int TN, typename T>
__global__ void __launch_bounds__(NT, 2)
narrow_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW0,
              const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmY, const float* __restrict__ as, const float* __restrict__ ws0,
              const float* __restrict__ ws1, int M, int N, int nkb, T* __restrict__ y, uint8_t* __restrict__ q,
              float* __restrict__ qs) {
  using C = Cfg<GATED, TN>;
  constexpr int S = C::S, NW = C::NW, KC = C::KC;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full = smem_u32(sm + C::OFF_BAR);
  const uint32_t empty = full + 8 * S;
  const uint32_t acc_full = empty + 8 * S;
  const uint32_t acc_empty = acc_full + 8 * 2;
  const uint32_t drain = acc_empty + 8 * 2;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MISC);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = int(cluster_rank()), ranks = int(cluster_size());
  const int wb = int(blockIdx.x) / ranks;  // block of 128 weight rows (and of output columns)
  const int kb_lo = int(int64_t(nkb) * rank / ranks), kb_hi = int(int64_t(nkb) * (rank + 1) / ranks);

  auto load_stage = [&](int s, int kb) {
    const uint32_t bar = full + 8 * s, st = smem_u32(sm) + uint32_t(s * C::STAGE);
    mbar_arrive_expect_tx(bar, C::STAGE);
    tma_load(st, &tmW0, kb * BK, wb * 128, bar);
    if (GATED) tma_load(st + C::W_BYTES, &tmW1, kb * BK, wb * 128, bar);
    tma_load(st + NW * C::W_BYTES, &tmA, kb * BK, 0, bar);
  };
  const int early = min(S, kb_hi - kb_lo);  // stages loaded before the set-up is over

  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmW0);
    if (GATED) prefetch_map(&tmW1);
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    wait_for_previous();
    for (int s = 0; s < early; ++s) load_stage(s, kb_lo + s);
  }
  if (warp == 5) tmem_alloc(smem_u32(const_cast<uint32_t*>(slot)), C::COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  wait_for_previous();

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    if (elect_one()) {
      int i = early;
      for (int kb = kb_lo + early; kb < kb_hi; ++kb, ++i) {
        const int s = i % S;
        ok = wait_one(empty + 8 * s, uint32_t((i / S) & 1) ^ 1u);
        if (!ok) break;
        load_stage(s, kb);
      }
      // whatever happens elsewhere, no copy is in flight when the CTA ends
      for (int j = i > S ? i - S : 0; j < i; ++j) ok = wait_one(full + 8 * (j % S), uint32_t((j / S) & 1)) && ok;
    }
    __syncwarp();
    if (!ok) record_error(QUAROT_ERR_TIMEOUT);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    if (elect_one()) {
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const int i = kb - kb_lo, s = i % S, b = i & 1;
        ok = wait_one(full + 8 * s, uint32_t((i / S) & 1)) && wait_one(acc_empty + 8 * b, uint32_t((i >> 1) & 1) ^ 1u);
        if (!ok) break;
        fence_after_sync();
        const uint32_t st = smem_u32(sm + s * C::STAGE);
        const uint64_t ad = sw128_desc(st + NW * C::W_BYTES);
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const uint64_t wd = sw128_desc(st + p * C::W_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma(tmem + uint32_t((b * NW + p) * TN), wd + uint64_t(2 * kk), ad + uint64_t(2 * kk), idesc(128, TN), kk != 0);
        }
        commit(acc_full + 8 * b);
        commit(empty + 8 * s);
      }
      commit(drain);
      next_may_start();  // with the sums still to be joined
    }
    __syncwarp();
    if (!wait_warp(drain, 0) || !ok) record_error(QUAROT_ERR_TIMEOUT);
  } else {
    // ------------------------------------------------------------ epilogue
    float2 acc[NW][TN / 2];
#pragma unroll
    for (int p = 0; p < NW; ++p)
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) acc[p][j] = make_float2(0.f, 0.f);
    // scales a_scale w_scale of KC k-blocks, in the warp's own rows of shared
    // memory; the token scales of the next KC are already in registers
    const uint32_t sc = smem_u32(sm + C::OFF_SC) + uint32_t(warp * KC * NW * TN * 4);
    constexpr int PL = KC * TN / 32;
    float pre[PL], pw[NW];
    const float* w0 = ws0 + size_t(wb) * nkb;
    const float* w1 = GATED ? ws1 + size_t(wb) * nkb : nullptr;
    auto fetch = [&](int kb) {
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const int k = (e * 32 + lane) / TN, n = (e * 32 + lane) % TN;
        pre[e] = kb + k < kb_hi && n < M ? __ldg(as + size_t(kb + k) * M + n) : 0.f;
      }
      pw[0] = lane < KC && kb + lane < kb_hi ? __ldg(w0 + kb + lane) : 0.f;
      if constexpr (GATED) pw[1] = lane < KC && kb + lane < kb_hi ? __ldg(w1 + kb + lane) : 0.f;
    };
    fetch(kb_lo);
    const uint32_t tm_row = tmem + (uint32_t(32 * warp) << 16);
    bool ok = true;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      const int i = kb - kb_lo, b = i & 1, kc = i % KC;
      if (kc == 0) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < PL; ++e) {
          const int k = (e * 32 + lane) / TN, n = (e * 32 + lane) % TN;
#pragma unroll
          for (int p = 0; p < NW; ++p)
            sts(sc + 4 * uint32_t((k * NW + p) * TN + n), pre[e] * __shfl_sync(0xffffffffu, pw[p], k));
        }
        __syncwarp();
        fetch(kb + KC);
      }
      ok = wait_warp(acc_full + 8 * b, uint32_t((i >> 1) & 1));
      if (!ok) break;
      fence_after_sync();
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        const uint32_t scp = sc + 4 * uint32_t((kc * NW + p) * TN);
        constexpr int CW = TN < 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < TN / CW; ++c) {
          uint32_t v[CW];
          tmem_ld(tm_row + uint32_t((b * NW + p) * TN + c * CW), v);
          wait_ld();
          if (p == NW - 1 && c == TN / CW - 1) {
            fence_before_sync();
            mbar_arrive_if(acc_empty + 8 * b, lane == 0);
          }
#pragma unroll
          for (int j = 0; j < CW / 4; ++j) {
            const float4 s4 = lds128(scp + 4 * (c * CW + 4 * j));
            float2* a2 = &acc[p][(c * CW + 4 * j) / 2];
            a2[0] = __ffma2_rn(make_float2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), make_float2(s4.x, s4.y), a2[0]);
            a2[1] = __ffma2_rn(make_float2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])), make_float2(s4.z, s4.w), a2[1]);
          }
        }
      }
    }
    // every k-block's accumulator was waited for, so the stages' loads and
    // reads are over: the sums [NW][TN][128 weight rows] take their place
    // (after an expired wait the values are void, the producer drains below)
    if (ok) {
      const uint32_t part = smem_u32(sm) + 4 * (32 * warp + lane);
#pragma unroll
      for (int p = 0; p < NW; ++p)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
          sts(part + 512 * (p * TN + 2 * j), acc[p][j].x);
          sts(part + 512 * (p * TN + 2 * j + 1), acc[p][j].y);
        }
    } else {
      record_error(QUAROT_ERR_TIMEOUT);
    }
  }

  fence_before_sync();
  __syncthreads();
  if (warp == 5) {  // before the cluster's barrier: no CTA holds tensor memory while it waits for another
    fence_after_sync();
    tmem_free(tmem, C::COLS);
  }
  cluster_sync();
  // ---- a warp per token: lane l holds weight rows 4 l .. 4 l + 3
  const uint32_t part = smem_u32(sm);
  const int n0 = wb * 128 + 4 * lane;
  for (int n = rank * (NT / 32) + warp; n < M; n += ranks * (NT / 32)) {
    float2 v[NW][2];
#pragma unroll
    for (int p = 0; p < NW; ++p) v[p][0] = v[p][1] = make_float2(0.f, 0.f);
    for (int k = 0; k < ranks; ++k)
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        const float4 f = lds128_cluster(mapa(part + uint32_t(((p * TN + n) * 128 + 4 * lane) * 4), uint32_t(k)));
        v[p][0] = __fadd2_rn(v[p][0], make_float2(f.x, f.y));
        v[p][1] = __fadd2_rn(v[p][1], make_float2(f.z, f.w));
      }
    const size_t row = size_t(n) * N;
    if constexpr (!GATED) {
      const uint32_t lo = from_f2<T>(v[0][0]), hi = from_f2<T>(v[0][1]);
      uint16_t* yr = reinterpret_cast<uint16_t*>(y) + row + n0;
      if ((N & 3) == 0) {
        if (n0 < N) *reinterpret_cast<uint2*>(yr) = make_uint2(lo, hi);
      } else {
        if (n0 < N) yr[0] = uint16_t(lo);
        if (n0 + 1 < N) yr[1] = uint16_t(lo >> 16);
        if (n0 + 2 < N) yr[2] = uint16_t(hi);
        if (n0 + 3 < N) yr[3] = uint16_t(hi >> 16);
      }
    } else {
      const float2 z0 = silu_mul(v[0][0], v[1][0]);
      const float2 z1 = silu_mul(v[0][1], v[1][1]);
      // weight rows past N were read as zeros: z = 0 there
      float m = max_nan(max_nan(fabsf(z0.x), fabsf(z0.y)), max_nan(fabsf(z1.x), fabsf(z1.y)));
      m = n0 < N ? m : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = block_amax(m);
      const Quotient quo(m);
      if (n0 < N) *reinterpret_cast<uint32_t*>(q + row + n0) = cvt_e4m3x4(quo(z0), quo(z1));
      if (lane == 0) qs[size_t(wb) * M + n] = block_scale(m);
    }
  }
  cluster_sync();  // the other ranks have read this CTA's sums
}

}  // namespace narrow

// One thread's wait on a barrier that nothing completes.
__global__ void selftest_wait_kernel() {
  __shared__ __align__(8) uint64_t bar;
  mbar_init(smem_u32(&bar), 1);
  fence_barrier_init();
  if (!wait_one(smem_u32(&bar), 0)) record_error(QUAROT_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host
static PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
static std::once_flag g_encode_once;

static bool get_encoder() {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult r;
    void* fn = nullptr;
    if (cuda_ok(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r)) &&
        r == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// [rows, K] bytes in boxes of 128 x box_rows, 128B swizzle; rows and depth past the end read as zeros.
static bool make_map(CUtensorMap* tm, const void* base, int64_t rows, int64_t K, int box_rows) {
  cuuint64_t gdim[2] = {cuuint64_t(K), cuuint64_t(rows)};
  cuuint64_t gstride[1] = {cuuint64_t(K)};
  cuuint32_t box[2] = {cuuint32_t(BK), cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The 16-bit output [rows, N], N % 8 == 0, in the boxes of 16 columns x 32 rows that an epilogue warp stores.
static bool make_out_map(CUtensorMap* tm, void* base, int64_t rows, int64_t N) {
  cuuint64_t gdim[2] = {cuuint64_t(N), cuuint64_t(rows)};
  cuuint64_t gstride[1] = {cuuint64_t(2 * N)};
  cuuint32_t box[2] = {16, 32};
  cuuint32_t estr[2] = {1, 1};
  return g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int sm_count() {
  int dev = 0, n = 0;
  if (!cuda_ok(cudaGetDevice(&dev))) return 0;
  if (!cuda_ok(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev))) return 0;
  return n;
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

static int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K <= 0) return QUAROT_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if (K % 16 != 0 || K > (int64_t(1) << 20) || M > lim || N > lim) return QUAROT_ERR_UNSUPPORTED;
  if (((M + 127) / 128) * ((N + 127) / 128) >= (int64_t(1) << 31) - 512) return QUAROT_ERR_UNSUPPORTED;
  return QUAROT_OK;
}

struct Args {
  const uint8_t *a, *w0, *w1;
  const float *as, *ws0, *ws1;
  int64_t M, N, K;
  void* y;
  uint8_t* q;
  float* qs;
  cudaStream_t st;
};

template <typename Kern, typename T>
static int launch(const Args& p, Kern* kern, AttrCache& attr, dim3 grid, int threads, int cluster, int smem, int a_box,
                  int w_box, T* y) {
  CUtensorMap ta, t0, t1, ty;
  if (!make_map(&ta, p.a, p.M, p.K, a_box) || !make_map(&t0, p.w0, p.N, p.K, w_box)) return QUAROT_ERR_CUDA;
  if (p.w1 == nullptr) t1 = t0;
  else if (!make_map(&t1, p.w1, p.N, p.K, w_box)) return QUAROT_ERR_CUDA;
  if (threads != wide::NT || y == nullptr || p.N % 8 != 0) ty = t0;
  else if (!make_out_map(&ty, y, p.M, p.N)) return QUAROT_ERR_CUDA;
  if (!smem_attr_once(kern, smem, attr)) return QUAROT_ERR_LAUNCH;
  return launch_dependent(kern, grid, unsigned(threads), size_t(smem), unsigned(cluster), p.st, ta, t0, t1, ty, p.as,
                          p.ws0, p.ws1, p.M, p.N, (p.K + BK - 1) / BK, y, p.q, p.qs);
}

template <bool GATED, int TN, typename T>
static int launch_narrow(const Args& p, int cluster) {
  static AttrCache attr;
  const unsigned wbs = unsigned((p.N + 127) / 128);
  return launch(p, narrow::narrow_kernel<GATED, TN, T>, attr, dim3(wbs * unsigned(cluster)), narrow::NT, cluster,
                narrow::Cfg<GATED, TN>::SMEM, TN, 128, static_cast<T*>(p.y));
}

// Over how many CTAs a tile's depth is split: as many as find an SM at once,
// with two k-blocks each at least.  A cluster of 8 finds room on 4/5 of the SMs
// only (the SMs of a GPC are not a multiple of 8), one of 4 on 18/19.  In us:
//
//   tiles, k-blocks                     1     2     4     8 ranks
//     8, 96    128 x 2048 x 12288    38.5  24.3  17.2  16.4
//    16, 32    128 x 4096 x 4096     15.9  13.1  11.5  24.1
//    32, 96    256 x 4096 x 12288    38.8  25.3  20.1  47.8
//    64, 32    512 x 4096 x 4096     16.3  13.9  24.3  59.9
//    96, 32    700 x 4096 x 4096     16.9  26.0  34.5  78.3
//    64, 32    gated 256 x 4096 x 4096  17.1  15.9  27.4  64.9
static int split_ranks(int64_t tiles, int64_t nkb, int sms) {
  if (tiles * 8 <= sms * 15 / 19 && nkb >= 16) return 8;
  if (tiles * 4 <= sms * 18 / 19 && nkb >= 8) return 4;
  if (tiles * 2 <= sms && nkb >= 4) return 2;
  return 1;
}

template <bool GATED, typename T>
static int run(const Args& p) {
  if (!get_encoder()) return QUAROT_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return QUAROT_ERR_CUDA;
  // Narrow up to here, where one token tile's sums still fit two CTAs' registers
  // (a second tile would read the weights again).  It and the split wide form:
  // 64 x 4096 x 12288 13.8 and 17.1 us, 16 x 12288 x 4096 11.6 and 17.6 us;
  // gated 32 x 12288 x 4096 21.0 and 21.9 us, 16 x 12288 x 4096 20.1 and 27.7 us.
  constexpr int kNarrow = GATED ? 32 : 64;
  const int64_t wbs = (p.N + 127) / 128, nkb = (p.K + BK - 1) / BK;
  if (p.M <= kNarrow) {
    // The depth over as many CTAs as two on every SM, of four k-blocks at least:
    // 1 x 4096 x 12288 24.7, 14.9, 11.3, 11.2 us over 1, 2, 4, 8; 37 x 12288 x 4096
    // (96 blocks of rows) 14.7, 12.8, 16.7, 21.6; gated 4 x 12288 x 4096 20.5, 18.8, 22.5, 27.3.
    int cl = 1;
    while (cl < 8 && wbs * cl * 2 <= 2 * sms && nkb / (2 * cl) >= 4) cl *= 2;
    if (p.M <= 16) return launch_narrow<GATED, 16, T>(p, cl);
    if (p.M <= 32) return launch_narrow<GATED, 32, T>(p, cl);
    if constexpr (!GATED) return launch_narrow<GATED, 64, T>(p, cl);
  }
  constexpr int TN = GATED ? 128 : 256;
  const int64_t tiles = ((p.M + 127) / 128) * ((p.N + TN - 1) / TN);
  const int ranks = split_ranks(tiles, nkb, sms);
  if (ranks > 1) {
    static AttrCache attr;
    return launch(p, wide::wide_kernel<GATED, true, T>, attr, dim3(unsigned(tiles * ranks)), wide::NT, ranks, wide::SMEM,
                  128, 128, static_cast<T*>(p.y));
  }
  static AttrCache attr;
  return launch(p, wide::wide_kernel<GATED, false, T>, attr, dim3(unsigned(tiles < sms ? tiles : sms)), wide::NT, 1,
                wide::SMEM, 128, 128, static_cast<T*>(p.y));
}

}  // namespace gemm
}  // namespace fp8
}  // namespace quarot

using namespace quarot;

bool quarot::launch_fp8_selftest_wait(cudaStream_t stream) {
  fp8::gemm::selftest_wait_kernel<<<1, 1, 0, stream>>>();
  return cudaGetLastError() == cudaSuccess;
}

bool quarot::take_fp8_error_word(unsigned int* word) {
  const unsigned int zero = 0;
  if (!cuda_ok(cudaMemcpyFromSymbol(word, g_error_word, sizeof(zero)))) return false;
  return *word == 0 || cuda_ok(cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)));
}

extern "C" int quarot_fp8_gemm(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q, const float* w_scale,
                               int64_t M, int64_t N, int64_t K, void* y, int dtype, void* stream) {
  using namespace quarot::fp8::gemm;
  if (dtype != QUAROT_FP16 && dtype != QUAROT_BF16) return QUAROT_ERR_INVALID_ARG;
  const int e = check_sizes(M, N, K);
  if (e != QUAROT_OK || M == 0 || N == 0) return e;
  if (!a_q || !a_scale || !w_q || !w_scale || !y) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(a_q, 16) || misaligned(w_q, 16) || misaligned(y, 16) || misaligned(a_scale, 4) || misaligned(w_scale, 4))
    return QUAROT_ERR_ALIGNMENT;
  const Args p{a_q, w_q, nullptr, a_scale, w_scale, nullptr, M, N, K, y, nullptr, nullptr, static_cast<cudaStream_t>(stream)};
  return dtype == QUAROT_FP16 ? run<false, __half>(p) : run<false, __nv_bfloat16>(p);
}

extern "C" int quarot_fp8_gated_gemm(const uint8_t* a_q, const float* a_scale, const uint8_t* wg_q,
                                     const float* wg_scale, const uint8_t* wu_q, const float* wu_scale, int64_t M,
                                     int64_t I, int64_t K, uint8_t* q_out, float* scale_out, void* stream) {
  using namespace quarot::fp8::gemm;
  const int e = check_sizes(M, I, K);
  if (e != QUAROT_OK) return e;
  if (I % 16 != 0) return QUAROT_ERR_UNSUPPORTED;
  if (M == 0 || I == 0) return QUAROT_OK;
  if (!a_q || !a_scale || !wg_q || !wg_scale || !wu_q || !wu_scale || !q_out || !scale_out) return QUAROT_ERR_INVALID_ARG;
  if (misaligned(a_q, 16) || misaligned(wg_q, 16) || misaligned(wu_q, 16) || misaligned(q_out, 16) ||
      misaligned(a_scale, 4) || misaligned(wg_scale, 4) || misaligned(wu_scale, 4) || misaligned(scale_out, 4))
    return QUAROT_ERR_ALIGNMENT;
  const Args p{a_q, wg_q, wu_q, a_scale, wg_scale, wu_scale, M, I, K, nullptr, q_out, scale_out,
               static_cast<cudaStream_t>(stream)};
  return run<true, __half>(p);
}
