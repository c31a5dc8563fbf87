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
//   namespace wide    many tokens: CTA pairs (cta_group::2), 256 tokens x 256
//                     weight rows (gated: 128 gate and 128 up rows)
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

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
// Arrives on the barrier (CG 2: on both CTAs') when all earlier MMAs of this thread are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
}
// The same on the barrier of each CTA in `mask`.
__device__ __forceinline__ void commit_to(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
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
// One box at (x, y) into this CTA's shared memory; `bar` is a shared::cluster
// address (CG 2: of either CTA of the pair).
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The same box into the same place of each CTA in `mask`, completing on each one's own barrier.
__device__ __forceinline__ void tma_load_to(uint32_t dst, const CUtensorMap* tm, int x, int y, uint32_t bar,
                                            uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster [%0], [%1, {%2, "
      "%3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "h"(mask)
      : "memory");
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
// Arrival on a barrier of either CTA (a shared::cluster address).  What it
// hands over are finished tensor-memory reads (tcgen05.wait::ld before it), no
// generic-proxy data.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool wait_s(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int n = 0; n < 100000; ++n)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
// One lane of a converged warp, in the form in which the compiler sees that it is one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Whether the phase is over, without waiting (try_wait may sleep).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort));
}
__device__ __forceinline__ bool warp_flag(volatile int* flag) { return __shfl_sync(0xffffffffu, *flag, 0) != 0; }
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* o) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
               "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}

// Four bytes from global to this CTA's shared memory, asynchronously; the
// arrival on the barrier follows this thread's copies so far.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float silu(float g) { return __fdiv_rn(g, 1.0f + expf(-g)); }

// ===================================================================== wide
// Persistent CTA pairs; a pair computes 256 tokens x 256 weight rows.  Each
// CTA loads its 128 token rows and half of the weight rows of a k-block (32
// KB, S stages) and holds the sums of its 128 tokens x 256 columns: 256
// epilogue threads x 128 fp32 registers.
//
//   warp 0      TMA producer; both CTAs' loads complete on the leader's barrier
//   warp 1      TMEM allocator; MMA issuer in the leader
//   warps 4-11  epilogue: warp w reads TMEM lane quadrant w % 4, column half (w - 4) / 4
//
// The first warpgroup hands registers to the other two (setmaxnreg), whose
// sums, tensor-memory reads in flight and scales need about 200 a thread.
//
// The MMAs of a k-block run as two of N = 128 (column halves), each with its
// own accumulator and barriers, two buffers each: 4 x 128 tensor-memory
// columns.  A half's buffer is free for 3/4 of two k-blocks' MMA time before
// its next MMA needs it.
//
// Column half h of a tile holds, from CTA 0's weight rows, columns [0, 64) and
// from CTA 1's [64, 128): weight rows n0 + 128 h + 64 rank + [0, 64) for the
// plain product; for the gated one CTA 0 loads gate rows and CTA 1 up rows
// i0 + 64 h + [0, 64), so a thread holds gate and up of the same columns.
namespace wide {

constexpr int S = 6;  // stages
constexpr int A_BYTES = 128 * BK, B_BYTES = 128 * BK;
constexpr int OFF_B = S * A_BYTES;
constexpr int OFF_BAR = OFF_B + S * B_BYTES;
constexpr int CH = 8;  // k-blocks whose scales are handed over together
constexpr int NBAR = 2 * S + 4 + 4 + 2 + 2 + 1 + 1;  // full empty acc_full[2][2] acc_empty[2][2] sc_full[2] sc_empty[2] exchange drain
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int OFF_AMAX = (OFF_MISC + 16 + 127) / 128 * 128;  // float [2][2][128]
constexpr int SLOT = 132;                                      // 128 token scales and the weight blocks' two
constexpr int OFF_SCALE = OFF_AMAX + 2 * 2 * 128 * 4;          // float [2][CH][SLOT]
constexpr int OFF_STG = OFF_SCALE + 2 * CH * SLOT * 4;         // 16-bit [8 warps][32 rows][STG_LD]
constexpr int STG_LD = 34;
constexpr int SMEM = OFF_STG + 8 * 32 * STG_LD * 2 + 1024;
constexpr int EPI0 = 4, NT = 32 * (EPI0 + 8);
constexpr int REG_LO = 104, REG_HI = 200;  // of the 168 a thread that the block is launched with
static_assert(128 * REG_LO + 256 * REG_HI <= NT * 168, "register split");
constexpr uint32_t TMEM_COLS = 512;
constexpr bool HALVES = true;
constexpr int CW = 16;                                    // columns of a tensor-memory read
constexpr int W_BOX = 64;                                 // weight rows of a copy: a half's from one CTA
constexpr int MN = HALVES ? 128 : 256;                    // columns of an MMA
static_assert(SMEM <= 227 * 1024, "shared memory");

template <bool GATED, typename T>
__global__ void __launch_bounds__(NT, 1)
wide_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW0,
            const __grid_constant__ CUtensorMap tmW1, const float* __restrict__ as, const float* __restrict__ ws0,
            const float* __restrict__ ws1, int M, int N, int nkb, T* __restrict__ y, uint8_t* __restrict__ q,
            float* __restrict__ qs) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 4;  // [buffer][half]
  uint64_t* sc_full = acc_empty + 4;
  uint64_t* sc_empty = sc_full + 2;
  uint64_t* exch = sc_empty + 2;
  uint64_t* drain = exch + 1;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(sm + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair_id = int(blockIdx.x) >> 1, n_pairs = int(gridDim.x) >> 1;
  constexpr int TN = GATED ? 128 : 256;  // output columns of a tile
  const int tiles_n = (N + TN - 1) / TN, nblk = (N + BLK - 1) / BLK;
  const int n_tiles = ((M + 255) / 256) * tiles_n;

  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmW0);
    if (GATED) prefetch_map(&tmW1);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], HALVES ? 8 : 16);  // the epilogue warps of both CTAs (used in the leader)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sc_full[i], 32);
      mbar_init(&sc_empty[i], 8);
    }
    mbar_init(exch, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(const_cast<uint32_t*>(slot)), TMEM_COLS);
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrival
  fence_after_sync();
  const uint32_t tmem = *slot;

  if (warp < EPI0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Both CTAs' bytes complete on the leader's barrier.  A stage is loaded
      // again once the MMAs that read it are done, which they are only after
      // that barrier's phase, so no byte lands in an earlier one.
      const CUtensorMap* tw = GATED && rank == 1 ? &tmW1 : &tmW0;
      if (lane == 0) {
        int s = 0;
        uint32_t par = 0;  // of the stage's current phase
        long issued = 0;
        bool ok = true;
        for (int tile = pair_id; ok && tile < n_tiles; tile += n_pairs) {
          const int m0 = tile / tiles_n * 256 + int(rank) * 128;
          const int nt = tile % tiles_n;
          const int w0 = GATED ? nt * 128 : nt * 256 + int(rank) * (HALVES ? 64 : 128);
          constexpr int WH = GATED || !HALVES ? 64 : 128;  // weight rows between the halves
          for (int kb = 0; kb < nkb; ++kb) {
            ok = wait_s(&empty[s], par ^ 1u, abort_flag);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (A_BYTES + B_BYTES));
            const uint32_t bar = mapa(smem_u32(&full[s]), 0);
            tma_load<2>(smem_u32(sm + s * A_BYTES), &tmA, kb * BK, m0, bar);
            const uint32_t bs = smem_u32(sm + OFF_B + s * B_BYTES);
            tma_load<2>(bs, tw, kb * BK, w0, bar);
            tma_load<2>(bs + W_BOX * BK, tw, kb * BK, w0 + WH, bar);
            ++issued;
            if (++s == S) { s = 0; par ^= 1u; }
          }
        }
        // the last stages' MMAs: no arrival is under way when the CTAs part
        for (int i = 0; ok && i < S; ++i) {
          ok = wait_s(&empty[s], par ^ 1u, abort_flag);
          if (++s == S) { s = 0; par ^= 1u; }
        }
        // after an expired wait: the copies in flight (the peer's complete here
        // too, and it stays until the final cluster barrier)
        if (!ok && rank == 0)
          for (long j = issued > S ? issued - S : 0; j < issued; ++j)
            wait_s(&full[j % S], uint32_t((j / S) & 1), nullptr);
      }
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint64_t a_desc = sw128_desc(smem_u32(sm)), b_desc = sw128_desc(smem_u32(sm + OFF_B));
      // One thread.  An MMA is accepted when the one before it is almost done,
      // so between two k-blocks there is one MMA's time for everything else:
      // whether the next k-block may start is asked before this one's last
      // MMA, and the stage is released after the next one's first.
      if (elect_one()) {
      int s = 0, last = -1;
      uint32_t par = 0, it = 0;
      bool ok = true;
      constexpr int H = HALVES ? 2 : 1;
      for (int tile = pair_id; ok && tile < n_tiles; tile += n_pairs) {
        for (int kb = 0; ok && kb < nkb; ++kb, ++it) {
          const int b = int(it & 1);
          const uint32_t acc_par = ((it >> 1) & 1) ^ 1u;
          const uint64_t ad = a_desc + uint64_t(s * (A_BYTES >> 4));
#pragma unroll
          for (int h = 0; h < H; ++h) {
            if (h == 0) ok = wait_s(&full[s], par, abort_flag);
            ok = ok && wait_s(&acc_empty[2 * b + h], acc_par, abort_flag);
            if (!ok) break;
            fence_after_sync();
            const uint64_t bd = b_desc + uint64_t(s * (B_BYTES >> 4) + h * (64 * BK >> 4));
            const uint32_t d = tmem + uint32_t(256 * b + 128 * h);
            mma<2>(d, ad, bd, idesc(256, MN), 0);
            mma<2>(d, ad + 2, bd + 2, idesc(256, MN), 1);
            mma<2>(d, ad + 4, bd + 4, idesc(256, MN), 1);
            mma<2>(d, ad + 6, bd + 6, idesc(256, MN), 1);
            commit<2>(&acc_full[2 * b + h]);
            if (h == H - 1) commit<2>(&empty[s]);
          }
          if (++s == S) { s = 0; par ^= 1u; }
        }
      }
      commit<2>(drain);
      }
      __syncwarp();
      warp_wait(drain, 0, nullptr);
    } else if (warp == 2) {
      // ---------------------------------------------------------- scales
      // Word by word with cp.async (rows of any alignment): each lane four
      // tokens' scales of a k-block, lanes 0 and 1 the weight blocks' (gated:
      // of gate and up), CH k-blocks to a barrier.
      const uint32_t sc = smem_u32(sm + OFF_SCALE) + 4 * lane;
      int tile = pair_id, kb = nkb;
      const float *pa = nullptr, *pw = nullptr;
      int m = 0;
      tile -= n_pairs;
      for (uint32_t it = 0;; ++it) {
        if (kb == nkb) {
          tile += n_pairs;
          if (tile >= n_tiles) {
            if (it % CH != 0) cp_async_arrive(&sc_full[it / CH & 1]);
            break;
          }
          const int nt = tile % tiles_n;
          m = tile / tiles_n * 256 + int(rank) * 128 + lane;
          pa = as + m;
          pw = lane == 0 ? ws0 + size_t(GATED ? nt : 2 * nt) * nkb
                         : (GATED ? ws1 + size_t(nt) * nkb : ws0 + size_t(min(2 * nt + 1, nblk - 1)) * nkb);
          kb = 0;
        }
        if (it % CH == 0 && !__all_sync(0xffffffffu, wait_s(&sc_empty[it / CH & 1], (it / (2 * CH) & 1) ^ 1u, abort_flag)))
          break;
        const uint32_t d = sc + it % (2 * CH) * (SLOT * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m + 32 * i < M) cp_async4(d + 128 * i, pa + 32 * i);
        if (lane < 2) cp_async4(d + 512, pw);
        pa += M;
        ++pw;
        ++kb;
        if (it % CH == CH - 1) cp_async_arrive(&sc_full[it / CH & 1]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HI));
    const int quad = warp & 3, h = (warp - EPI0) >> 2;
    const int r = 32 * quad + lane;
    const uint32_t tm_row = tmem + uint32_t((GATED && !HALVES ? 64 : 128) * h) + (uint32_t(32 * quad) << 16);
    auto col = [](int c) { return uint32_t(c + (GATED && !HALVES && c >= 64 ? 64 : 0)); };
    uint32_t it = 0;
    int ti = 0;
    bool ok = true;
    const float* sc = reinterpret_cast<const float*>(sm + OFF_SCALE);
    const uint32_t free0 = mapa(smem_u32(&acc_empty[HALVES ? h : 0]), 0);  // the leader's, of buffer 0
    for (int tile = pair_id; ok && tile < n_tiles && !*abort_flag; tile += n_pairs, ++ti) {
      const int gm = tile / tiles_n * 256 + int(rank) * 128 + r;
      const int nt = tile % tiles_n;
      const bool in = gm < M;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int b = int(it & 1);
        if (it % CH == 0) {
          ok = __all_sync(0xffffffffu, wait_s(&sc_full[it / CH & 1], it / (2 * CH) & 1, abort_flag));
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, wait_s(&acc_full[2 * b + (HALVES ? h : 0)], (it >> 1) & 1, abort_flag));
        if (!ok) break;
        fence_after_sync();
        const uint32_t t = tm_row + uint32_t(256 * b);
        uint32_t v[2][CW];
        tmem_ld(t, v[0]);
        const float* sl = sc + it % (2 * CH) * SLOT;
        const float s0 = sl[r] * sl[GATED ? 128 : 128 + h], s1 = GATED ? sl[r] * sl[129] : s0;
        if (it % CH == CH - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_empty[it / CH & 1]);
        }
#pragma unroll
        for (int c = 0; c < 128 / CW; ++c) {
          wait_ld();
          if (c < 128 / CW - 1) {
            tmem_ld(t + col(CW * (c + 1)), v[(c + 1) & 1]);
          } else {  // the last read is done: the buffer is free
            if (lane == 0) arrive_cluster(free0 + uint32_t(16 * b));
          }
          const float sc2 = GATED && c >= 64 / CW ? s1 : s0;
          const float2 s2 = make_float2(sc2, sc2);
#pragma unroll
          for (int j = 0; j < CW / 2; ++j)
            acc[CW / 2 * c + j] = __ffma2_rn(
                make_float2(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1])), s2, acc[CW / 2 * c + j]);
        }
      }
      if (!ok) break;
      if constexpr (!GATED) {
        const int n0 = nt * 256 + 128 * h;
        const bool vec = (N % 16) == 0 && (reinterpret_cast<uintptr_t>(y) & 31) == 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int gn = n0 + 32 * c;
          if (gn >= N) break;
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = from_f2<T>(acc[16 * c + j]);
          if (vec) {
            if (in) {
              T* yr = y + size_t(gm) * N + gn;
              st_global_v8(yr, o);
              if (gn + 16 < N) st_global_v8(yr + 16, o + 8);
            }
          } else {
            // rows of any alignment: through shared memory, a row's 32 columns by the 32 lanes
            uint16_t* stg = reinterpret_cast<uint16_t*>(sm + OFF_STG) + (warp - EPI0) * 32 * STG_LD;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) *reinterpret_cast<uint32_t*>(stg + lane * STG_LD + 2 * j) = o[j];
            __syncwarp();
            uint16_t* y16 = reinterpret_cast<uint16_t*>(y);
            const int row0 = gm - lane, rows = min(32, M - row0);
            if (gn + lane < N)
              for (int i = 0; i < rows; ++i) y16[size_t(row0 + i) * N + gn + lane] = stg[i * STG_LD + lane];
          }
        }
      } else {
        // acc[0 .. 31]: gate of columns 64 h + [0, 64), acc[32 .. 63]: up
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          acc[j] = make_float2(silu(acc[j].x) * acc[32 + j].x, silu(acc[j].y) * acc[32 + j].y);
          m = max_nan(m, max_nan(fabsf(acc[j].x), fabsf(acc[j].y)));
        }
        // the block's other 64 columns are the other half's: exchange the abs-max
        float* am = reinterpret_cast<float*>(sm + OFF_AMAX) + (ti & 1) * 256;
        am[h * 128 + r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(exch);
        ok = __all_sync(0xffffffffu, wait_s(exch, uint32_t(ti & 1), abort_flag));
        if (!ok) break;
        m = block_amax(max_nan(m, am[(h ^ 1) * 128 + r]));
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
  }

  fence_before_sync();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory
  if (warp == 1) {
    fence_after_sync();
    tmem_free<2>(tmem, TMEM_COLS);
  }
}

}  // namespace wide

// ===================================================================== narrow
// Few tokens: the time is that of reading the weights once.  A CTA takes 128
// weight rows (gated: 128 gate and 128 up rows) as the MMA's M, TN tokens as
// its N, and 1 / cluster_size of the depth.  Its thread (lane quadrant, lane)
// holds one weight row's sums of the TN tokens.  At the end every CTA writes
// its sums to its shared memory, and the warps of all the cluster's CTAs take
// tokens in turn, adding the ranks' sums in rank order through distributed
// shared memory: no workspace, no atomics, the same bits every time.
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
  static constexpr int S = TN == 128 ? 3 : GATED ? (TN == 64 ? 2 : 3) : (TN == 64 ? 4 : TN == 32 ? 5 : 6);
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
              const __grid_constant__ CUtensorMap tmW1, const float* __restrict__ as, const float* __restrict__ ws0,
              const float* __restrict__ ws1, int M, int N, int nkb, T* __restrict__ y, uint8_t* __restrict__ q,
              float* __restrict__ qs) {
  using C = Cfg<GATED, TN>;
  constexpr int S = C::S, NW = C::NW, KC = C::KC;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  volatile uint32_t* slot = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank()), ranks = int(cluster_size());
  const int wb = int(blockIdx.x) / ranks;  // block of 128 weight rows (and of output columns)
  const int m0 = int(blockIdx.y) * TN;
  const int kb_lo = int(int64_t(nkb) * rank / ranks), kb_hi = int(int64_t(nkb) * (rank + 1) / ranks);

  if (threadIdx.x == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmW0);
    if (GATED) prefetch_map(&tmW1);
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc<1>(smem_u32(const_cast<uint32_t*>(slot)), C::COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *slot;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    int issued = 0;
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      const int i = kb - kb_lo, s = i % S;
      if (!warp_wait(&empty[s], uint32_t((i / S) & 1) ^ 1u, abort_flag)) break;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&full[s]), st = smem_u32(sm + s * C::STAGE);
        mbar_arrive_expect_tx(&full[s], C::STAGE);
        tma_load<1>(st, &tmW0, kb * BK, wb * 128, bar);
        if (GATED) tma_load<1>(st + C::W_BYTES, &tmW1, kb * BK, wb * 128, bar);
        tma_load<1>(st + NW * C::W_BYTES, &tmA, kb * BK, m0, bar);
      }
      __syncwarp();
      issued = i + 1;
    }
    if (warp_flag(abort_flag) && lane == 0)
      for (int j = issued > S ? issued - S : 0; j < issued; ++j)
        mbar_wait_bounded(&full[j % S], uint32_t((j / S) & 1), nullptr);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      const int i = kb - kb_lo, s = i % S, b = i & 1;
      if (!warp_wait(&full[s], uint32_t((i / S) & 1), abort_flag) ||
          !warp_wait(&acc_empty[b], uint32_t((i >> 1) & 1) ^ 1u, abort_flag))
        break;
      fence_after_sync();
      if (lane == 0) {
        const uint32_t st = smem_u32(sm + s * C::STAGE);
        const uint64_t ad = sw128_desc(st + NW * C::W_BYTES);
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const uint64_t wd = sw128_desc(st + p * C::W_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma<1>(tmem + uint32_t((b * NW + p) * TN), wd + uint64_t(2 * kk), ad + uint64_t(2 * kk), idesc(128, TN), kk != 0);
        }
        commit<1>(&acc_full[b]);
        commit<1>(&empty[s]);
      }
      __syncwarp();
    }
    if (lane == 0) {
      commit<1>(drain);
      mbar_wait_bounded(drain, 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    float2 acc[NW][TN / 2];
#pragma unroll
    for (int p = 0; p < NW; ++p)
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) acc[p][j] = make_float2(0.f, 0.f);
    // scales a_scale w_scale of KC k-blocks, in the warp's own rows of shared
    // memory; the token scales of the next KC are already in registers
    float* sc = reinterpret_cast<float*>(sm + C::OFF_SC) + warp * KC * NW * TN;
    constexpr int PL = KC * TN / 32;
    float pre[PL], pw[NW];
    const float* w0 = ws0 + size_t(wb) * nkb;
    const float* w1 = GATED ? ws1 + size_t(wb) * nkb : nullptr;
    auto fetch = [&](int kb) {
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const int k = (e * 32 + lane) / TN, n = (e * 32 + lane) % TN;
        pre[e] = kb + k < kb_hi && m0 + n < M ? __ldg(as + size_t(kb + k) * M + m0 + n) : 0.f;
      }
      pw[0] = lane < KC && kb + lane < kb_hi ? __ldg(w0 + kb + lane) : 0.f;
      if constexpr (GATED) pw[1] = lane < KC && kb + lane < kb_hi ? __ldg(w1 + kb + lane) : 0.f;
    };
    fetch(kb_lo);
    const uint32_t tm_row = tmem + (uint32_t(32 * warp) << 16);
    for (int kb = kb_lo; kb < kb_hi; ++kb) {
      const int i = kb - kb_lo, b = i & 1, kc = i % KC;
      if (kc == 0) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < PL; ++e) {
          const int k = (e * 32 + lane) / TN, n = (e * 32 + lane) % TN;
#pragma unroll
          for (int p = 0; p < NW; ++p) sc[(k * NW + p) * TN + n] = pre[e] * __shfl_sync(0xffffffffu, pw[p], k);
        }
        __syncwarp();
        fetch(kb + KC);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[b], uint32_t((i >> 1) & 1), abort_flag))) break;
      fence_after_sync();
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        const float* scp = sc + (kc * NW + p) * TN;
        constexpr int CW = TN < 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < TN / CW; ++c) {
          uint32_t v[CW];
          tmem_ld(tm_row + uint32_t((b * NW + p) * TN + c * CW), v);
          wait_ld();
          if (p == NW - 1 && c == TN / CW - 1) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
          }
#pragma unroll
          for (int j = 0; j < CW / 4; ++j) {
            const float4 s4 = *reinterpret_cast<const float4*>(scp + c * CW + 4 * j);
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
    if (!warp_flag(abort_flag)) {
      float* part = reinterpret_cast<float*>(sm);
#pragma unroll
      for (int p = 0; p < NW; ++p)
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
          part[(p * TN + 2 * j) * 128 + 32 * warp + lane] = acc[p][j].x;
          part[(p * TN + 2 * j + 1) * 128 + 32 * warp + lane] = acc[p][j].y;
        }
    }
  }

  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 5) {
    fence_after_sync();
    tmem_free<1>(tmem, C::COLS);
  }
  // ---- a warp per token: lane l holds weight rows 4 l .. 4 l + 3
  const uint32_t part = smem_u32(sm);
  const int n0 = wb * 128 + 4 * lane;
  const int tokens = min(TN, M - m0);
  for (int n = rank * (NT / 32) + warp; n < tokens; n += ranks * (NT / 32)) {
    float2 v[NW][2];
#pragma unroll
    for (int p = 0; p < NW; ++p) v[p][0] = v[p][1] = make_float2(0.f, 0.f);
    for (int k = 0; k < ranks; ++k)
#pragma unroll
      for (int p = 0; p < NW; ++p) {
        float4 f;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                     : "r"(mapa(part + uint32_t(((p * TN + n) * 128 + 4 * lane) * 4), uint32_t(k))));
        v[p][0] = __fadd2_rn(v[p][0], make_float2(f.x, f.y));
        v[p][1] = __fadd2_rn(v[p][1], make_float2(f.z, f.w));
      }
    const size_t row = size_t(m0 + n) * N;
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
      const float2 z0 = make_float2(silu(v[0][0].x) * v[1][0].x, silu(v[0][0].y) * v[1][0].y);
      const float2 z1 = make_float2(silu(v[0][1].x) * v[1][1].x, silu(v[0][1].y) * v[1][1].y);
      // weight rows past N were read as zeros: z = 0 there
      float m = max_nan(max_nan(fabsf(z0.x), fabsf(z0.y)), max_nan(fabsf(z1.x), fabsf(z1.y)));
      m = n0 < N ? m : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = block_amax(m);
      const Quotient quo(m);
      if (n0 < N) *reinterpret_cast<uint32_t*>(q + row + n0) = cvt_e4m3x4(quo(z0), quo(z1));
      if (lane == 0) qs[size_t(wb) * M + m0 + n] = block_scale(m);
    }
  }
  cluster_sync();  // the other ranks have read this CTA's sums
}

}  // namespace narrow

// ------------------------------------------------------------------ host
static PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
static std::once_flag g_encode_once;

static bool get_encoder() {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult r;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) == cudaSuccess &&
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

static int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

static int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K <= 0) return QUAROT_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if (K % 16 != 0 || K > (int64_t(1) << 20) || M > lim || N > lim) return QUAROT_ERR_UNSUPPORTED;
  if (((M + 255) / 256) * ((N + 127) / 128) >= (int64_t(1) << 31) - 512) return QUAROT_ERR_UNSUPPORTED;
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
  CUtensorMap ta, t0, t1;
  if (!make_map(&ta, p.a, p.M, p.K, a_box) || !make_map(&t0, p.w0, p.N, p.K, w_box)) return QUAROT_ERR_CUDA;
  if (p.w1 == nullptr) t1 = t0;
  else if (!make_map(&t1, p.w1, p.N, p.K, w_box)) return QUAROT_ERR_CUDA;
  if (!smem_attr_once(kern, smem, attr)) return QUAROT_ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = p.st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(cluster);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ta, t0, t1, p.as, p.ws0, p.ws1, int(p.M), int(p.N),
                                           int((p.K + BK - 1) / BK), y, p.q, p.qs);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? QUAROT_OK : QUAROT_ERR_LAUNCH;
}

template <bool GATED, int TN, typename T>
static int launch_narrow(const Args& p, int cluster) {
  static AttrCache attr;
  const unsigned wbs = unsigned((p.N + 127) / 128), mts = unsigned((p.M + TN - 1) / TN);
  return launch(p, narrow::narrow_kernel<GATED, TN, T>, attr, dim3(wbs * unsigned(cluster), mts), narrow::NT, cluster,
                narrow::Cfg<GATED, TN>::SMEM, TN, 128, static_cast<T*>(p.y));
}

template <bool GATED, typename T>
static int run(const Args& p) {
  if (!get_encoder()) return QUAROT_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return QUAROT_ERR_CUDA;
  constexpr int kNarrow = GATED ? 64 : 128;
  const int64_t wbs = (p.N + 127) / 128, nkb = (p.K + BK - 1) / BK;
  if (p.M <= kNarrow && wbs <= (int64_t(1) << 27)) {
    int cl = 1;
    while (cl < 8 && wbs * cl * 2 <= 2 * sms && nkb / (2 * cl) >= 4) cl *= 2;
    if (p.M <= 16) return launch_narrow<GATED, 16, T>(p, cl);
    if (p.M <= 32) return launch_narrow<GATED, 32, T>(p, cl);
    if (p.M <= 64) return launch_narrow<GATED, 64, T>(p, cl);
    if constexpr (!GATED) return launch_narrow<GATED, 128, T>(p, cl);
  }
  if (sms < 2) return QUAROT_ERR_UNSUPPORTED;
  static AttrCache attr;
  constexpr int TN = GATED ? 128 : 256;
  const int64_t tiles = ((p.M + 255) / 256) * ((p.N + TN - 1) / TN);
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch(p, wide::wide_kernel<GATED, T>, attr, dim3(unsigned(2 * pairs)), wide::NT, 2, wide::SMEM, 128, wide::W_BOX,
                static_cast<T*>(p.y));
}

}  // namespace gemm
}  // namespace fp8
}  // namespace quarot

using namespace quarot;

bool quarot::take_fp8_error_word(unsigned int* word) {
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(word, g_error_word, sizeof(zero)) != cudaSuccess) return false;
  return *word == 0 || cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) == cudaSuccess;
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
