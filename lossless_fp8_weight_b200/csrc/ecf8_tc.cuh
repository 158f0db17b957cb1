// Thin wrappers of the sm_100a instructions the tensor-core kernels use:
// mbarriers, TMA tile loads, tcgen05 (tensor memory, matrix products).
// Every wait for an mbarrier has a limit in clock cycles, after which it fails,
// marks the CTA as failed and lets every other such wait of the CTA fail as well.
// The others end by construction: every thread arrives at the barriers of the
// CTA and the cluster whether it has failed or not, a kernel that is waited for
// has what it needs to end, and tensor memory is freed by CTAs that do.
#ifndef ECF8_TC_CUH_
#define ECF8_TC_CUH_

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ecf8_tc {

constexpr long long kWaitCycles = 4000000000ll;  // about two seconds

struct Waits {
  volatile int* failed;  // in shared memory
  long long limit;       // clock cycles of a wait
};

__device__ inline uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ inline void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ inline void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ inline void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ inline void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrives on the barrier at this offset of another CTA of the cluster.
__device__ inline void mbar_arrive_at(uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n"
      " mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(bar),
      "r"(rank)
      : "memory");
}
// CLUSTER: another CTA's arrivals are among those waited for.
template <bool CLUSTER = false>
__device__ inline bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
// Waits for the phase of this parity to complete; false when the limit ran out or another wait of the CTA has failed.
// The clock is read rarely: waiting warps should leave the issue slots to the working ones.
template <bool CLUSTER = false>
__device__ inline bool mbar_poll(uint32_t bar, uint32_t parity, const Waits& w) {
  if (mbar_try<CLUSTER>(bar, parity)) return true;
  const long long start = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try<CLUSTER>(bar, parity)) return true;
    if (*w.failed) return false;
    if (clock64() - start > w.limit) {
      *w.failed = 1;
      return false;
    }
  }
}
// The same for a whole warp, with one answer for all lanes: each has a limit of its own, and a warp that parted could not
// elect a lane any more.  Every lane polls, which suits a warp that loads or issues products (with one lane polling 8192
// rows of 14336x4096 took 1010 us, 890 so).
template <bool CLUSTER = false>
__device__ inline bool mbar_wait_lanes(uint32_t bar, uint32_t parity, const Waits& w) {
  const bool ok = __all_sync(~0u, mbar_poll<CLUSTER>(bar, parity, w));
  __syncwarp();
  return ok;
}
// One lane polls: in a warp that widens, 32 take turns (some 500 clocks a wait, measured).
__device__ inline bool mbar_wait(uint32_t bar, uint32_t parity, const Waits& w) {
  bool ok = true;
  if (threadIdx.x % 32 == 0) ok = mbar_poll(bar, parity, w);
  ok = __all_sync(~0u, ok);
  __syncwarp();  // what the lane that waited may read, all may
  return ok;
}
// The same for what has to end before a CTA that has failed does.
__device__ inline void mbar_wait_out(uint32_t bar, uint32_t parity, const Waits& w) {
  if (threadIdx.x % 32 == 0) {
    const long long start = clock64();
    while (!mbar_try(bar, parity) && clock64() - start < w.limit) {
    }
  }
  __syncwarp();
}

// True in one lane of a converged warp.  Around it the warp stays together, so that addresses and descriptors are
// computed once for the warp: in a branch of one lane every product's operands are moved over one by one first, which
// took 230 clocks for four products.
__device__ inline bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}

__device__ inline void tma_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ inline void tma_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// P: CTAs that act as one, 1 or 2.  With 2, both CTAs of a pair allocate and free; one thread of the even CTA
// issues the products, whose 128 output rows a CTA lie in its own tensor memory and whose other operand comes half
// from each CTA's shared memory; a commit arrives on the barriers at this offset of every CTA in `mask`.
template <int P>
__device__ inline void tmem_alloc(uint32_t smem_dst, uint32_t columns) {
  if constexpr (P == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns)
                 : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns)
                 : "memory");
}
template <int P>
__device__ inline void tmem_release_permit() {
  if constexpr (P == 1) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <int P>
__device__ inline void tmem_free(uint32_t tmem, uint32_t columns) {
  if constexpr (P == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}
__device__ inline void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ inline void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// shared memory written by threads, read by the matrix unit or TMA
__device__ inline void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Arrives on bar once every matrix product issued so far by this thread has ended.
template <int P>
__device__ inline void mma_commit(uint32_t bar, uint32_t mask) {
  if constexpr (P == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::
                     "r"(bar),
                 "h"((uint16_t)mask)
                 : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], 128 * P x n x 16.
template <int P>
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (P == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[smem] * B[smem], 128 x n x 16.
__device__ inline void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory operand of 128-byte rows (64 values of 16 bits), the reduction along the row,
// 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ inline uint64_t desc_k128(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}

// Shared-memory operand of 128-byte rows along the output dimension (64 values of 16 bits), one row for each term
// of the reduction, 128-byte swizzle: 8-row groups 1024 bytes apart, the next 64 values `next` bytes apart.
__device__ inline uint64_t desc_mn128(uint32_t addr, uint32_t next) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(next >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kTransposeA = 1u << 15, kTransposeB = 1u << 16;  // in the instruction descriptor: A, B is desc_mn128

// 16-bit inputs of one type, float32 sums, m x n; both operands with the reduction contiguous.
__host__ __device__ inline uint32_t idesc_f16(bool bf16, uint32_t m, uint32_t n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (n >> 3) << 17 | (m >> 4) << 24;
}

__device__ inline void tmem_st32(uint32_t tmem, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(tmem),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ inline void tmem_st16(uint32_t tmem, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(tmem),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// The wait is part of the statement: nothing may read v between the two.  The lanes have to be together, which after a
// branch of some (the columns or rows that exist) they need not be.
__device__ inline void tmem_ld16(uint32_t tmem, float (&v)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(tmem)
      : "memory");
}
__device__ inline void tmem_ld8(uint32_t tmem, float (&v)[8]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(tmem)
      : "memory");
}

// A kernel launched to overlap its predecessor waits for that one's end and results with the first; the predecessor
// lets it start with the second.
__device__ inline void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ inline void start_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ inline uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ inline void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared-memory location in another CTA of the cluster, and loads from it.  The loads are not
// volatile, so that a thread has many in flight: they are for what does not change after a cluster_sync.
__device__ inline uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// Adds up to 8 CTAs' four floats at this offset, in the order of their ranks.
__device__ inline float4 cluster_sum4(uint32_t addr, uint32_t count) {
  float4 v[8];
#pragma unroll
  for (uint32_t r = 0; r < 8; ++r) {
    v[r] = make_float4(0, 0, 0, 0);
    if (r < count)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                   : "r"(cluster_map(addr, r)));
  }
  float4 s = v[0];
#pragma unroll
  for (uint32_t r = 1; r < 8; ++r)
    if (r < count) s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
  return s;
}
__device__ inline void cluster_stu(uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile("{\n .reg .u32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.u32 [a], %2;\n}" ::"r"(addr),
               "r"(rank), "r"(v)
               : "memory");
}

}  // namespace ecf8_tc

#endif  // ECF8_TC_CUH_
