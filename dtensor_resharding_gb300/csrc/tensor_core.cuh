// Blackwell's asynchronous units as device functions: mbarriers with bounded waits, TMA tile loads, tensor memory and
// the tcgen05 matrix product of 8-bit values.
#pragma once
#include <cuda.h>

#include "ops_common.cuh"

namespace reshard {
namespace ops {

#ifdef __CUDACC__

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 4 bytes to shared memory, and an arrival at `bar` when this thread's copies so far are there.
__device__ __forceinline__ void copy4(uint32_t to, const void *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void bar_arrive_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Every wait is bounded: a try suspends the thread for some microseconds at most, and after kTries of them (seconds) the
// wait gives up, marks the CTA (so that what it computed is not stored) and sets the status word. The loop is written
// out because waits are on the path of every block: a clock read and a call in it cost more than the block's products.
constexpr uint32_t kTries = 1u << 20;
struct Stop {
  volatile int *cta;    // shared memory
  int *status;          // global memory
};
__device__ __forceinline__ bool bar_spin(uint32_t bar, uint32_t parity, uint32_t tries) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
               "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra done;\n"
               " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra again;\n"
               "done:\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(bar), "r"(parity), "r"(tries) : "memory");
  return ok;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Stop &s) {
  const bool ok = bar_spin(bar, parity, kTries);
  if (!ok) {
    *s.cta = 1;
    atomicOr(s.status, 1);
  }
  return ok;
}
// The same for what is in flight when a CTA stops.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) { bar_spin(bar, parity, kTries); }

// x (bytes) is a multiple of 16; what lies outside the tensor reads as 0.
__device__ __forceinline__ void tma_2d(uint32_t to, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// Four rows of a matrix, each as a tensor map whose box is one row describes it, one below the other.
__device__ __forceinline__ void tma_rows4(uint32_t to, const CUtensorMap *map, int x, const int (&y)[4], uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
               ::"r"(to), "l"(map), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns) {   // a whole warp; a power of two, 32 .. 512
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {    // the warp that allocated
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand of rows of 128 bytes as a 128-byte-swizzled TMA box leaves them, K along the row: 8 rows are
// 1024 bytes; the tile starts on a 1024-byte boundary. A step of 32 values along K adds 2 (x 16 bytes) to the address.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// e4m3 x e4m3 -> fp32, both operands with K along the rows, 128 rows of A and n rows of B (a multiple of 16, to 256).
__device__ __forceinline__ uint32_t instruction(int n) { return 1u << 4 | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24; }

// D[tmem] = A B^T over 32 values of K, added to D where `add`. One thread.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// Arrives at `bar` when every product that this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Columns of the warp's 32 lanes of tensor memory; the values are there after tmem_loaded(), which the compiler keeps
// before every use of them.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// A tile of shared memory to global memory by the copy engine: what lies outside the tensor is not written. Writes to
// the tile come before it by copy_fence() of their threads and a barrier. bulk_read(): the engine is done reading what
// this thread has handed over; bulk_done(): and writing it.
__device__ __forceinline__ void copy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t from, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(from) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ float shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory"); }
// What another CTA of the cluster holds at this CTA's shared address. Not a barrier to other loads: several are in flight.
__device__ __forceinline__ float cluster_f32(uint32_t addr, int rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ bool elect_one() {     // one lane of a converged warp
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p;
}

// Registers of a warpgroup's threads from here on; the shares of a CTA's warpgroups sum to what it was launched with.
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

#endif  // __CUDACC__

}  // namespace ops
}  // namespace reshard
