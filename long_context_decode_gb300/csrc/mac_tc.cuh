// mac_tc.cuh -- tensor core (tcgen05), packed fp32 and bounded-wait helpers of
// the chunk-attention kernels.
#pragma once

#include "mac_chunk.cuh"

namespace mac {

#ifdef __CUDACC__

// ---- tcgen05 ---------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One arrival on `bar` once the products issued so far have ended.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Shared memory descriptor, 128-byte swizzle: address / 16 and leading byte
// offset / 16 (bit 16) in the low word; in the high one, stride byte offset
// / 16 (groups of eight rows are 1024 bytes apart), version 1 (bit 46) and
// swizzle mode 2 (bit 61).  A tile is two halves of 64 columns, 128-byte rows: Q and K
// step 16 columns along a row (32 bytes); V, whose columns are the
// product's N, steps 16 rows (2048 bytes), its halves a leading offset apart.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

// Two arrivals at once (the stages of a key and a value tile).
__device__ __forceinline__ void tc_commit2(uint32_t bar0, uint32_t bar1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(bar0), "r"(bar1)
      : "memory");
}

// Instruction descriptor: fp32 sums (bit 4), bf16 A and B (bits 7, 10), B
// along N where asked (bit 16), N/8 from bit 17, M/16 (M = 128) from bit 24.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128 >> 4) << 24);
}

__device__ __forceinline__ void tc_ld32(float *r, uint32_t addr) {
  uint32_t *u = reinterpret_cast<uint32_t *>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(u[0]),
      "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
      "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]),
      "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]),
      "r"(u[29]), "r"(u[30]), "r"(u[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(u[0]),
      "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
      "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(float *r, uint32_t addr) {
  uint32_t *u = reinterpret_cast<uint32_t *>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(addr));
}
// Registers that a load has filled are used after the wait only.
__device__ __forceinline__ void tc_loaded16(float *r) {
  asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
               "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]));
}
__device__ __forceinline__ void tc_loaded32(float *r) {
  asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
               "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]));
  asm volatile("" : "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
               "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]));
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- packed fp32 -----------------------------------------------------------
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Waits that every role makes, a whole warp at a time.  After one has run out (or another role's
// has: *abort) all return false at once; the roles then walk through
// their loops without touching anything, so that their barriers still meet.
struct Waiter {
  int *abort;
  uint32_t *status;
  long long limit;
  bool dead;
  __device__ __forceinline__ bool operator()(unsigned long long *bar, uint32_t parity) {
    if (!__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity)) || dead) return slow(smem_addr(bar), parity);
    return true;
  }
  __device__ __forceinline__ bool slow(uint32_t bar, uint32_t parity) {
    if (dead) return false;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, (volatile int *)abort, limit))) {
      dead = true;
      *(volatile int *)abort = 1;
      set_status(status, MAC_DEV_WAIT_TIMEOUT);
      return false;
    }
    return true;
  }
};

// Before a CTA gives its shared memory and TMEM up, everything that writes or
// reads them has ended: the phase of `parity` of `bar`, waited for even after
// a wait has run out, and for about half a second whatever limit the other
// waits were given (a copy or product that was issued ends within microseconds).
constexpr long long kDrainLimit = 1LL << 30;
__device__ __forceinline__ bool drained(unsigned long long *bar, uint32_t parity) {
  const int never = 0;
  return mbar_wait_bounded(smem_addr(bar), parity, (volatile int *)&never, kDrainLimit);
}

// The warp that works out the pieces waits for whole pieces (room for the next
// ones, a piece's last tile), not for one copy or product, so its limit grows
// by 2^14 cycles with every key tile that it has posted (a tile takes 2900
// to 7200).  A role that is stuck gives up by its own limit and sets *abort.
constexpr int kTileLimitLog = 14;

// The pieces of a CTA, from the one warp that works them out to the warps of
// the other roles (`readers` of them): a short ring in shared memory.  The
// walk's code runs in one place only, ahead of its use; in every role it was
// out of the instruction cache each time and took 5000 cycles per piece.
template <typename P>
struct PieceRing {
  static constexpr uint32_t kSlots = 4;
  unsigned long long full[kSlots], empty[kSlots];
  P d[kSlots];
  __device__ void init(int readers) {
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(smem_addr(&full[i]), 1);
      mbar_init(smem_addr(&empty[i]), readers);
    }
  }
  // The i-th piece (a whole warp calls these); one with t0 == t1 ends the walk.
  __device__ void post(Waiter &wait, uint32_t i, const P &q) {
    const uint32_t s = i % kSlots;
    if (wait(&empty[s], (i / kSlots + 1) & 1) && (threadIdx.x & 31) == 0) {
      d[s] = q;
      mbar_arrive(smem_addr(&full[s]));
    }
    __syncwarp();
  }
  __device__ bool take(Waiter &wait, uint32_t &i, P &q) {
    const uint32_t s = i % kSlots;
    if (!wait(&full[s], i / kSlots & 1)) return false;
    ++i;
    q = d[s];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&empty[s]));
    return q.t1 > q.t0;
  }
};

__device__ __forceinline__ bool bad_page(const ChunkParams &p, int id) {
  return id < 0 || id >= p.kv.n_pages;
}

#endif  // __CUDACC__

}  // namespace mac
