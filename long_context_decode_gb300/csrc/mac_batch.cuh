// mac_batch.cuh -- parameter blocks and launchers of the calls on a batch of
// new tokens: page tables and slots, the cache writer, chunk attention.
#pragma once

#include <atomic>

#include "mac_common.cuh"

namespace mac {

constexpr int kPage = 16;         // tokens per page of a paged cache

struct TablesParams {
  int B, T;
  int paged;
  int64_t limit;                  // longest length a request may reach
  int64_t capacity;               // contiguous: slots per request
  int max_pages, n_pages;
  int32_t *table, *free_pages;
  const int32_t *n_free_in;
  int32_t *n_free_out;
  const int32_t *flags, *len_in, *new_len;
  int32_t *len_out, *q_start, *pos;
  int64_t *slot;
  uint32_t *status;
};

struct WriteParams {
  int T, Hq, Hkv, rope_mode, paged;
  int64_t capacity;               // contiguous: slots per request
  int64_t n_slots;                // slots of the whole cache
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements
  const int32_t *pos;
  const int64_t *slot;
  void *cache_k, *cache_v, *q_out;
  uint32_t *status;
  unsigned long long rope_f[kHeadDim / 2];
};

// Chunk attention.  A unit is (request b, KV head g, tile i of the request's
// new tokens): ROWS packed rows, token-major, the G heads of a token next to
// one another, so that the group loads each K/V tile once.
struct ChunkParams {
  int B, Hq, Hkv, G, T;
  float q_scale;                  // log2(e)/sqrt(d)
  int64_t max_len;
  KvView kv;
  const void *q;
  const int32_t *q_start, *seq_len;
  void *out;
  float *lse;                     // or null
  uint32_t *status;
  int4 *notes;                    // [kChunkGrid] the cut unit whose first tile a CTA holds
  float *part;                    // [2 * grid][part_rows][kChunkStride]
  int part_rows;
  long long wait_limit;           // cycles that a wait on a copy, a product or another role may take
  int withhold;                   // run-out test only: the stage use (>= 0) whose copy is never issued
};

// Most CTAs of a launch (one per SM).  The workspace is laid out for as many,
// so that its size (71 MB of bf16 pieces at most, of which 152 SMs use 42) can
// be asked where there is no device.
constexpr int kChunkGrid = 256;
// What the plan of a chunk attention launch counts with, per kernel: rows of
// a unit, keys of a tile, and costs: a unit's start and end, a key tile of
// a unit and of one of at most half the rows, the least worth a CTA of its
// own, and what cutting units costs a launch (partials, notes, the merge).
// bf16, in quarters of a full unit's tile (2900 cycles): half the rows compute
// half as much per tile but copy as much; a start and end cost as three tiles.
// fp32: in tiles (7200 cycles).
struct ChunkBf16 {
  static constexpr int kRows = 256, kKeys = 128;
  static constexpr int kStart = 12, kTile = 4, kTileHalf = 3, kMinShare = 16, kCut = 35;
  static constexpr bool kHalves = true;  // units of half the rows, where there are CTAs for all of them
};
struct ChunkF32 {
  static constexpr int kRows = 128, kKeys = 64;
  static constexpr int kStart = 3, kTile = 1, kTileHalf = 1, kMinShare = 4, kCut = 4;
  static constexpr bool kHalves = false;
};
constexpr int kChunkStride = kHeadDim + 8;  // floats per row of a partial: o[d], m, l, and to a multiple of 32 bytes
constexpr int kMaxTokens = 1 << 24;

// Launch with programmatic stream serialization: the kernel may start while
// the previous one on the stream finishes, and waits (griddep_wait) before it
// touches global memory.
template <typename K, typename... A>
cudaError_t launch_dependent(K *kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Shared memory limit of a chunk kernel, set once per device; `smem` bytes and
// at least `regs` registers per thread are what its launch counts on.
// `done`: the kernel's own flags, one per device.
using DeviceFlags = std::atomic<bool>[64];
template <typename K>
cudaError_t prepare_chunk(K *kernel, DeviceFlags &done, int smem, int regs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes fa;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
      (e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess)
    return e;
  if (fa.numRegs < regs) return cudaErrorInvalidValue;
  if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

// The attention kernels, `grid` CTAs (one per SM).
cudaError_t launch_chunk_f32(const ChunkParams &p, int grid, cudaStream_t s);
cudaError_t launch_chunk_bf16(const ChunkParams &p, int grid, cudaStream_t s);
// The cut units of an attention launch of `grid` CTAs.
cudaError_t launch_chunk_merge(const ChunkParams &p, int grid, bool f32, cudaStream_t s);

cudaError_t launch_tables(const TablesParams &p, cudaStream_t s);
cudaError_t launch_write(const WriteParams &p, int dtype, cudaStream_t s);

}  // namespace mac
