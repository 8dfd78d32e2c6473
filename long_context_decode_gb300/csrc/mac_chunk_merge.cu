// mac_chunk_merge.cu -- the pieces of chunk attention's cut units.
//
// Pieces of disjoint keys with states (o, m, l), o and l relative to 2^m:
//   M = max m;  out = sum 2^(m - M) o / sum 2^(m - M) l;  lse = M ln 2 + ln sum.
// Every CTA reads the notes of all CTAs of the attention kernel and lays the
// cut units' rows out as items of one to four rows; the items are dealt to the
// warps of all CTAs in turn, and a warp has all loads of an item (eight pieces
// of a row, four of two rows or two of four) on their way at once, four dims
// per lane.  Bound by two trips to L2, the notes' and the pieces', and by the
// launch; after a long call the pieces come from HBM (40 MB, 13 us).
// Against a CTA for every eight rows of every CTA's note: nothing to merge
// 12 x 60 tokens at 1200 29.9 -> 27.4 us, few and short units 22 -> 20.3; four
// rows of 64 units in three pieces each 24.2 -> 25.3.  Two CTAs per SM leave
// 128 registers a thread: with four (64) it spilled, which took longer than
// all the rest (30 us where 24 bytes were spilled).
// (Merged by the CTA that finished a unit's last piece, 128 rows of five
// pieces took 60 us.)
#include <math.h>

#include "mac_chunk.cuh"

namespace mac {
namespace {

constexpr int kThr = 256, kPerSm = 2, kLoads = 8;
static_assert(kChunkGrid == kThr, "a thread reads a note");

// rows of an item of a unit in n pieces
__device__ __forceinline__ int item_rows(int n) { return n <= 2 ? 4 : n <= 4 ? 2 : 1; }

struct Unit {
  const float *part;  // of its first piece, row 0
  int64_t slot;       // floats per partial
  int4 note;          // first token, KV head, rows, last CTA
  int n;              // pieces
  __device__ const float *at(int row, int j) const { return part + (2 * j + (j == 0)) * slot + (int64_t)row * kChunkStride; }
  __device__ float2 state(int row, int j) const {
    return row < note.z && j < n ? __ldcg(reinterpret_cast<const float2 *>(at(row, j) + kHeadDim)) : make_float2(-INFINITY, 0.f);
  }
  __device__ float4 output(int row, int j) const {
    return row < note.z && j < n ? __ldcg(reinterpret_cast<const float4 *>(at(row, j)) + (threadIdx.x & 31)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
};

__device__ __forceinline__ void add(float4 &o, float w, float4 v) {
  o.x = fmaf(w, v.x, o.x);
  o.y = fmaf(w, v.y, o.y);
  o.z = fmaf(w, v.z, o.z);
  o.w = fmaf(w, v.w, o.w);
}

template <typename T>
__device__ __forceinline__ void finish(const ChunkParams &p, const Unit &u, int row, float4 o, float m, float l) {
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)(u.note.x + row / p.G) * p.Hq + u.note.y * p.G + row % p.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store_out((T *)p.out + at * kHeadDim + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// ROWS rows of a unit in at most kLoads / ROWS pieces
template <typename T, int ROWS>
__device__ __forceinline__ void merge_few(const ChunkParams &p, const Unit &u, int row) {
  constexpr int N = kLoads / ROWS;
  const int lane = threadIdx.x & 31;
  const float2 ml = lane < kLoads ? u.state(row + lane / N, lane % N) : make_float2(-INFINITY, 0.f);
  float4 v[ROWS][N];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) v[i][j] = u.output(row + i, j);
  float m = ml.x;
#pragma unroll
  for (int d = N / 2; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (m == -INFINITY) m = 0.f;
  const float w = ex2(ml.x - m);
  float l = w * ml.y;
#pragma unroll
  for (int d = N / 2; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N; ++j) add(o, __shfl_sync(0xffffffffu, w, i * N + j), v[i][j]);
    const float mi = __shfl_sync(0xffffffffu, m, i * N), li = __shfl_sync(0xffffffffu, l, i * N);
    if (row + i < u.note.z) finish<T>(p, u, row + i, o, mi, li);
  }
}

// a row of a unit in any number of pieces
template <typename T>
__device__ __forceinline__ void merge_many(const ChunkParams &p, const Unit &u, int row) {
  const int lane = threadIdx.x & 31;
  float4 v[kLoads];
  float2 ml = u.state(row, lane);
#pragma unroll
  for (int e = 0; e < kLoads; ++e) v[e] = u.output(row, e);
  float m = ml.x;
  for (int j = 32 + lane; j < u.n; j += 32) m = fmaxf(m, u.state(row, j).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (m == -INFINITY) m = 0.f;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < u.n; j0 += 32) {
    if (j0) ml = u.state(row, j0 + lane);
    const float w = ex2(ml.x - m);
    l = fmaf(w, ml.y, l);
    for (int j = 0; j < min(32, u.n - j0); j += kLoads) {
      if (j0 + j) {
#pragma unroll
        for (int e = 0; e < kLoads; ++e) v[e] = u.output(row, j0 + j + e);
      }
#pragma unroll
      for (int e = 0; e < kLoads; ++e) add(o, __shfl_sync(0xffffffffu, w, j + e), v[e]);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  finish<T>(p, u, row, o, m, l);
}

template <typename T>
__global__ void __launch_bounds__(kThr, kPerSm) merge_kernel(const __grid_constant__ ChunkParams p, int n_ctas) {
  __shared__ int4 notes[kThr];
  __shared__ int first[kThr];  // item
  __shared__ int tot[kThr / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int4 note = t < n_ctas ? __ldcg(p.notes + t) : make_int4(0, 0, 0, 0);
  const int per = item_rows(note.w - t + 1), items = (note.z + per - 1) / per;
  int sum = items;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 31) tot[warp] = sum;
  notes[t] = note;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) {
    if (w < warp) sum += tot[w];
    total += tot[w];
  }
  first[t] = sum - items;
  __syncthreads();
  for (int item = warp * gridDim.x + blockIdx.x; item < total; item += gridDim.x * (kThr / 32)) {
    // the last CTA whose items start no later: of CTAs without items none is last
    int c = 31 - __clz(__ballot_sync(0xffffffffu, first[lane * 8] <= item));
    c = c * 8 + 31 - __clz(__ballot_sync(0xffffffffu, lane < 8 && first[c * 8 + (lane & 7)] <= item));
    Unit u;
    u.note = notes[c];
    u.n = u.note.w - c + 1;
    u.slot = (int64_t)p.part_rows * kChunkStride;
    u.part = p.part + 2 * c * u.slot;
    const int row = (item - first[c]) * item_rows(u.n);
    if (u.n <= 2) merge_few<T, 4>(p, u, row);
    else if (u.n <= 4) merge_few<T, 2>(p, u, row);
    else merge_many<T>(p, u, row);
  }
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkParams &p, int grid, bool f32, cudaStream_t s) {
  const int ctas = grid * kPerSm;
  return f32 ? launch_dependent(merge_kernel<float>, ctas, kThr, 0, s, p, grid)
             : launch_dependent(merge_kernel<uint16_t>, ctas, kThr, 0, s, p, grid);
}

}  // namespace mac
