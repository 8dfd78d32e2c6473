// mac_chunk_merge.cu -- the pieces of chunk attention's cut units.
//
// Pieces of disjoint keys with states (o, m, l), o and l relative to 2^m:
//   M = max m;  out = sum 2^(m - M) o / sum 2^(m - M) l;  lse = M ln 2 + ln sum.
// One CTA per (CTA of the attention kernel, 8 rows): it looks at that CTA's
// note and is done if no cut unit starts there.  A warp takes a row, four
// dims per lane: lane j reads piece j's state while the outputs of the first
// eight pieces are on their way, so that up to eight pieces cost one trip to
// L2.  Bound by these trips and the launch: 5 us of the 48 us of an fp32 call
// (two requests of up to 4096 tokens, 8 query and 2 KV heads); four rows per
// warp in turn took 11.
// (Merged by the CTA that finished a unit's last piece, 128 rows of five
// pieces took 60 us.)
#include <math.h>

#include "mac_chunk.cuh"

namespace mac {
namespace {

constexpr int kThr = 256, kRowsPerCta = kThr / 32, kBatch = 8;

template <typename T>
__global__ void __launch_bounds__(kThr, 4) merge_kernel(const __grid_constant__ ChunkParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 note = __ldcg(p.notes + c0);  // first token, KV head, rows, last CTA
  const int n = note.w - c0 + 1;
  const int64_t slot = (int64_t)p.part_rows * kChunkStride;  // floats per partial
  const int r = blockIdx.y * kRowsPerCta + (threadIdx.x >> 5);
  if (r >= note.z) return;
  const float *row = p.part + 2 * c0 * slot + (int64_t)r * kChunkStride;
  auto piece = [&](int j) { return row + (2 * j + (j == 0)) * slot; };
  auto state = [&](int j) {
    return j < n ? __ldcg(reinterpret_cast<const float2 *>(piece(j) + kHeadDim)) : make_float2(-INFINITY, 0.f);
  };
  float4 v[kBatch];
  auto outputs = [&](int j0) {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j0 + e < n) v[e] = __ldcg(reinterpret_cast<const float4 *>(piece(j0 + e)) + lane);
    }
  };
  float2 ml = state(lane);
  outputs(0);
  float m = ml.x;
  for (int j = 32 + lane; j < n; j += 32) m = fmaxf(m, state(j).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (m == -INFINITY) m = 0.f;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < n; j0 += 32) {
    if (j0) ml = state(j0 + lane);
    const float w = ex2(ml.x - m);
    l = fmaf(w, ml.y, l);
    for (int j = 0; j < min(32, n - j0); j += kBatch) {
      if (j0 + j) outputs(j0 + j);
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const float x = __shfl_sync(0xffffffffu, w, j + e);
        o.x = fmaf(x, v[e].x, o.x);
        o.y = fmaf(x, v[e].y, o.y);
        o.z = fmaf(x, v[e].z, o.z);
        o.w = fmaf(x, v[e].w, o.w);
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const int64_t at = (int64_t)(note.x + r / p.G) * p.Hq + note.y * p.G + r % p.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store_out((T *)p.out + at * kHeadDim + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkParams &p, int grid, bool f32, cudaStream_t s) {
  const dim3 g(grid, (p.part_rows + kRowsPerCta - 1) / kRowsPerCta);
  return f32 ? launch_dependent(merge_kernel<float>, g, kThr, 0, s, p) : launch_dependent(merge_kernel<uint16_t>, g, kThr, 0, s, p);
}

}  // namespace mac
