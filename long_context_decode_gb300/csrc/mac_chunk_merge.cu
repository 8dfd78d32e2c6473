// mac_chunk_merge.cu -- the pieces of chunk attention's cut units.
//
// Pieces of disjoint keys with states (o, m, l), o and l relative to 2^m:
//   M = max m;  out = sum 2^(m - M) o / sum 2^(m - M) l;  lse = M ln 2 + ln sum.
// One CTA per (CTA of the attention kernel, 16 rows): it looks at that CTA's
// note and is done if no cut unit starts there.  A warp takes two rows, four
// dims per lane; lane j holds piece j's weight, so that the outputs are read
// eight pieces at a time.  Bound by reading the partials (from L2) and by
// the launch.  (Merged by the CTA that finished a unit's last piece, 256
// rows of 4 pieces took 5 us and 128 rows of 5 pieces 60.)
#include <math.h>

#include "mac_chunk.cuh"

namespace mac {
namespace {

constexpr int kThr = 256, kR = 2, kRowsPerCta = kThr / 32 * kR;

template <typename T>
__global__ void __launch_bounds__(kThr) merge_kernel(const __grid_constant__ ChunkParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, r0 = blockIdx.y * kRowsPerCta + (threadIdx.x >> 5) * kR;
  const int4 note = __ldcg(p.notes + c0);  // first token, KV head, rows, last CTA
  if (r0 >= note.z) return;
  const int n = note.w - c0 + 1;
  const int64_t slot = (int64_t)p.part_rows * kChunkStride;  // floats per partial
  auto piece = [&](int j, int i) { return p.part + (2 * (c0 + j) + (j == 0)) * slot + (int64_t)min(r0 + i, note.z - 1) * kChunkStride; };
  float m[kR], l[kR];
  float4 o[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    m[i] = -INFINITY;
    for (int j = lane; j < n; j += 32) m[i] = fmaxf(m[i], __ldcg(piece(j, i) + kHeadDim));
#pragma unroll
    for (int d = 16; d; d >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    if (m[i] == -INFINITY) m[i] = 0.f;
    l[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int j0 = 0; j0 < n; j0 += 32) {
    float w[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      w[i] = 0.f;
      if (j0 + lane < n) {
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(piece(j0 + lane, i) + kHeadDim));
        w[i] = ex2(ml.x - m[i]);
        l[i] = fmaf(w[i], ml.y, l[i]);
      }
    }
    const int k = min(32, n - j0);
    for (int j = 0; j < k; j += 8) {
      float4 v[kR][8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          v[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (j + e < k) v[i][e] = __ldcg(reinterpret_cast<const float4 *>(piece(j0 + j + e, i)) + lane);
        }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const float x = __shfl_sync(0xffffffffu, w[i], (j + e) & 31);
          o[i].x = fmaf(x, v[i][e].x, o[i].x);
          o[i].y = fmaf(x, v[i][e].y, o[i].y);
          o[i].z = fmaf(x, v[i][e].z, o[i].z);
          o[i].w = fmaf(x, v[i][e].w, o[i].w);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    for (int d = 16; d; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    const int r = r0 + i;
    if (r >= note.z) break;
    const int64_t row = (int64_t)(note.x + r / p.G) * p.Hq + note.y * p.G + r % p.G;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    store_out((T *)p.out + row * kHeadDim + lane * 4, make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv));
    if (p.lse && lane == 0) p.lse[row] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
  }
}

}  // namespace

cudaError_t launch_chunk_merge(const ChunkParams &p, int grid, bool f32, cudaStream_t s) {
  const dim3 g(grid, (p.part_rows + kRowsPerCta - 1) / kRowsPerCta);
  return f32 ? launch_dependent(merge_kernel<float>, g, kThr, 0, s, p) : launch_dependent(merge_kernel<uint16_t>, g, kThr, 0, s, p);
}

}  // namespace mac
