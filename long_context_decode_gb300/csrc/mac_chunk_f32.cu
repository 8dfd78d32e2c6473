// mac_chunk_f32.cu -- chunk attention in fp32 on the CUDA cores.
//
// For a row with rotated query q at position p:
//   x_j = q . k_j log2(e)/sqrt(d), j <= p;  m = max x_j;
//   l = sum 2^(x_j - m);  out = sum 2^(x_j - m) v_j / l;  lse = m ln 2 + ln l
// in one pass over the keys with a running m, l and o.  A CTA of 256
// threads holds 64 rows and takes keys 64 at a time; a thread owns 4 rows x
// 4 keys of the scores (rows ty + 16 i, keys tx + 16 j) and 4 rows x 8 dims of the
// output, so each 16-byte read of shared memory feeds 8 multiply-adds.
#include <math.h>

#include "mac_chunk.cuh"

namespace mac {
namespace {

constexpr int kRows = kChunkRowsF32, kKeys = 64, kThr = 256, kCost0 = 2, kMinShare = 4;  // costs in key tiles
constexpr int kPad = kHeadDim + 4;   // floats per Q/K row: neighbouring rows start 4 banks apart
constexpr int kPPad = kKeys + 4;     // floats per row of probabilities
using Plan = ChunkPlan<kRows, kKeys, kCost0, 1, 1>;
using Walk = ChunkWalk<Plan, kCost0, 1, 1>;

struct Shared {
  float q[kRows][kPad];
  union {
    float k[kKeys][kPad];
    float pr[kRows][kPPad];          // probabilities, once the scores are done with K
  };
  float v[kKeys][kHeadDim];
  Plan plan;
  int last;
};

template <typename T>
__device__ __forceinline__ void load_row16(float *dst, const T *src, bool ok) {
  constexpr int PER = 16 / (int)sizeof(T);
  float f[PER];
  if (ok) {
    unpack16<T>(*reinterpret_cast<const uint4 *>(src), f);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < PER; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

// Row of token `key` (0-based) of request b, KV head g; -1: on no page.
__device__ __forceinline__ int64_t cache_row(const ChunkParams &p, int b, int g, int key) {
  if (!p.kv.paged) return ((int64_t)b * p.Hkv + g) * p.kv.capacity + key;
  const int id = p.kv.page_table[(int64_t)b * p.kv.max_pages + key / kPage];
  if (id < 0 || id >= p.kv.n_pages) return -1;
  return ((int64_t)id * p.Hkv + g) * kPage + key % kPage;
}

template <typename T>
__global__ void __launch_bounds__(kThr, 2) chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &sm = *reinterpret_cast<Shared *>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  griddep_launch_dependents();
  griddep_wait();
  sm.plan.build(p, kMinShare);
  if (sm.plan.any_bad) chunk_bad_requests<T, Plan>(p);
  Walk walk;
  if (!walk.start(p, sm.plan)) return;
  uint32_t status = 0;
  ChunkPiece piece;

  while (walk.next(p, piece)) {
    const ChunkUnit &u = piece.u;
    const int t0 = piece.t0, t1 = piece.t1;
    const int n_rows = u.n_tok * p.G;
    __syncthreads();  // the last unit's shared memory has been read
    for (int i = tid; i < kRows * (kHeadDim / 4); i += kThr) {
      const int r = i / (kHeadDim / 4), c = i % (kHeadDim / 4) * 4;
      const int64_t at = ((int64_t)(u.tok0 + r / p.G) * p.Hq + u.g * p.G + r % p.G) * kHeadDim + c;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n_rows) f = make_float4(elem_f32<T>(p.q, at), elem_f32<T>(p.q, at + 1), elem_f32<T>(p.q, at + 2), elem_f32<T>(p.q, at + 3));
      *reinterpret_cast<float4 *>(&sm.q[r][c]) = f;
    }
    float m[4], l[4], o[4][8];
    int lim[4];  // keys [0, lim) are the row's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      lim[i] = u.pos0 + (ty + 16 * i) / p.G;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[i][j] = 0.f;
    }
    const int n_keys = u.pos0 + u.n_tok - 1;
    for (int t = t0; t < t1; ++t) {
      const int key0 = t * kKeys;
      __syncthreads();  // K, V and the probabilities of the last tile have been read
      constexpr int PER = 16 / (int)sizeof(T), CH = kHeadDim / PER;
      for (int i = tid; i < kKeys * CH; i += kThr) {
        const int r = i / CH, c = i % CH * PER;
        int64_t row = -1;
        if (key0 + r < n_keys) {
          row = cache_row(p, u.b, u.g, key0 + r);
          if (row < 0) status |= MAC_DEV_BAD_PAGE;
        }
        load_row16<T>(&sm.k[r][c], (const T *)p.kv.k + row * kHeadDim + c, row >= 0);
        load_row16<T>(&sm.v[r][c], (const T *)p.kv.v + row * kHeadDim + c, row >= 0);
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < kHeadDim; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(&sm.q[ty + 16 * i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
            s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
            s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
            s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
          }
      }
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + tx + 16 * j;
        on[j] = key < n_keys && (!p.kv.paged || cache_row(p, u.b, u.g, key) >= 0);
      }
      float corr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + tx + 16 * j;
          s[i][j] = on[j] && key < lim[i] ? s[i][j] * p.q_scale : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
        corr[i] = ex2(m[i] - ms);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = ex2(s[i][j] - ms);
          sum += s[i][j];
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = l[i] * corr[i] + sum;
      }
      __syncthreads();  // K has been read
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.pr[ty + 16 * i][tx + 16 * j] = s[i][j];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[i][j] *= corr[i];
#pragma unroll 2
      for (int k = 0; k < kKeys; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(&sm.pr[ty + 16 * i][k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v0 = *reinterpret_cast<const float4 *>(&sm.v[k + e][tx * 4]);
          const float4 v1 = *reinterpret_cast<const float4 *>(&sm.v[k + e][64 + tx * 4]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
            o[i][0] = fmaf(w, v0.x, o[i][0]);
            o[i][1] = fmaf(w, v0.y, o[i][1]);
            o[i][2] = fmaf(w, v0.z, o[i][2]);
            o[i][3] = fmaf(w, v0.w, o[i][3]);
            o[i][4] = fmaf(w, v1.x, o[i][4]);
            o[i][5] = fmaf(w, v1.y, o[i][5]);
            o[i][6] = fmaf(w, v1.z, o[i][6]);
            o[i][7] = fmaf(w, v1.w, o[i][7]);
          }
        }
      }
    }
    // a whole unit goes out; a piece of one leaves its state
    if (!piece.cut()) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= n_rows) continue;
        const int64_t row = (int64_t)(u.tok0 + r / p.G) * p.Hq + u.g * p.G + r % p.G;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        T *dst = (T *)p.out + row * kHeadDim;
        store_out(dst + tx * 4, make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv));
        store_out(dst + 64 + tx * 4, make_float4(o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv));
        if (p.lse && tx == 0) p.lse[row] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
      }
      continue;
    }
    const int c = blockIdx.x, c0 = walk.cta_of(p, u, 0), c1 = walk.cta_of(p, u, u.tiles - 1);
    float *part = p.part + (int64_t)(2 * c + (c == c0 ? 1 : 0)) * p.part_rows * kPartStride;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      if (r >= n_rows) continue;
      float *dst = part + r * kPartStride;
      store_out(dst + tx * 4, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
      store_out(dst + 64 + tx * 4, make_float4(o[i][4], o[i][5], o[i][6], o[i][7]));
      if (tx == 0) store_out(dst + kHeadDim, make_float4(m[i], l[i], 0.f, 0.f));
    }
    __syncthreads();
    if (tid == 0) {
      const uint32_t n = c1 - c0 + 1, old = add_acq_rel(p.count + c0, 1);
      sm.last = old == n - 1;
      if (sm.last) p.count[c0] = 0;  // for the next launch
    }
    __syncthreads();
    if (!sm.last) continue;
    chunk_merge<T>(p, u, c0, c1, n_rows, tid, kThr);
  }
  if (status) set_status(p.status, status);
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkParams &p, int sms, cudaStream_t s) {
  static_assert(2 * sizeof(Shared) <= 227 * 1024, "two CTAs per SM");
  static DeviceFlags done;
  const cudaError_t e = prepare_chunk(chunk_kernel<float>, done, sizeof(Shared), 0);
  if (e != cudaSuccess) return e;
  const int grid = 2 * sms < kChunkGrid ? 2 * sms : kChunkGrid;
  return launch_dependent(chunk_kernel<float>, grid, kThr, sizeof(Shared), s, p);
}

}  // namespace mac
