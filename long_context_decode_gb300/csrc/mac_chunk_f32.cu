// mac_chunk_f32.cu -- chunk attention in fp32 on the CUDA cores.
//
// For a row with rotated query q at position p:
//   x_j = q . k_j log2(e)/sqrt(d), j <= p;  m = max x_j;
//   l = sum 2^(x_j - m);  out = sum 2^(x_j - m) v_j / l;  lse = m ln 2 + ln l
// in one pass over the keys with a running m, l and o.  (The tensor cores
// keep no more than 10 bits of an fp32 factor.)
//
// A CTA of 256 threads takes 16 I packed rows and keys 64 at a time; a thread
// owns I rows (ty + 16 i) x 4 keys (tx + 16 j) of the scores and the same
// rows x 8 dims of the output.  The multiply-adds are packed in pairs
// (fma.rn.f32x2: over even and odd dims for the scores, over two dims for
// the output, the weights stored twice), which halves the instructions; a
// loop of them alone reaches 102 multiply-adds per cycle and SM, this kernel
// 63 (4096 tokens, 8 heads: 945 us, 36 TFLOP/s) with shared memory 73% busy.
// The weights overwrite K and are made and used by the same half warp.  Two
// CTAs share an SM: one computes while the other waits for its copies or
// takes its maxima.  (One CTA with 8 x 4 microtiles: 870 us, but 35 us
// instead of 25 for seven rows; two of 128 threads with 8 x 4: 982 us.)
//   I = 4: 64 rows, for batches of many rows per request (the multiply-adds
//          are the bound); I = 1: 16 rows, for a few (reading shared memory is).
#include <math.h>

#include "mac_chunk.cuh"

namespace mac {
namespace {

constexpr int kKeys = 64, kThr = 256, kCost0 = 1, kMinShare = 2;  // costs in key tiles
constexpr int kPad = kHeadDim + 4;   // floats per Q/K row: neighbouring rows start 4 banks apart
constexpr int kPPad = 2 * kKeys + 4; // floats per row of doubled weights
template <int I>
using Plan = ChunkPlan<16 * I, kKeys, kCost0, 1, 1>;

template <int I>
struct Shared {
  float q[16 * I][kPad];
  union {
    float k[kKeys][kPad];
    float pr[16 * I][kPPad];  // once the scores are done with K
  };
  float v[kKeys][kHeadDim];
  Plan<I> plan;
  int last;
};

__device__ __forceinline__ void fma2(float2 &d, float2 a, float2 b) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 d, {%0, %1};\n\t"
      "fma.rn.f32x2 d, a, b, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d.x), "+f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// 16 bytes into shared memory, asynchronously; zeros where !ok.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Row of token `key` (0-based) of request b, KV head g; -1: on no page.
__device__ __forceinline__ int64_t cache_row(const ChunkParams &p, int b, int g, int key) {
  if (!p.kv.paged) return ((int64_t)b * p.Hkv + g) * p.kv.capacity + key;
  const int id = p.kv.page_table[(int64_t)b * p.kv.max_pages + key / kPage];
  if (id < 0 || id >= p.kv.n_pages) return -1;
  return ((int64_t)id * p.Hkv + g) * kPage + key % kPage;
}

template <int I>
__global__ void __launch_bounds__(kThr, 2) chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<I> &sm = *reinterpret_cast<Shared<I> *>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  griddep_launch_dependents();
  griddep_wait();
  sm.plan.build(p, kMinShare);
  if (sm.plan.any_bad) chunk_bad_requests<float, Plan<I>>(p);
  ChunkWalk<Plan<I>, kCost0, 1, 1> walk;
  if (!walk.start(p, sm.plan)) return;
  uint32_t status = 0;
  ChunkPiece piece;

  while (walk.next(p, piece)) {
    const ChunkUnit &u = piece.u;
    const int t0 = piece.t0, t1 = piece.t1;
    const int n_rows = u.n_tok * p.G, n_keys = u.pos0 + u.n_tok - 1;
    // a warp copies whole rows
    auto copy_tile = [&](float *dst, int pitch, const void *src, int t) {
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int r = i * 8 + (tid >> 5), c = (tid & 31) * 4, key = t * kKeys + r;
        int64_t row = -1;
        if (key < n_keys) {
          row = cache_row(p, u.b, u.g, key);
          if (row < 0) status |= MAC_DEV_BAD_PAGE;
        }
        copy16(dst + r * pitch + c, (const float *)src + (row < 0 ? 0 : row) * kHeadDim + c, row >= 0);
      }
    };
    __syncthreads();  // the last unit's shared memory has been read
#pragma unroll
    for (int i = 0; i < 2 * I; ++i) {
      const int r = i * 8 + (tid >> 5), c = (tid & 31) * 4;
      const bool ok = r < n_rows;
      const int64_t row = ok ? (int64_t)(u.tok0 + r / p.G) * p.Hq + u.g * p.G + r % p.G : 0;
      copy16(&sm.q[r][c], (const float *)p.q + row * kHeadDim + c, ok);
    }
    copy_tile(&sm.k[0][0], kPad, p.kv.k, t0);
    copy_commit();
    copy_tile(&sm.v[0][0], kHeadDim, p.kv.v, t0);
    copy_commit();
    float m[I], l[I];
    float2 o[I][4];
    int lim[I];  // keys [0, lim) are the row's
#pragma unroll
    for (int i = 0; i < I; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      lim[i] = u.pos0 + (ty + 16 * i) / p.G;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    for (int t = t0; t < t1; ++t) {
      const int key0 = t * kKeys;
      copy_wait<1>();  // K (and Q); V may be on its way
      __syncthreads();
      float2 s2[I][4];
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int d = 0; d < kHeadDim; d += 4) {
        float4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const float4 a = *reinterpret_cast<const float4 *>(&sm.q[ty + 16 * i][d]);
#pragma unroll
          for (int j = 0; j < 4; ++j) fma2(s2[i][j], make_float2(a.x, a.y), make_float2(b[j].x, b[j].y));
#pragma unroll
          for (int j = 0; j < 4; ++j) fma2(s2[i][j], make_float2(a.z, a.w), make_float2(b[j].z, b[j].w));
        }
      }
      __syncthreads();  // K has been read
      bool on[4];  // keys tx + 16 j lie on page j of the tile
#pragma unroll
      for (int j = 0; j < 4; ++j) on[j] = key0 + 16 * j < n_keys && cache_row(p, u.b, u.g, key0 + 16 * j) >= 0;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        float s[4], mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] = on[j] && key0 + tx + 16 * j < lim[i] ? (s2[i][j].x + s2[i][j].y) * p.q_scale : -INFINITY;
          mx = fmaxf(mx, s[j]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
        const float corr = ex2(m[i] - ms);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] = ex2(s[j] - ms);
          sum += s[j];
          *reinterpret_cast<float2 *>(&sm.pr[ty + 16 * i][2 * (tx + 16 * j)]) = make_float2(s[j], s[j]);
        }
        l[i] = l[i] * corr + sum;  // this lane's keys; the lanes are summed at the end
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[i][j].x *= corr;
          o[i][j].y *= corr;
        }
      }
      copy_wait<0>();   // V
      __syncthreads();  // (and the half warp's weights)
#pragma unroll 4
      for (int k = 0; k < kKeys; k += 2) {
        float4 v[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[e][0] = *reinterpret_cast<const float4 *>(&sm.v[k + e][tx * 4]);
          v[e][1] = *reinterpret_cast<const float4 *>(&sm.v[k + e][64 + tx * 4]);
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const float4 w = *reinterpret_cast<const float4 *>(&sm.pr[ty + 16 * i][2 * k]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 w2 = e ? make_float2(w.z, w.w) : make_float2(w.x, w.y);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              fma2(o[i][2 * h], w2, make_float2(v[e][h].x, v[e][h].y));
              fma2(o[i][2 * h + 1], w2, make_float2(v[e][h].z, v[e][h].w));
            }
          }
        }
      }
      __syncthreads();  // V and the weights have been read
      if (t + 1 < t1) {
        copy_tile(&sm.k[0][0], kPad, p.kv.k, t + 1);
        copy_commit();
        copy_tile(&sm.v[0][0], kHeadDim, p.kv.v, t + 1);
        copy_commit();
      }
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    // a whole unit goes out; a piece of one leaves its state
    const bool whole = !piece.cut();
    const int c = blockIdx.x, c0 = whole ? c : walk.cta_of(p, u, 0), c1 = whole ? c : walk.cta_of(p, u, u.tiles - 1);
    float *part = p.part + (int64_t)(2 * c + (c == c0 ? 1 : 0)) * p.part_rows * kPartStride;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int r = ty + 16 * i;
      if (r >= n_rows) continue;
      const int64_t row = (int64_t)(u.tok0 + r / p.G) * p.Hq + u.g * p.G + r % p.G;
      const float f = !whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
      float *dst = whole ? (float *)p.out + row * kHeadDim : part + r * kPartStride;
      store_out(dst + tx * 4, make_float4(o[i][0].x * f, o[i][0].y * f, o[i][1].x * f, o[i][1].y * f));
      store_out(dst + 64 + tx * 4, make_float4(o[i][2].x * f, o[i][2].y * f, o[i][3].x * f, o[i][3].y * f));
      if (tx == 0) {
        if (!whole) store_out(dst + kHeadDim, make_float4(m[i], l[i], 0.f, 0.f));
        else if (p.lse) p.lse[row] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
      }
    }
    if (whole) continue;
    __syncthreads();
    if (tid == 0) {
      const uint32_t n = c1 - c0 + 1, old = add_acq_rel(p.count + c0, 1);
      sm.last = old == n - 1;
      if (sm.last) p.count[c0] = 0;  // for the next launch
    }
    __syncthreads();
    if (sm.last) chunk_merge<float>(p, u, c0, c1, n_rows, tid, kThr);
  }
  if (status) set_status(p.status, status);
}

template <int I>
cudaError_t launch(const ChunkParams &p, int ctas, cudaStream_t s) {
  static DeviceFlags done;
  const cudaError_t e = prepare_chunk(chunk_kernel<I>, done, sizeof(Shared<I>), 0);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_kernel<I>, ctas < kChunkGrid ? ctas : kChunkGrid, kThr, sizeof(Shared<I>), s, p);
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkParams &p, int sms, cudaStream_t s) {
  static_assert(2 * (sizeof(Shared<4>) + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(kChunkRowsF32 == 16 * 4, "rows of the largest unit");
  // the lengths are on the device: go by the mean rows per request and KV head
  return (int64_t)p.T * p.G <= 16LL * p.B ? launch<1>(p, 2 * sms, s) : launch<4>(p, 2 * sms, s);
}

}  // namespace mac
