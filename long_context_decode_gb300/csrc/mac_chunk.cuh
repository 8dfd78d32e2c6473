// mac_chunk.cuh -- the work of a chunk-attention launch and how it is cut
// over the CTAs, shared by the bf16 (tensor core) and fp32 kernels.
//
// Units are laid end to end in order (request, KV head, row tile) on a cost
// axis: a unit costs COST0 plus one per tile of KT keys that its last row
// attends.  CTA c works on positions [c share, (c+1) share): any number of
// whole units and at most two cut ones, so rows of very different lengths,
// one long row and many short ones all spread evenly.  A cut unit's pieces
// leave (o, max, sum) partials; the CTA that finishes the last one merges
// them in CTA order, so results do not depend on timing.
#pragma once

#include "mac_batch.cuh"

namespace mac {

#ifdef __CUDACC__

// sum of ceil(j / s), j = 1 .. n
__device__ __forceinline__ long long ceil_sum(long long n, int s) {
  const long long q = n / s, r = n % s;
  return s * (q * (q + 1) / 2) + r * (q + 1);
}

struct ChunkUnit {
  int b, g, i;         // request, KV head, row tile of the request's new tokens
  int a, n, row0;      // the request's tokens before the new ones, new tokens, first row
  int tok0, n_tok;     // first row (token) of the unit in the batch, tokens in it
  int pos0;            // tokens attended by its first token (its 1-based position)
  int tiles;           // key tiles its last token attends
  long long at;        // cost position of its first tile
};

// One request's work, per KV head.
template <int ROWS, int KT, int COST0>
struct ChunkPlan {
  // tiles attended by the first k units of a request with `a` tokens before
  // its new ones, all k of them whole (tt tokens each)
  __device__ static long long tiles_before(int a, int tt, int k) {
    if (tt <= KT) {
      const int s = KT / tt;
      const long long e = (a + (long long)tt - 1) / tt;
      return ceil_sum(e + k, s) - ceil_sum(e, s);
    }
    const int m = tt / KT;
    return (long long)k * ((a + (long long)KT - 1) / KT) + (long long)m * k * (k + 1) / 2;
  }
  // exact because KT divides tt or tt divides KT
  __device__ static long long cost(int a, int n, int tt) {
    if (n <= 0) return 0;
    const int u = (n + tt - 1) / tt;
    return tiles_before(a, tt, u - 1) + ((long long)a + n + KT - 1) / KT + (long long)u * COST0;
  }

  long long prefix[kMaxUnits + 1];  // cost of all requests before b, all KV heads
  long long warp_tot[32];
  long long share;
  int any_bad;

  // All threads of the block (a multiple of 32, at most 1024) call it.
  // MIN_SHARE: least cost worth a CTA of its own.
  __device__ void build(const ChunkParams &p, int min_share) {
    const int tt = ROWS / p.G, n_thr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long carry = 0;
    if (threadIdx.x == 0) any_bad = 0;
    __syncthreads();
    for (int b0 = 0; b0 < p.B; b0 += n_thr) {
      const int b = b0 + threadIdx.x;
      long long v = 0;
      if (b < p.B) {
        int a, n;
        const int st = request(p, b, &a, &n);
        if (st) any_bad = 1;
        v = cost(a, n, tt) * p.Hkv;
      }
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      if (lane == 31) warp_tot[warp] = v;
      __syncthreads();
      long long add = carry, all = carry;
      for (int w = 0; w < n_thr / 32; ++w) {
        if (w < warp) add += warp_tot[w];
        all += warp_tot[w];
      }
      if (b < p.B) prefix[b + 1] = v + add;
      carry = all;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      prefix[0] = 0;
      long long ctas = carry / min_share;
      if (ctas > gridDim.x) ctas = gridDim.x;
      if (ctas < 1) ctas = 1;
      share = (carry + ctas - 1) / ctas;
      if (share < 1) share = 1;
    }
    __syncthreads();
  }

  // Lengths of request b: tokens before the new ones, new tokens (0: nothing
  // to attend).  Returns the status bits of a bad request; *rows, where
  // given, is the number of its rows that lie in the batch.
  __device__ static int request(const ChunkParams &p, int b, int *a, int *n, int *row0 = nullptr, int *rows = nullptr) {
    const int r0 = p.q_start[b], r1 = p.q_start[b + 1], m = p.seq_len[b];
    const bool in = r0 >= 0 && r1 >= r0 && r1 <= p.T;
    const int k = in ? r1 - r0 : 0;
    if (row0) *row0 = r0;
    if (rows) *rows = k;
    *n = k;
    *a = m - k;
    if (!in) return MAC_DEV_BAD_SEQ_LEN;
    if (k == 0) return 0;
    if (m < k || m > p.max_len) {
      *a = *n = 0;
      return MAC_DEV_BAD_SEQ_LEN;
    }
    return 0;
  }

  // The unit that holds cost position x, 0 <= x < prefix[B].
  __device__ ChunkUnit find(const ChunkParams &p, long long x) const {
    ChunkUnit u;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= x) lo = mid; else hi = mid;
    }
    const int tt = ROWS / p.G;
    request(p, lo, &u.a, &u.n, &u.row0);
    const int a = u.a, n = u.n;
    const long long per = cost(a, n, tt);
    const long long off = x - prefix[lo];
    u.b = lo;
    u.g = (int)(off / per);
    const long long rem = off - u.g * per;
    int i0 = 0, i1 = (n + tt - 1) / tt;
    while (i1 - i0 > 1) {
      const int mid = (i0 + i1) >> 1;
      if (tiles_before(a, tt, mid) + (long long)mid * COST0 <= rem) i0 = mid; else i1 = mid;
    }
    set(u, p, i0);
    u.at = prefix[lo] + u.g * per + tiles_before(a, tt, i0) + (long long)i0 * COST0 + COST0;
    return u;
  }

  // The unit after u (there is one).
  __device__ static void advance(ChunkUnit &u, const ChunkParams &p) {
    const int tt = ROWS / p.G;
    const long long at = u.at + u.tiles + COST0;
    int i = u.i + 1;
    if (i * tt >= u.n) {
      i = 0;
      if (++u.g == p.Hkv) {
        u.g = 0;
        do {
          ++u.b;
          request(p, u.b, &u.a, &u.n, &u.row0);
        } while (u.n == 0);
      }
    }
    set(u, p, i);
    u.at = at;
  }

  __device__ static void set(ChunkUnit &u, const ChunkParams &p, int i) {
    const int tt = ROWS / p.G;
    u.i = i;
    u.tok0 = u.row0 + i * tt;
    u.n_tok = min(tt, u.n - i * tt);
    u.pos0 = u.a + i * tt + 1;
    u.tiles = (int)(((long long)u.a + i * tt + u.n_tok + KT - 1) / KT);
  }
};

// Rows of requests that cannot be attended (a length below its new tokens or
// beyond the cache): out 0, lse -inf.  All threads of the grid take part.
template <typename T, typename PLAN>
__device__ void chunk_bad_requests(const ChunkParams &p) {
  for (int b = 0; b < p.B; ++b) {
    int a, n, row0, rows;
    const int st = PLAN::request(p, b, &a, &n, &row0, &rows);
    if (!st) continue;
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, st);
    T *out = (T *)p.out + (int64_t)row0 * p.Hq * kHeadDim;
    const int64_t step = (int64_t)gridDim.x * blockDim.x, i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < (int64_t)rows * p.Hq * kHeadDim; i += step) out[i] = (T)0;
    if (p.lse)
      for (int64_t i = i0; i < (int64_t)rows * p.Hq; i += step) p.lse[(int64_t)row0 * p.Hq + i] = -INFINITY;
  }
}

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t *p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ void store_out(float *dst, float4 v) { *reinterpret_cast<float4 *>(dst) = v; }
__device__ __forceinline__ void store_out(uint16_t *dst, float4 v) {
  uint2 w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
  *reinterpret_cast<uint2 *>(dst) = w;
}

// Pieces c0 .. c1 of a unit into its output rows: a warp per row, four dims
// per lane, the pieces in CTA order.  All `n_thr` threads (from `tid` 0) of
// the CTA that finished the last piece call it.
template <typename T>
__device__ void chunk_merge(const ChunkParams &p, const ChunkUnit &u, int c0, int c1, int n_rows, int tid, int n_thr) {
  const int lane = tid & 31;
  for (int r = tid >> 5; r < n_rows; r += n_thr >> 5) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + lane; c <= c1; c += 32)
      m = fmaxf(m, __ldcg(p.part + ((int64_t)(2 * c + (c == c0)) * p.part_rows + r) * kPartStride + kHeadDim));
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float *src = p.part + ((int64_t)(2 * c + (c == c0)) * p.part_rows + r) * kPartStride;
      const float2 ml = __ldcg(reinterpret_cast<const float2 *>(src + kHeadDim));
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(src) + lane);
      const float w = ex2(ml.x - ms);
      l = fmaf(w, ml.y, l);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const int64_t row = (int64_t)(u.tok0 + r / p.G) * p.Hq + u.g * p.G + r % p.G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store_out((T *)p.out + row * kHeadDim + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : ms * kLn2 + logf(l);
  }
}

#endif  // __CUDACC__

}  // namespace mac
