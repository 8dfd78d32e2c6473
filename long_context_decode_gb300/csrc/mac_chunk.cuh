// mac_chunk.cuh -- the work of a chunk-attention launch and how it is cut
// over the CTAs, shared by the bf16 and fp32 kernels.
//
// Units are laid end to end in order (request, KV head, row tile) on a cost
// axis (ChunkBf16, ChunkF32: a unit's start plus its key tiles, as many as its
// last row attends).  CTA c works on positions [c share, (c+1) share): any
// number of whole units and at most two cut ones, so rows of very different
// lengths, one long row and many short ones all spread evenly.  A cut unit's
// pieces leave (o, max, sum) partials and the CTA of its first tile a note of
// them; a second kernel merges them in CTA order, so results do not depend on
// timing.  When there is a CTA for every unit and the longest is done before
// an equal share and what cutting costs, each CTA takes one whole unit
// instead, of half the rows if there are CTAs for those as well (us, cut and
// whole): 4 chunks of 60 tokens at 1000, 8 / 2 heads, 19.5 and 16.5; 12 at 1200,
// 32 / 8 heads, 36.1 and 26.9; 16 single tokens at 1100, 23.2 and 17.0; but two
// single tokens at 1900, few and long, 17.2 and 20.9.
#pragma once

#include "mac_batch.cuh"

namespace mac {

#ifdef __CUDACC__

// sum of ceil(j / 2^k), j = 1 .. n
__device__ __forceinline__ long long ceil_sum(long long n, int k) {
  const long long q = n >> k, r = n - (q << k);
  return ((q * (q + 1) >> 1) << k) + r * (q + 1);
}

__host__ __device__ constexpr int log2i(int x) { return x <= 1 ? 0 : 1 + log2i(x >> 1); }

struct ChunkUnit {
  int b, g, i;         // request, KV head, row tile of the request's new tokens
  int a, n, row0;      // the request's tokens before the new ones, new tokens, first row
  int tok0, n_tok;     // first row (token) of the unit in the batch, tokens in it
  int pos0;            // tokens attended by its first token (its 1-based position)
  int tiles;           // key tiles its last token attends
  long long at;        // cost position of its first tile
};

// A CTA's share of a unit.
struct ChunkPiece {
  ChunkUnit u;
  int t0, t1;          // its key tiles
  __device__ bool cut() const { return t0 > 0 || t1 < u.tiles; }
};

template <typename C>
struct ChunkPlan {
  static constexpr int ROWS = C::kRows, KT = C::kKeys, COST0 = C::kStart, W = C::kTile, WS = C::kTileHalf;
  static constexpr int kKt = log2i(KT);

  // of all requests before b, all KV heads: cost; units, those of half the rows
  // in the upper 32 bits
  static_assert(8LL * kMaxTokens / (C::kHalves ? ROWS / 2 : ROWS) * kMaxUnits < 1LL << 31, "units, each request with every row of the batch");
  long long prefix[2][kMaxUnits + 1];
  long long warp_tot[2][32];
  long long share;
  int whole;
  int flags;  // 1: a bad request; 2, 4: a unit, one of half the rows, too long to be taken whole; 8: q_start goes back
  int lt, shift;  // log2 of the tokens per unit, place of its count

  __device__ long long axis(int b) const { return whole ? (uint32_t)(prefix[1][b] >> shift) : prefix[0][b]; }
  __device__ static int units(int n, int lt) { return (n + (1 << lt) - 1) >> lt; }  // n <= kMaxTokens
  __device__ static int weight(int n_tok, int lt) { return 2 * n_tok > 1 << lt ? W : WS; }

  // tiles attended by the first k units, all of them full, of a request
  // with `a` tokens before its new ones; exact because one of KT and the
  // tokens per unit divides the other
  __device__ static long long tiles_before(int a, int lt, int k) {
    if (lt <= kKt) {
      const long long e = (a + (1LL << lt) - 1) >> lt;
      return ceil_sum(e + k, kKt - lt) - ceil_sum(e, kKt - lt);
    }
    return (long long)k * ((a + (long long)KT - 1) >> kKt) + ((long long)k * (k + 1) << (lt - kKt)) / 2;
  }
  // cost of the units before unit k, and of all units of one KV head
  __device__ static long long before(int a, int lt, int k, bool whole) {
    return whole ? k : tiles_before(a, lt, k) * W + (long long)k * COST0;
  }
  __device__ static long long cost(int a, int n, int lt, bool whole) {
    if (n <= 0) return 0;
    const int u = units(n, lt);
    if (whole) return u;
    return before(a, lt, u - 1, false) + COST0 + (((long long)a + n + KT - 1) >> kKt) * weight(n - ((u - 1) << lt), lt);
  }

  // All threads of the block (a multiple of 32, at most 1024) call it.
  __device__ void build(const ChunkParams &p) {
    const int lt0 = log2i(ROWS) - (31 - __clz(p.G)), n_thr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long sum[2] = {0, 0};  // cost, units
    int bad = 0, back = 0, top = 0, top_half = 0;  // highest cost of a unit
    if (threadIdx.x == 0) prefix[0][0] = prefix[1][0] = flags = 0;
    for (int b0 = 0; b0 < p.B; b0 += n_thr) {
      const int b = b0 + threadIdx.x;
      long long v[2] = {0, 0};
      if (b < p.B) {
        int a, n;
        if (request(p, b, &a, &n) != 0) {
          bad = 1;
          back |= p.q_start[b + 1] < p.q_start[b];
        }
        if (n > 0) {
          const int tiles = (int)(((long long)a + n + KT - 1) >> kKt);
          top = max(top, COST0 + tiles * weight(n, lt0));
          top_half = max(top_half, COST0 + tiles * WS);
        }
        v[0] = cost(a, n, lt0, false) * p.Hkv;
        v[1] = (units(n, lt0) + (C::kHalves ? (long long)units(n, lt0 - 1) << 32 : 0)) * p.Hkv;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        for (int d = 1; d < 32; d <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, v[i], d);
          if (lane >= d) v[i] += o;
        }
        if (lane == 31) warp_tot[i][warp] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        long long add = sum[i], all = sum[i];
        for (int w = 0; w < n_thr >> 5 && b0 + w * 32 < p.B; ++w) {
          if (w < warp) add += warp_tot[i][w];
          all += warp_tot[i][w];
        }
        if (b < p.B) prefix[i][b + 1] = v[i] + add;
        sum[i] = all;
      }
      if (b0 + n_thr < p.B) __syncthreads();
    }
    long long ctas = (int)min(sum[0], 1LL << 30) / C::kMinShare;
    if (ctas > gridDim.x) ctas = gridDim.x;
    if (ctas < 1) ctas = 1;
    auto too_long = [&](int cost) { return (cost - C::kCut - 1) * ctas >= sum[0]; };  // cost > ceil(sum / ctas) + kCut
    const int mine = bad | (too_long(top) ? 2 : 0) | (too_long(top_half) ? 4 : 0) | (back ? 8 : 0);
    const int of_warp = __reduce_or_sync(0xffffffffu, mine);
    if (lane == 0 && of_warp) atomicOr(&flags, of_warp);
    __syncthreads();
    const bool half = C::kHalves && !(flags & 4) && sum[1] >> 32 <= gridDim.x;
    const bool each = half || (!(flags & 2) && (uint32_t)sum[1] <= gridDim.x);
    // Rows that several requests claim (only where q_start goes back) make more
    // units than the host counts on when it leaves the merge out: none is cut.
    const bool uncut = !each && (flags & 8);
    if (threadIdx.x == 0) {
      whole = each || uncut;
      lt = half ? lt0 - 1 : lt0;
      shift = half ? 32 : 0;
      share = each ? 1 : uncut ? ((uint32_t)sum[1] + gridDim.x - 1) / gridDim.x : max(1LL, (sum[0] + ctas - 1) / ctas);
    }
    __syncthreads();
  }

  __device__ bool any_bad() const { return flags & 1; }
  __device__ bool has_work(const ChunkParams &p) const { return blockIdx.x * share < axis(p.B); }

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

  // Largest k in [0, n) with f(k) <= x, for a rising f with f(0) <= x: the
  // lanes of each warp (all of them call it) test 32 places at a time.
  template <typename F>
  __device__ static int last_not_above(int n, long long x, F f) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
      const int step = (n + 31) >> 5, k = lo + lane * step;
      const uint32_t yes = __ballot_sync(0xffffffffu, lane * step < n && f(k) <= x);
      const int hit = 31 - __clz(yes);
      n = min(step, n - hit * step);
      lo += hit * step;
    }
    return lo;
  }

  // The unit that holds position x of the axis in use.
  __device__ ChunkUnit find(const ChunkParams &p, long long x) const {
    ChunkUnit u;
    const bool by_units = whole;
    u.b = last_not_above(p.B, x, [&](int b) { return axis(b); });
    request(p, u.b, &u.a, &u.n, &u.row0);
    const int a = u.a;
    const long long per = cost(a, u.n, lt, by_units);
    long long rem = x - axis(u.b);
    u.g = last_not_above(p.Hkv, rem, [&](int g) { return g * per; });
    rem -= u.g * per;
    const int i = last_not_above(units(u.n, lt), rem, [&](int k) { return before(a, lt, k, by_units); });
    set(u, lt, i);
    u.at = x - rem + before(a, lt, i, by_units) + (by_units ? 0 : COST0);
    return u;
  }

  __device__ static void set(ChunkUnit &u, int lt, int i) {
    u.i = i;
    u.tok0 = u.row0 + (i << lt);
    u.n_tok = min(1 << lt, u.n - (i << lt));
    u.pos0 = u.a + (i << lt) + 1;
    u.tiles = (int)(((long long)u.a + (i << lt) + u.n_tok + KT - 1) >> kKt);
  }
};

// A CTA's walk through its pieces.
template <typename C>
struct ChunkWalk {
  using PLAN = ChunkPlan<C>;
  static constexpr int COST0 = C::kStart, W = C::kTile, WS = C::kTileHalf;
  long long x, end, share;
  ChunkUnit u;
  int lt;
  bool first, whole;

  // A whole warp calls it, of a CTA with work.
  __device__ void start(const ChunkParams &p, const PLAN &plan) {
    share = plan.share;
    whole = plan.whole;
    lt = plan.lt;
    x = blockIdx.x * share;
    end = min(plan.axis(p.B), x + share);
    first = true;
    u = plan.find(p, x);
  }
  // Next piece with a tile; false when the CTA's work is done.
  __device__ bool next(const ChunkParams &p, ChunkPiece &q) {
    while (x < end) {
      if (!first) advance(p);
      first = false;
      int t0 = 0, t1 = u.tiles;
      if (whole) {
        x = u.at + 1;
      } else {
        const int w = PLAN::weight(u.n_tok, lt);
        auto first_tile = [&](long long y) { return (int)(w == W ? (y + W - 1) / W : (y + WS - 1) / WS); };
        if (x > u.at) t0 = first_tile(x - u.at);
        if (end < u.at + (long long)u.tiles * w) t1 = end > u.at ? first_tile(end - u.at) : 0;
        x = u.at + (long long)u.tiles * w;
      }
      if (t0 >= t1) continue;
      q.u = u;
      q.t0 = t0;
      q.t1 = t1;
      return true;
    }
    return false;
  }
  // CTAs that hold the pieces of a cut unit: the one of its first tile, and of its last.
  __device__ int cta_of(const ChunkUnit &v, int tile) const {
    return (int)((v.at + (long long)tile * PLAN::weight(v.n_tok, lt)) / share);
  }

 private:
  // The unit after u (there is one).
  __device__ void advance(const ChunkParams &p) {
    const long long at = u.at + (whole ? 1 : (long long)u.tiles * PLAN::weight(u.n_tok, lt) + COST0);
    int i = u.i + 1;
    if (i << lt >= u.n) {
      i = 0;
      if (++u.g == p.Hkv) {
        u.g = 0;
        do {
          ++u.b;
          PLAN::request(p, u.b, &u.a, &u.n, &u.row0);
        } while (u.n == 0);
      }
    }
    PLAN::set(u, lt, i);
    u.at = at;
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

// The note of a cut unit: its first token, KV head, rows, and the CTA of its
// last tile.  Every CTA leaves one (no rows: none of its units is cut after it).
__device__ __forceinline__ void leave_note(const ChunkParams &p, int4 note) { p.notes[blockIdx.x] = note; }

__device__ __forceinline__ void store_out(float *dst, float4 v) { *reinterpret_cast<float4 *>(dst) = v; }
__device__ __forceinline__ void store_out(uint16_t *dst, float4 v) {
  uint2 w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
  *reinterpret_cast<uint2 *>(dst) = w;
}

#endif  // __CUDACC__

}  // namespace mac
