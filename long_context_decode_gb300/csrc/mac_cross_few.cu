// mac_cross_few.cu -- cross attention of few rows per source: a decode step's
// beams over their source's states.
//
// For a row with query q, over the keys of its source's memory:
//   x_j = q . k_j log2(e)/sqrt(d);  m a running reference of the row's maximum;
//   l = sum 2^(x_j - m);  o = sum 2^(x_j - m) v_j;  out = o / l;  lse = m ln 2 + ln l.
// A unit is up to 16 packed rows (token-major, the G heads of a token together)
// of one KV head (more rows of a source are more units).  Bound by HBM: every key
// and value is read once for a unit, and 16 rows are few enough for the warps' own
// matrix instructions (m16n8, 32 to 96 of them per 8 KB), which start on 4 KB of
// keys where a tcgen05 tile wants 128 rows and 32 KB.
//
// One CTA per SM, eight warps.  Within a key tile a warp has keys of its own,
// copies them into stages of its own and keeps maximum, sum and output of its
// own: no warp waits for another until a piece ends, and the copies of the next
// piece are under way by then.  There the eight states are joined through the
// stages that have been read last.
//
// Units are cut over the CTAs as chunk attention's are: they lie end to end on a
// cost axis and a CTA takes an equal span of it, or a whole unit where there are
// CTAs for all and none is long.  Every warp works out its CTA's pieces for
// itself, as its copies reach them: a small call waits for code that has not been
// fetched yet (some 5 ns an instruction), so the plan is short rather than
// shared.  Of a cut unit's pieces the one that is done last joins them all, if
// they are few; else the merge kernel of chunk attention does.
//
// fp32: a = a0 + a1 of 11 bits each (rounded, so a1 is good to 2^-22 of a), and
//   a b = a0 b0 + a0 b1 + a1 b0 + (a1 b1, up to 2^-22 of a b, left out):
// three products in tf32, each exact in the sums, so a product is off by at most
// 2^-20 of its size (2^-24 on average).  The tensor cores cut their sums off, by up
// to 2^-23 each time and always towards zero: a tile's products are summed there
// (2^-22 in all) and added to o with rounding to nearest.  With o among the tensor
// cores' sums, outputs over values of one sign came out 2^-14.5 too small after 32768
// keys of a CTA, 2^-12.5 after 131072; now 2^-24, which costs 4 to 9% (4 x 32768 keys
// 195 and 210 us; with single adds, not pairs, 216).
//
// In a graph (us; floor: bytes at 6.7 TB/s): 16 rows of each of 4 sources of 32768
// keys, 32 / 8 heads, 84.5 (80.1; 6.4 TB/s), in fp32 210 (160); 64 rows over 16
// sources of 1024 keys 10.8 from L2, 15.2 from HBM (10.2); of 400 to 1500 keys, cut,
// 14.6 and 18.3 (9.6); one row over 57 keys 4.4.  What is left over the floor is the
// start (3.5 us until the first keys are there), some 2.5 us of every further piece of
// a CTA and, of cut units, join, count and output behind the last key (3 us).
#include <math.h>

#include "mac_tc.cuh"

namespace mac {
namespace {

constexpr int kWarps = 8, kThr = kWarps * 32, kRows = 16, kStages = 3;
constexpr int kStep = 8192;                   // bytes of a warp's keys and values in a tile; of 16 rows of output
static_assert(kStep == 16 * kHeadDim * 4, "a stage that has been read takes the outputs of a row tile");

template <typename T>
constexpr int kKeysOf = sizeof(T) == 4 ? 8 : 16;  // keys of a warp in a tile
constexpr int kLoads = 8;                     // pieces of a row that are read at once
constexpr int kQStride = kHeadDim + 16;       // floats between rows of the fp32 queries' parts

// A piece of a unit.
struct Piece {
  int b, g;           // source, KV head
  int tok0, n_tok;    // first row of the batch, rows
  int keys;           // of the memory
  int t0, t1;         // key tiles; none: the walk has ended
  int tiles;          // of the unit
  long long first;    // place of the unit's first tile on the cost axis
  __device__ bool cut() const { return t1 - t0 < tiles; }
};

// A cut unit: its pieces' CTAs, its rows.
struct Cut {
  int c0, n, tok0, g, n_rows;
};

template <typename T>
struct Shared {
  static constexpr bool kF32 = sizeof(T) == 4;
  uint8_t stage[kWarps][kStages][kStep];
  float q[kF32 ? 2 : 1][kF32 ? kRows * kQStride : 4];  // fp32: the queries' parts
  // bf16: the queries of four pieces, on their way to registers (their swizzle is an exclusive or of the address)
  __align__(256) uint8_t qb[kF32 ? 1 : 4][kF32 ? 16 : kRows * kHeadDim * 2];
  float2 ml[kWarps][kRows];
  Piece pieces[kWarps][4];
  int2 ctas[kWarps];     // that hold the first and last tile of a cut unit
  Cut cut[2];            // the units of this CTA's first and last piece
  uint32_t arrived[2];   // pieces of a cut unit that were done before this CTA's
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_if(uint32_t dst, const void *src, bool there) {
  const int n = there ? 16 : 0;  // zeros where there is nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldm4(uint32_t *r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t *r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float *c, const float *a, float b0, float b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
                 "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
__device__ __forceinline__ void mma_tf32_first(float *c, const float *a, float b0, float b1) {  // c = a b
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
                 "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(0.f));
}
__device__ __forceinline__ float tf32(float x) {
  uint32_t u;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(u) : "f"(x));
  return __uint_as_float(u);
}
__device__ __forceinline__ void split(float x, float &hi, float &lo) {
  hi = tf32(x);
  lo = tf32(x - hi);
}

// Where 16 bytes of a row lie in a stage's half (keys, values), so that the
// lanes that read at once meet no bank twice.
template <typename T>
__device__ __forceinline__ int place(int row, int chunk, bool values) {
  if (sizeof(T) == 2) return row * 256 + ((chunk ^ (row & 7)) << 4);
  return row * 512 + ((chunk ^ (values ? (row >> 1 & 3) << 1 : (row & 1) << 2)) << 4);
}

// a / b for a >= 0, b > 0
__device__ __forceinline__ long long div_down(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? div_s64(a, b) : (uint32_t)a / (uint32_t)b;
}

// Sum over the warp's lanes, each up to 2^52.
__device__ __forceinline__ long long warp_sum(long long v) {
  const uint32_t a = (uint32_t)v & 0x3ffffff, b = (uint32_t)(v >> 26);
  return ((long long)__reduce_add_sync(0xffffffffu, b) << 26) + __reduce_add_sync(0xffffffffu, a);
}

// A source, as the plan sees it.
struct Source {
  int row0, n, keys;   // first row, rows (0: nothing to attend), states
  int blocks, tiles;   // units of a KV head; key tiles
  bool odd;            // rows that are not attended: bad lengths, or no states
  bool back;           // q_start goes back here
};

// The pieces of a CTA, worked out by every warp for itself (all lanes call it).
template <typename C>
struct Walk {
  static constexpr int START = C::kStart, TILE = C::kTile;
  int lg, lt;          // log2 of the heads of a KV head, and of the tokens of a unit
  int b, k;            // source, unit (KV head by head, in each its rows' blocks)
  Source src;
  bool whole, odd;     // no unit is cut; some source is odd
  long long x, end, share, at;  // this CTA's span (whole: units); the unit's place

  __device__ __forceinline__ Source source(const ChunkParams &p, int i) const {
    Source s;
    const int r0 = p.q_start[i * p.group], r1 = p.q_start[(i + 1) * p.group], m = p.seq_len[i];
    const bool in = r0 >= 0 && r1 >= r0 && r1 <= p.T;
    s.row0 = r0;
    s.keys = m;
    s.odd = !in || (r1 > r0 && (m < 1 || m > p.max_len));
    s.back = r1 < r0;
    s.n = s.odd ? 0 : r1 - r0;
    s.blocks = (s.n + (1 << lt) - 1) >> lt;
    s.tiles = (int)(((long long)m + C::kKeys - 1) / C::kKeys);
    return s;
  }
  __device__ __forceinline__ int cost(const Source &s) const { return START + TILE * s.tiles; }  // tiles <= 2^25

  // false: nothing to do
  __device__ bool start(const ChunkParams &p) {
    const int lane = threadIdx.x & 31;
    lg = 31 - __clz(p.G);
    lt = log2i(C::kRows) - lg;
    long long total = 0;
    int units = 0, top = 0;  // 2^24 and 2^28 at most
    odd = false;
    bool back = false;
    Source mine;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      mine = {};
      if (b0 + lane < p.B) mine = source(p, b0 + lane);
      odd |= mine.odd;
      back |= mine.back;
      if (mine.blocks) {
        total += (long long)mine.blocks * p.Hkv * cost(mine);
        units += mine.blocks * p.Hkv;
        top = max(top, cost(mine));
      }
    }
    odd = __any_sync(0xffffffffu, odd);
    total = warp_sum(total);
    units = __reduce_add_sync(0xffffffffu, units);
    top = __reduce_max_sync(0xffffffffu, top);
    const long long ctas = max(1, (int)min(total / C::kMinShare, (long long)gridDim.x));
    whole = units <= (int)gridDim.x && (top - C::kCut - 1) * ctas < total;
    share = whole ? 1 : div_down(total + ctas - 1, ctas);
    // Rows that several sources claim, as a q_start that goes back has them, may be more
    // units than the host counted when it left the merge kernel out: then none is cut.
    if (odd && __any_sync(0xffffffffu, back)) {
      whole = true;
      share = div_down(units + gridDim.x - 1, gridDim.x);
    }
    x = blockIdx.x * share;
    end = min(whole ? units : total, x + share);
    if (x >= end) return false;
    long long before = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.B && !found; b0 += 32) {
      if (p.B > 32) {
        mine = {};
        if (b0 + lane < p.B) mine = source(p, b0 + lane);
      }
      const long long v = whole ? mine.blocks * p.Hkv : mine.blocks ? (long long)mine.blocks * p.Hkv * cost(mine) : 0;
      long long sum = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, x < before + sum);
      if (!past) {
        before += __shfl_sync(0xffffffffu, sum, 31);
        continue;
      }
      const int hit = __ffs(past) - 1;
      b = b0 + hit;
      src.row0 = __shfl_sync(0xffffffffu, mine.row0, hit);
      src.n = __shfl_sync(0xffffffffu, mine.n, hit);
      src.keys = __shfl_sync(0xffffffffu, mine.keys, hit);
      src.blocks = __shfl_sync(0xffffffffu, mine.blocks, hit);
      src.tiles = __shfl_sync(0xffffffffu, mine.tiles, hit);
      before += __shfl_sync(0xffffffffu, sum - v, hit);
      found = true;
    }
    if (!found) return false;  // (not while the arrays stay as they are)
    k = (int)(whole ? x - before : div_down(x - before, cost(src)));
    at = before + (whole ? k : (long long)k * cost(src));
    return true;
  }

  // CTAs that hold a cut unit's first and last tile.
  __device__ int first_cta(const Piece &q) const { return (int)div_down(q.first, share); }
  __device__ int last_cta(const Piece &q) const { return (int)div_down(q.first + (long long)TILE * (q.tiles - 1), share); }

  // The next piece with a tile; one without: the CTA's work is done.
  __device__ Piece next(const ChunkParams &p) {
    while (x < end) {
      int t0 = 0, t1 = src.tiles;
      const long long first = at + START, last = first + (long long)TILE * (src.tiles - 1);  // of its first and last tile
      if (whole) {
        x = ++at;
      } else {
        if (x > first) t0 = (int)((x - first + TILE - 1) / TILE);
        if (end <= last) t1 = end > first ? (int)((end - first + TILE - 1) / TILE) : 0;
        at = x = last + TILE;
      }
      const int g = src.blocks == 1 ? k : k / src.blocks, i = k - g * src.blocks;
      const Piece q = {b, g, src.row0 + (i << lt), min(1 << lt, src.n - (i << lt)), src.keys, t0, t1, src.tiles, first};
      if (++k == src.blocks * p.Hkv && x < end) {
        k = 0;
        do {
          if (++b == p.B) {  // (nor this)
            x = end;
            break;
          }
          src = source(p, b);
        } while (src.blocks == 0);
      }
      if (t0 < t1) return q;
    }
    return Piece{};
  }
};

// One more piece of a cut unit is done: how many were before.  What the CTA
// wrote ahead of the barrier that thread 0 has come through is seen by whoever
// finds it counted.
__device__ __forceinline__ uint32_t arrive(uint32_t *count) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  return before;
}

// A state of weight f joins (x, y, sum).
__device__ __forceinline__ void add_state(float4 &x, float4 &y, float &sum, float f, float4 u, float4 v, float l) {
  sum = fmaf(f, l, sum);
  x = make_float4(fmaf(f, u.x, x.x), fmaf(f, u.y, x.y), fmaf(f, u.z, x.z), fmaf(f, u.w, x.w));
  y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
}

// Row `at` of a unit that starts at tok0, of KV head g: 4 columns from 4 col and 64 + 4 col on.
template <typename T>
__device__ __forceinline__ void write_row(const ChunkParams &p, int tok0, int g, int lg, int at, int col, float4 x, float4 y, float m, float l) {
  const int64_t to = (int64_t)(tok0 + (at >> lg)) * p.Hq + (g << lg) + (at & ((1 << lg) - 1));
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T *dst = (T *)p.out + to * kHeadDim + col * 4;
  store_out(dst, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  store_out(dst + 64, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
  if (p.lse && col == 0) p.lse[to] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

template <typename T, bool PAGED, typename C>
__global__ void __launch_bounds__(kThr, 1) few_kernel(const __grid_constant__ ChunkParams p) {
  using SM = Shared<T>;
  constexpr bool F32 = SM::kF32;
  constexpr int KW = kKeysOf<T>, AHEAD = kStages - 1;
  static_assert(C::kRows == kRows && C::kKeys == kWarps * KW && KW * kHeadDim * (int)sizeof(T) * 2 == kStep, "tiles");
  static_assert(AHEAD <= 2, "the copies are at most three pieces ahead, and their place in the ring is free");
  extern __shared__ __align__(1024) uint8_t smem[];
  SM &sm = *reinterpret_cast<SM *>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();
  Walk<C> walk;
  const bool work = walk.start(p);
  if (walk.odd) chunk_bad_requests<T, ChunkPlan<C>>(p);
  if (!work) {
    if (tid == 0 && !p.counts) leave_note(p, make_int4(0, 0, 0, 0));
    return;
  }
  int known = 0;  // pieces worked out
  auto walk_on = [&] {
    const Piece q = walk.next(p);
    if (lane == 0) sm.pieces[warp][known & 3] = q;
    ++known;
    __syncwarp();
  };

  // ---- queries: bf16 by way of shared memory, with the copies of their piece's
  // first step, into registers as the products' operands (read straight into
  // registers by every warp they took up to 1 us of a piece); fp32 by way of
  // registers into shared memory, which a piece's end must leave first
  constexpr int UNITS = kHeadDim * (int)sizeof(T) / 16;  // 16-byte parts of a row
  uint32_t qa[F32 ? 1 : 8][4];
  float4 fresh[F32 ? kRows * kHeadDim / 4 / kThr : 1];
  auto q_row = [&](const Piece &q, int r) {
    return (const T *)p.q + ((int64_t)(q.tok0 + (r >> walk.lg)) * p.Hq + (q.g << walk.lg) + (r & ((1 << walk.lg) - 1))) * kHeadDim;
  };
  auto load_q = [&](const Piece &q) {
    if constexpr (F32) {
      const int n_rows = q.n_tok << walk.lg;
#pragma unroll
      for (int i = 0; i < kRows * kHeadDim / 4 / kThr; ++i) {
        const int e = i * kThr + tid, r = e / UNITS;
        fresh[i] = r < n_rows ? *reinterpret_cast<const float4 *>(q_row(q, r) + e % UNITS * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  };
  // bf16: a thread copies 16 bytes; rows that are not there are the last one
  auto copy_q = [&](const Piece &q, int number) {
    if constexpr (!F32) {
      static_assert(kRows * UNITS == kThr, "a part for each thread");
      const int r = tid >> 4, c = tid & 15;
      copy16(smem_addr(sm.qb[number & 3]) + place<T>(r, c, false), q_row(q, min(r, (q.n_tok << walk.lg) - 1)) + c * 8);
    }
  };
  auto take_q = [&](int number) {
    if constexpr (!F32) {
      const uint32_t at = smem_addr(sm.qb[number & 3]) + place<T>(lane & 15, lane >> 4, false);
#pragma unroll
      for (int c = 0; c < 8; ++c) ldm4(qa[c], (at ^ (c & 3) << 5) + (c >> 2) * 128);
    }
  };
  auto put_q = [&] {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < kRows * kHeadDim / 4 / kThr; ++i) {
        const int e = i * kThr + tid, at = e / UNITS * kQStride + e % UNITS * 4;
        float4 hi, lo;
        split(fresh[i].x, hi.x, lo.x);
        split(fresh[i].y, hi.y, lo.y);
        split(fresh[i].z, hi.z, lo.z);
        split(fresh[i].w, hi.w, lo.w);
        *reinterpret_cast<float4 *>(sm.q[0] + at) = hi;
        *reinterpret_cast<float4 *>(sm.q[F32] + at) = lo;
      }
      __syncthreads();
    }
  };

  // ---- copies
  const uint32_t stages = smem_addr(sm.stage[warp]);
  uint32_t status = 0;
  int stage_in = 0;
  Piece in;           // the piece that is copied, and its next tile
  int in_tile = 0;
  uint32_t gone = 0;  // steps in flight whose page does not exist, the last issued in bit 0
  // page of the warp's keys in a tile (contiguous: 0), -1: none, -2: no keys
  auto page_of = [&] {
    const int key0 = in_tile * C::kKeys + warp * KW;
    if (in.t1 <= in.t0 || key0 >= in.keys) return -2;
    if (!PAGED) return 0;
    const int id = p.kv.page_table[(int64_t)in.b * p.kv.max_pages + key0 / kPage];
    return id >= 0 && id < p.kv.n_pages ? id : -1;
  };
  auto enter = [&] {  // the next piece
    walk_on();
    in = sm.pieces[warp][known - 1 & 3];
    in_tile = in.t0;
    if (in.t1 > in.t0) copy_q(in, known - 1);  // (four places: the copies are at most three pieces ahead)
  };
  enter();
  if (in.t1 <= in.t0) {  // a span behind the last tile, or before the next unit's first
    if (tid == 0 && !p.counts) leave_note(p, make_int4(0, 0, 0, 0));
    return;
  }
  load_q(in);
  int page = page_of();
  // A lane's part of a step: bf16 16 bytes of every second row, fp32 of every row.
  // A row's 16-byte parts are swizzled by bits of the row, which change from
  // copy to copy by an exclusive or of the lane's first place.
  constexpr int N = kStep / 2 / 512;
  const uint32_t to_k = stages + place<T>(lane / UNITS, lane % UNITS, false);
  const uint32_t to_v = stages + kStep / 2 + place<T>(lane / UNITS, lane % UNITS, true);
  auto swizzle = [](int i, bool values) {  // of copy i against copy 0
    return F32 ? (uint32_t)(values ? (i >> 1 & 3) << 5 : (i & 1) << 6) : (uint32_t)((2 * i & 6) << 4);
  };
  auto issue = [&] {
    gone = gone << 1 | (page == -1);
    if (page >= 0) {
      const int key0 = in_tile * C::kKeys + warp * KW;
      const int64_t row0 = PAGED ? ((int64_t)page * p.Hkv + in.g) * kPage + key0 % kPage : ((int64_t)in.b * p.Hkv + in.g) * p.kv.capacity + key0;
      const uint8_t *k = (const uint8_t *)p.kv.k + row0 * kHeadDim * sizeof(T) + lane * 16;
      const uint8_t *v = (const uint8_t *)p.kv.v + row0 * kHeadDim * sizeof(T) + lane * 16;
      const uint32_t dk = to_k + stage_in * kStep, dv = to_v + stage_in * kStep;
      const int n = in.keys - key0;
      if (n >= KW) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          copy16((dk ^ swizzle(i, false)) + i * 512, k + i * 512);
          copy16((dv ^ swizzle(i, true)) + i * 512, v + i * 512);
        }
      } else {  // rows behind the last are not read
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          const bool there = i * (32 / UNITS) + lane / UNITS < n;
          const int at = there ? i * 512 : -lane * 16;
          copy16_if((dk ^ swizzle(i, false)) + i * 512, k + at, there);
          copy16_if((dv ^ swizzle(i, true)) + i * 512, v + at, there);
        }
      }
    }
    copies_end();
    if (in.t1 <= in.t0) return;
    if (++stage_in == kStages) stage_in = 0;
    if (++in_tile == in.t1) enter();
    page = page_of();
  };
#pragma unroll 1
  for (int i = 0; i < AHEAD; ++i) issue();
  put_q();
  if constexpr (!F32) {
    copies_wait<AHEAD - 1>();
    __syncthreads();
    take_q(0);
  }

  const float scale = p.q_scale, lazy = 8.f / scale;
  // a lane's rows of the bf16 operands; two 16-byte parts further on are an exclusive or away
  const uint32_t of_k = place<uint16_t>((lane & 7) + (lane >> 4 << 3), lane >> 3 & 1, false);
  const uint32_t of_v = place<uint16_t>(lane & 15, lane >> 4, true);
  int4 note = make_int4(0, 0, 0, 0);
  int stage = 0;
  int n_cut = 0;
#pragma unroll 1
  for (int number = 0;; ++number) {
    const Piece q = sm.pieces[warp][number & 3];
    if (q.t1 <= q.t0) break;
    if (q.cut() && lane == 0) sm.ctas[warp] = make_int2(walk.first_cta(q), walk.last_cta(q));  // while keys are on their way
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll 1
    for (int tile = q.t0; tile < q.t1; ++tile) {
      __syncwarp();  // the stage that comes next has been read
      issue();
      copies_wait<AHEAD>();
      __syncwarp();
      const uint32_t kb = stages + stage * kStep, vb = kb + kStep / 2;
      const uint8_t *kp = sm.stage[warp][stage], *vp = kp + kStep / 2;
      if (++stage == kStages) stage = 0;
      const int left = q.keys - (tile * C::kKeys + warp * KW);  // keys of the warp's that exist
      if (left <= 0) continue;
      if (gone >> AHEAD & 1) {
        status |= MAC_DEV_BAD_PAGE;
        continue;
      }
      // scores: KW keys, 8 per column tile.  A product waits 21 cycles for one into
      // the same sums, so there are four sums in turn
      constexpr int NT = KW / 8;
      float s[NT][4], x[4][4];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e >> 2][e & 3] = 0.f;
      if constexpr (F32) {
        // column order within 16: a lane's four neighbours are columns t and t + 4 of two products
#pragma unroll
        for (int c = 0; c < kHeadDim / 16; ++c) {
          const float4 kx = *reinterpret_cast<const float4 *>(kp + place<T>(g, c * 4 + t, false));
          float h[4], r[4];
          split(kx.x, h[0], r[0]);
          split(kx.y, h[1], r[1]);
          split(kx.z, h[2], r[2]);
          split(kx.w, h[3], r[3]);
          const float *at = sm.q[0] + g * kQStride + c * 16 + t * 4, *at1 = sm.q[F32] + g * kQStride + c * 16 + t * 4;
          const float4 x0 = *reinterpret_cast<const float4 *>(at), x1 = *reinterpret_cast<const float4 *>(at + 8 * kQStride);
          const float4 y0 = *reinterpret_cast<const float4 *>(at1), y1 = *reinterpret_cast<const float4 *>(at1 + 8 * kQStride);
          const float a0[4] = {x0.x, x1.x, x0.y, x1.y}, a1[4] = {y0.x, y1.x, y0.y, y1.y};
          const float b0[4] = {x0.z, x1.z, x0.w, x1.w}, b1[4] = {y0.z, y1.z, y0.w, y1.w};
          mma_tf32(x[0], a1, h[0], h[1]);
          mma_tf32(x[1], b1, h[2], h[3]);
          mma_tf32(x[2], a0, h[0], h[1]);
          mma_tf32(x[3], b0, h[2], h[3]);
          mma_tf32(x[0], a0, r[0], r[1]);
          mma_tf32(x[1], b0, r[2], r[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][e] = (x[2][e] + x[3][e]) + (x[0][e] + x[1][e]);
      } else {
        const uint32_t at = kb + of_k;
        uint32_t b[2][4];
        ldm4(b[0], at);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c < 7) ldm4(b[c + 1 & 1], (at ^ (c + 1 & 3) << 5) + (c + 1 >> 2) * 128);
          mma_bf16(x[c & 1], qa[c], b[c & 1][0], b[c & 1][1]);
          mma_bf16(x[2 + (c & 1)], qa[c], b[c & 1][2], b[c & 1][3]);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = x[2 * j][e] + x[2 * j + 1][e];
      }
      if (left < KW) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j * 8 + t * 2 + (e & 1) >= left) s[j][e] = -INFINITY;
      }
      // weights
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
      bool grows = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        grows |= top[h] > m[h] + lazy;
      }
      if (__any_sync(0xffffffffu, grows)) {  // the reference moves where the maximum has grown by 8 in base 2
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m[h], top[h]), ms = mn == -INFINITY ? 0.f : mn;
          const float corr = ex2((m[h] - ms) * scale);
          m[h] = mn;
          l[h] *= corr;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][2 * h] *= corr;
            o[j][2 * h + 1] *= corr;
          }
        }
      }
      float ms[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) ms[h] = m[h] == -INFINITY ? 0.f : m[h] * scale;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j][e] = ex2(fmaf(s[j][e], scale, -ms[e >> 1]));
          l[e >> 1] += s[j][e];
        }
      // values
      if constexpr (F32) {
        // the key order of the products is (2 t, 2 t + 1) for columns t and t + 4: what a lane has
        const float w[4] = {s[0][0], s[0][2], s[0][1], s[0][3]};
        float ph[4], pl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(w[e], ph[e], pl[e]);
#pragma unroll
        for (int c = 0; c < kHeadDim / 32; ++c) {  // 32 columns: a lane's four neighbours are a column of four products
          const float4 v0 = *reinterpret_cast<const float4 *>(vp + place<T>(2 * t, c * 8 + g, true));
          const float4 v1 = *reinterpret_cast<const float4 *>(vp + place<T>(2 * t + 1, c * 8 + g, true));
          const float a[4] = {v0.x, v0.y, v0.z, v0.w}, b[4] = {v1.x, v1.y, v1.z, v1.w};
          float ah[4], al[4], bh[4], bl[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            split(a[e], ah[e], al[e]);
            split(b[e], bh[e], bl[e]);
          }
          float y[4][4];  // of this tile alone: see above
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_tf32_first(y[e], pl, ah[e], bh[e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_tf32(y[e], ph, al[e], bl[e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_tf32(y[e], ph, ah[e], bh[e]);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float *to = &o[c * 4 + (e >> 2)][e & 3];
            const float2 sum = add2(make_float2(to[0], to[1]), make_float2(y[e >> 2][e & 3], y[e >> 2][(e & 3) + 1]));
            to[0] = sum.x;
            to[1] = sum.y;
          }
        }
      } else {
        // the weights in two bf16 parts: the tensor cores have the time, and the output
        // is then as good as its own rounding (one part: 2.1e-3 against 64 bits where that is 1.6e-3)
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float *w = &s[e >> 1 ? NT - 1 : 0][(e & 1) * 2];
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pa[e]) : "f"(w[1]), "f"(w[0]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pb[e]) : "f"(w[1] - bf16_hi(pa[e])), "f"(w[0] - bf16_lo(pa[e])));
        }
        const uint32_t at = vb + of_v;
        uint32_t b[2][4];
        ldm4t(b[0], at);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c < 7) ldm4t(b[c + 1 & 1], (at ^ (c + 1 & 3) << 5) + (c + 1 >> 2) * 128);
          mma_bf16(o[2 * c], pb, b[c & 1][0], b[c & 1][1]);
          mma_bf16(o[2 * c + 1], pb, b[c & 1][2], b[c & 1][3]);
          mma_bf16(o[2 * c], pa, b[c & 1][0], b[c & 1][1]);
          mma_bf16(o[2 * c + 1], pa, b[c & 1][2], b[c & 1][3]);
        }
      }
    }

    // ---- the piece's end: the warps' states joined
    const Piece after = sm.pieces[warp][number + 1 & 3];
    if (after.t1 > after.t0) load_q(after);  // on its way meanwhile
    const int last = stage == 0 ? kStages - 1 : stage - 1;  // the stage that has been read
    const int n_rows = q.n_tok << walk.lg, c = blockIdx.x;
    const bool whole = !q.cut();
    const int2 ctas = sm.ctas[warp];
    const int c0 = ctas.x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t == 0) sm.ml[warp][h * 8 + g] = make_float2(m[h] * scale, l[h]);  // base 2
    }
    // The outputs take the warps' stages that have been read last: rows of 512 bytes,
    // 16 bytes swizzled by the row, so that neither a store's lanes nor a load's
    // meet a bank twice.
    const int row = tid >> 4, col = tid & 15;  // a thread joins columns 4 col .. and 64 + 4 col .. of a row
    auto joint = [&](int w, int r, int unit) { return reinterpret_cast<float *>(sm.stage[w][last] + r * 512 + ((unit ^ (r & 7)) << 4)); };
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * 8 + g;
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          *reinterpret_cast<float4 *>(joint(warp, r, j * 8 + t * 2)) = make_float4(o[j * 4][2 * h], o[j * 4 + 1][2 * h], o[j * 4 + 2][2 * h], o[j * 4 + 3][2 * h]);
          *reinterpret_cast<float4 *>(joint(warp, r, j * 8 + t * 2 + 1)) =
              make_float4(o[j * 4][2 * h + 1], o[j * 4 + 1][2 * h + 1], o[j * 4 + 2][2 * h + 1], o[j * 4 + 3][2 * h + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<float2 *>(joint(warp, r, j * 2 + (t >> 1)) + (t & 1) * 2) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
      }
    }
    __syncthreads();
    if (row < n_rows) {
      float2 ml[kWarps];
      float big = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = sm.ml[w][row];
        big = fmaxf(big, ml[w].x);
      }
      const float ref = big == -INFINITY ? 0.f : big;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 u = *reinterpret_cast<const float4 *>(joint(w, row, col)), v = *reinterpret_cast<const float4 *>(joint(w, row, col + 16));
        add_state(x, y, sum, ex2(ml[w].x - ref), u, v, ml[w].y);
      }
      if (whole) {
        write_row<T>(p, q.tok0, q.g, walk.lg, row, col, x, y, big, sum);
      } else {
        float *dst = p.part + ((int64_t)(2 * c + (c == c0 ? 1 : 0)) * p.part_rows + row) * kChunkStride;
        *reinterpret_cast<float4 *>(dst + col * 4) = x;
        *reinterpret_cast<float4 *>(dst + 64 + col * 4) = y;
        if (col == 0) *reinterpret_cast<float2 *>(dst + kHeadDim) = make_float2(big, sum);
      }
    }
    if constexpr (!F32) copies_wait<AHEAD - 1>();  // the next piece's queries
    __syncthreads();  // the stages are free again, the partials written
    put_q();
    if (after.t1 > after.t0) take_q(number + 1);
    if (whole) continue;
    if (c == c0) note = make_int4(q.tok0, q.g, n_rows, ctas.y);
    if (p.counts) {
      if (tid == 0) {
        sm.cut[n_cut] = Cut{c0, ctas.y - c0 + 1, q.tok0, q.g, n_rows};
        sm.arrived[n_cut] = arrive(p.counts + c0);
      }
      ++n_cut;
    }
  }
  copies_wait<0>();
  if (status && lane == 0) set_status(p.status, status);
  if (!p.counts) {
    if (tid == 0) leave_note(p, note);
    return;
  }
  // ---- cut units whose last piece was this CTA's
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < n_cut; ++i) {
    const Cut q = sm.cut[i];
    const int c0 = q.c0, n = q.n;
    if (sm.arrived[i] + 1 != (uint32_t)n) continue;
    if (tid == 0) p.counts[c0] = 0;  // for the next call
    const int row = tid >> 4, col = tid & 15;
    if (row >= q.n_rows) continue;
    float big = -INFINITY, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += kLoads) {  // in one trip to L2 for so many pieces
      float2 ml[kLoads];
      float4 u[kLoads], v[kLoads];
      float most = big;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const float *part = p.part + ((int64_t)(2 * (c0 + j0 + j) + (j0 + j == 0)) * p.part_rows + row) * kChunkStride;
        ml[j] = make_float2(-INFINITY, 0.f);
        u[j] = v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + j < n) {
          ml[j] = __ldcg(reinterpret_cast<const float2 *>(part + kHeadDim));
          u[j] = __ldcg(reinterpret_cast<const float4 *>(part + col * 4));
          v[j] = __ldcg(reinterpret_cast<const float4 *>(part + 64 + col * 4));
        }
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) most = fmaxf(most, ml[j].x);
      const float ref = most == -INFINITY ? 0.f : most, keep = ex2(big - ref);
      sum *= keep;
      x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
      y = make_float4(y.x * keep, y.y * keep, y.z * keep, y.w * keep);
      big = most;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) add_state(x, y, sum, ex2(ml[j].x - ref), u[j], v[j], ml[j].y);
    }
    write_row<T>(p, q.tok0, q.g, walk.lg, row, col, x, y, big, sum);
  }
}

template <typename T, typename C>
cudaError_t launch(const ChunkParams &p, int grid, cudaStream_t s) {
  constexpr int kBytes = sizeof(Shared<T>);
  static_assert(kBytes <= (int)kMaxSmem, "shared memory of a CTA");
  static DeviceFlags done[2];
  cudaError_t e;
  if (p.kv.paged) {
    if ((e = prepare_chunk(few_kernel<T, true, C>, done[1], kBytes, 0)) != cudaSuccess) return e;
    return launch_dependent(few_kernel<T, true, C>, grid, kThr, kBytes, s, p);
  }
  if ((e = prepare_chunk(few_kernel<T, false, C>, done[0], kBytes, 0)) != cudaSuccess) return e;
  return launch_dependent(few_kernel<T, false, C>, grid, kThr, kBytes, s, p);
}

}  // namespace

cudaError_t launch_cross_few(const ChunkParams &p, bool f32, int grid, cudaStream_t s) {
  return f32 ? launch<float, FewF32>(p, grid, s) : launch<uint16_t, FewBf16>(p, grid, s);
}

}  // namespace mac
