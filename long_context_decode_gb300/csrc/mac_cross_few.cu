// mac_cross_few.cu -- cross attention of few rows per source: a decode step's
// beams over their source's states.
//
// For a row with query q, over the keys of its source's memory:
//   x_j = q . k_j log2(e)/sqrt(d);  m a running reference of the row's maximum;
//   l = sum 2^(x_j - m);  o = sum 2^(x_j - m) v_j;  out = o / l;  lse = m ln 2 + ln l.
// A unit is up to 16 MT packed rows (token-major, the G heads of a token
// together) of one KV head, cut over the CTAs as chunk attention's units are.
// Bound by HBM: every key and value is read once for a unit, and 16 rows are few
// enough for the warps' own matrix instructions (m16n8, 32 to 128 of them per
// 8 KB), which start on 4 KB of keys where a tcgen05 tile wants 128 rows and 32 KB.
//
// One CTA per SM, eight warps.  Within a key tile a warp has keys of its own,
// copies them into stages of its own and keeps maximum, sum and output of its
// own: no warp waits for another until a piece ends, and the copies of the next
// piece are under way by then.  There the eight states are joined through shared
// memory, 16 or 32 columns at a time.
//
// fp32: a = a0 + a1 of 11 bits each (rounded, so a1 is exact to 2^-22 of a), and
//   a b = a0 b0 + a0 b1 + a1 b0 + a1 b1: four products in tf32, exact in the sums,
// each off by at most 2^-21 of its size.
#include <math.h>

#include "mac_tc.cuh"

namespace mac {
namespace {

constexpr int kWarps = 8, kThr = kWarps * 32;
constexpr int kStep = 8192;                   // bytes of a warp's keys and values in a tile

template <typename T>
constexpr int kKeysOf = sizeof(T) == 4 ? 8 : 16;  // keys of a warp in a tile
constexpr int kQStride = kHeadDim + 16;       // floats between rows of the fp32 queries' parts

// A piece of a unit.
struct Piece {
  int b, g;           // source, KV head
  int tok0, n_tok;    // first row of the batch, rows
  int keys;           // of the memory
  int t0, t1;         // key tiles; none: the walk has ended
  int c0, c1;         // a cut unit's first and last CTA; else -1
};

template <typename T, int MT>
struct Shared {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kRows = 16 * MT;
  static constexpr int kStages = kF32 && MT == 2 ? 2 : 3;
  // columns joined at a time, and floats between their rows: no two of a store's lanes in a bank
  static constexpr int kCols = !kF32 && MT == 2 ? 16 : 32, kStride = kCols + (kF32 ? 4 : 8);
  uint8_t stage[kWarps][kStages][kStep];
  union {
    float join[kWarps][kRows][kStride];
    float q[kF32 ? 2 : 1][kF32 ? kRows : 1][kF32 ? kQStride : 1];  // fp32: the two parts of the queries
  };
  float2 ml[kWarps][kRows];
  Piece pieces[8];
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
// c += a b of two parts each, smallest products first
__device__ __forceinline__ void mma_parts(float *c, const float *a0, const float *a1, float b00, float b01, float b10, float b11) {
  mma_tf32(c, a1, b10, b11);
  mma_tf32(c, a0, b10, b11);
  mma_tf32(c, a1, b00, b01);
  mma_tf32(c, a0, b00, b01);
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

// A warp's way through its steps: the piece (its number in the CTA) and tile.
struct Steps {
  int piece, tile;
};

template <typename T, int MT, bool PAGED, typename C>
__global__ void __launch_bounds__(kThr, 1) few_kernel(const __grid_constant__ ChunkParams p) {
  using SM = Shared<T, MT>;
  using Plan = ChunkPlan<C>;
  constexpr bool F32 = SM::kF32;
  constexpr int KW = kKeysOf<T>, ROWS = SM::kRows, COLS = SM::kCols, NST = SM::kStages, AHEAD = NST - 1;
  static_assert(C::kRows == ROWS && C::kKeys == kWarps * KW && KW * kHeadDim * (int)sizeof(T) * 2 == kStep, "tiles");
  static_assert(sizeof(Plan) <= sizeof(SM::stage), "the plan is made where the stages go");
  static_assert(AHEAD <= 2, "a piece's three successors are known");
  extern __shared__ __align__(1024) uint8_t smem[];
  SM &sm = *reinterpret_cast<SM *>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();
  Plan &plan = *reinterpret_cast<Plan *>(smem);
  plan.build(p);
  if (plan.any_bad()) chunk_bad_requests<T, Plan>(p);
  if (!plan.has_work(p)) {
    if (tid == 0) leave_note(p, make_int4(0, 0, 0, 0));
    return;
  }
  // The last warp works out the pieces: when a piece begins, the three after it are
  // known, as far as the copies of two more tiles and the place after them may reach.
  ChunkWalk<C> walk;
  auto walk_on = [&](int i) {
    ChunkPiece x = {};
    Piece q = {};
    if (walk.next(p, x)) {
      const ChunkUnit &u = x.u;
      const bool cut = x.cut();
      q = {u.b, u.g, u.tok0, u.n_tok, u.pos0, x.t0, x.t1, cut ? walk.cta_of(u, 0) : -1, cut ? walk.cta_of(u, u.tiles - 1) : -1};
    }
    if (lane == 0) sm.pieces[i & 7] = q;
  };
  if (warp == kWarps - 1) {
    walk.start(p, plan);
    for (int i = 0; i < 4; ++i) walk_on(i);
  }
  __syncthreads();  // the plan has been read: its place is the stages'

  // ---- copies
  const uint32_t stages = smem_addr(sm.stage[warp]);
  const bool paged = PAGED;
  uint32_t status = 0;
  int stage_in = 0;
  Steps in = {0, sm.pieces[0].t0};
  uint32_t gone = 0;  // steps in flight whose page does not exist, the last issued in bit 0
  // page of the warp's keys in a tile (contiguous: 0), -1: none, -2: no keys
  auto page_of = [&](const Steps &s) {
    const Piece &q = sm.pieces[s.piece & 7];
    const int key0 = s.tile * C::kKeys + warp * KW;
    if (q.t1 <= q.t0 || key0 >= q.keys) return -2;
    if (!paged) return 0;
    const int id = p.kv.page_table[(int64_t)q.b * p.kv.max_pages + key0 / kPage];
    return id >= 0 && id < p.kv.n_pages ? id : -1;
  };
  int page = page_of(in);
  // A lane's part of a step: bf16 16 bytes of every second row, fp32 of every row.
  // A row's 16-byte parts are swizzled by bits of the row, which change from
  // copy to copy by an exclusive or of the lane's first place.
  constexpr int N = kStep / 2 / 512, PER_ROW = kHeadDim * (int)sizeof(T) / 16;
  const uint32_t to_k = stages + place<T>(lane / PER_ROW, lane % PER_ROW, false);
  const uint32_t to_v = stages + kStep / 2 + place<T>(lane / PER_ROW, lane % PER_ROW, true);
  auto swizzle = [](int i, bool values) {  // of copy i against copy 0
    return F32 ? (uint32_t)(values ? (i >> 1 & 3) << 5 : (i & 1) << 6) : (uint32_t)((2 * i & 6) << 4);
  };
  auto issue = [&] {
    const Piece &q = sm.pieces[in.piece & 7];
    const int key0 = in.tile * C::kKeys + warp * KW;
    gone = gone << 1 | (page == -1);
    if (page >= 0) {
      const int64_t row0 = paged ? ((int64_t)page * p.Hkv + q.g) * kPage + key0 % kPage : ((int64_t)q.b * p.Hkv + q.g) * p.kv.capacity + key0;
      const uint8_t *k = (const uint8_t *)p.kv.k + row0 * kHeadDim * sizeof(T) + lane * 16;
      const uint8_t *v = (const uint8_t *)p.kv.v + row0 * kHeadDim * sizeof(T) + lane * 16;
      const uint32_t dk = to_k + stage_in * kStep, dv = to_v + stage_in * kStep;
      const int n = q.keys - key0;
      if (n >= KW) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          copy16((dk ^ swizzle(i, false)) + i * 512, k + i * 512);
          copy16((dv ^ swizzle(i, true)) + i * 512, v + i * 512);
        }
      } else {  // rows behind the last are not read
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          const bool there = i * (32 / PER_ROW) + lane / PER_ROW < n;
          const int at = there ? i * 512 : -lane * 16;
          copy16_if((dk ^ swizzle(i, false)) + i * 512, k + at, there);
          copy16_if((dv ^ swizzle(i, true)) + i * 512, v + at, there);
        }
      }
    }
    copies_end();
    if (q.t1 <= q.t0) return;
    if (++stage_in == NST) stage_in = 0;
    if (++in.tile == q.t1) in = {in.piece + 1, sm.pieces[(in.piece + 1) & 7].t0};
    page = page_of(in);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) issue();

  const float scale = p.q_scale, lazy = 8.f / scale;
  // a lane's rows of the bf16 operands; two 16-byte parts further on are an exclusive or away
  const uint32_t of_k = place<uint16_t>((lane & 7) + (lane >> 4 << 3), lane >> 3 & 1, false);
  const uint32_t of_v = place<uint16_t>(lane & 15, lane >> 4, true);
  int stage = 0;
  int4 note = make_int4(0, 0, 0, 0);
  for (int number = 0;; ++number) {
    const Piece q = sm.pieces[number & 7];
    if (q.t1 <= q.t0) break;
    const int n_rows = q.n_tok * p.G;
    auto q_row = [&](int r) { return (const T *)p.q + ((int64_t)(q.tok0 + r / p.G) * p.Hq + q.g * p.G + r % p.G) * kHeadDim; };
    // the queries: bf16 as the products' operands, fp32 split into shared memory
    uint32_t qa[F32 ? 1 : MT][F32 ? 1 : 8][4];
    if constexpr (F32) {
      for (int e = tid; e < ROWS * (kHeadDim / 4); e += kThr) {
        const int r = e / (kHeadDim / 4), c = e % (kHeadDim / 4) * 4;
        const float4 x = r < n_rows ? *reinterpret_cast<const float4 *>(q_row(r) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 hi, lo;
        split(x.x, hi.x, lo.x);
        split(x.y, hi.y, lo.y);
        split(x.z, hi.z, lo.z);
        split(x.w, hi.w, lo.w);
        *reinterpret_cast<float4 *>(&sm.q[0][r][c]) = hi;
        *reinterpret_cast<float4 *>(&sm.q[1][r][c]) = lo;
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = i * 16 + h * 8 + g;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(q_row(min(r, n_rows - 1)));
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            qa[i][s][h] = src[s * 8 + t];
            qa[i][s][h + 2] = src[s * 8 + 4 + t];
          }
        }
    }
    if (warp == kWarps - 1) walk_on(number + 4);  // known to all from the barriers at the piece's end
    if (F32) __syncthreads();

    float o[MT][16][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
    for (int tile = q.t0; tile < q.t1; ++tile) {
      __syncwarp();  // the stage that comes next has been read
      issue();
      copies_wait<AHEAD>();
      __syncwarp();
      const uint32_t kb = stages + stage * kStep, vb = kb + kStep / 2;
      const uint8_t *kp = sm.stage[warp][stage], *vp = kp + kStep / 2;
      if (++stage == NST) stage = 0;
      const int left = q.keys - (tile * C::kKeys + warp * KW);  // keys of the warp's that exist
      if (left <= 0) continue;
      if (gone >> AHEAD & 1) {
        status |= MAC_DEV_BAD_PAGE;
        continue;
      }
      // scores: KW keys, 8 per column tile
      constexpr int NT = KW / 8;
      float s[MT][NT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.f;
      if constexpr (F32) {
        // column order within 16: a lane's four neighbours are columns t and t + 4 of two products
#pragma unroll 4
        for (int c = 0; c < kHeadDim / 16; ++c) {
          const float4 kx = *reinterpret_cast<const float4 *>(kp + place<T>(g, c * 4 + t, false));
          float h[4], r[4];
          split(kx.x, h[0], r[0]);
          split(kx.y, h[1], r[1]);
          split(kx.z, h[2], r[2]);
          split(kx.w, h[3], r[3]);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const int at = c * 16 + t * 4;
            const float4 x0 = *reinterpret_cast<const float4 *>(&sm.q[0][i * 16 + g][at]), x1 = *reinterpret_cast<const float4 *>(&sm.q[0][i * 16 + g + 8][at]);
            const float4 y0 = *reinterpret_cast<const float4 *>(&sm.q[1][i * 16 + g][at]), y1 = *reinterpret_cast<const float4 *>(&sm.q[1][i * 16 + g + 8][at]);
            const float a0[4] = {x0.x, x1.x, x0.y, x1.y}, a1[4] = {y0.x, y1.x, y0.y, y1.y};
            mma_parts(s[i][0], a0, a1, h[0], h[1], r[0], r[1]);
            const float b0[4] = {x0.z, x1.z, x0.w, x1.w}, b1[4] = {y0.z, y1.z, y0.w, y1.w};
            mma_parts(s[i][0], b0, b1, h[2], h[3], r[2], r[3]);
          }
        }
      } else {
        const uint32_t at = kb + of_k;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t b[4];
          ldm4(b, (at ^ (c & 3) << 5) + (c >> 2) * 128);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            mma_bf16(s[i][0], qa[i][c], b[0], b[1]);
            mma_bf16(s[i][NT - 1], qa[i][c], b[2], b[3]);
          }
        }
      }
      if (left < KW) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j * 8 + t * 2 + (e & 1) >= left) s[i][j][e] = -INFINITY;
      }
      // weights
      uint32_t pa[MT][4];      // bf16: the weights as an operand
      float ph[MT][4], pl[MT][4];  // fp32: their parts
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            top[e >> 1] = fmaxf(top[e >> 1], s[i][j][e]);
          }
        bool grows = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          grows |= top[h] > m[i][h] + lazy;
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[i][h], top[h]), ms = mn == -INFINITY ? 0.f : mn;
            const float corr = ex2((m[i][h] - ms) * scale);
            m[i][h] = mn;
            l[i][h] *= corr;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              o[i][j][2 * h] *= corr;
              o[i][j][2 * h + 1] *= corr;
            }
          }
        }
        float ms[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) ms[h] = m[i][h] == -INFINITY ? 0.f : m[i][h] * scale;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][j][e] = ex2(fmaf(s[i][j][e], scale, -ms[e >> 1]));
            l[i][e >> 1] += s[i][j][e];
          }
        if constexpr (F32) {
          // the key order of the products is (2 t, 2 t + 1) for columns t and t + 4: what a lane has
          const float w[4] = {s[i][0][0], s[i][0][2], s[i][0][1], s[i][0][3]};
#pragma unroll
          for (int e = 0; e < 4; ++e) split(w[e], ph[i][e], pl[i][e]);
        } else {
          // the weights to bf16, as chunk attention's: the product takes both factors so
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pa[i][0]) : "f"(s[i][0][1]), "f"(s[i][0][0]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pa[i][1]) : "f"(s[i][0][3]), "f"(s[i][0][2]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pa[i][2]) : "f"(s[i][NT - 1][1]), "f"(s[i][NT - 1][0]));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pa[i][3]) : "f"(s[i][NT - 1][3]), "f"(s[i][NT - 1][2]));
        }
      }
      // values
      if constexpr (F32) {
#pragma unroll
        for (int c = 0; c < kHeadDim / 32; ++c) {  // 32 columns: a lane's four neighbours are a column of four products
          const float4 v0 = *reinterpret_cast<const float4 *>(vp + place<T>(2 * t, c * 8 + g, true));
          const float4 v1 = *reinterpret_cast<const float4 *>(vp + place<T>(2 * t + 1, c * 8 + g, true));
          const float a[4] = {v0.x, v0.y, v0.z, v0.w}, b[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float ah, al, bh, bl;
            split(a[e], ah, al);
            split(b[e], bh, bl);
#pragma unroll
            for (int i = 0; i < MT; ++i) mma_parts(o[i][c * 4 + e], ph[i], pl[i], ah, bh, al, bl);
          }
        }
      } else {
        const uint32_t at = vb + of_v;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t b[4];
          ldm4t(b, (at ^ (c & 3) << 5) + (c >> 2) * 128);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            mma_bf16(o[i][2 * c], pa[i], b[0], b[1]);
            mma_bf16(o[i][2 * c + 1], pa[i], b[2], b[3]);
          }
        }
      }
    }

    // ---- the warps' states joined
    if (F32) __syncthreads();  // the queries have been read: their place is the joint's
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
        if (t == 0) sm.ml[warp][i * 16 + h * 8 + g] = make_float2(m[i][h] * scale, l[i][h]);  // base 2
      }
    const int c = blockIdx.x;
    const bool whole = q.c0 < 0;
    constexpr int PER_ROW = COLS / 4;            // threads per row of the joint
    const int row = tid / PER_ROW, col = tid % PER_ROW * 4;
    const bool mine = row < ROWS && row < n_rows;
    float f[kWarps], big = -INFINITY, sum = 0.f;
    float *part = p.part + ((int64_t)(2 * c + (c == q.c0 ? 1 : 0)) * p.part_rows + row) * kChunkStride;
    const int64_t out_row = (int64_t)(q.tok0 + row / p.G) * p.Hq + q.g * p.G + row % p.G;
    float norm = 1.f;
#pragma unroll
    for (int j = 0; j < kHeadDim / COLS; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float *dst = &sm.join[warp][i * 16 + h * 8 + g][t * 8];
            *reinterpret_cast<float4 *>(dst) = make_float4(o[i][j * 4][2 * h], o[i][j * 4 + 1][2 * h], o[i][j * 4 + 2][2 * h], o[i][j * 4 + 3][2 * h]);
            *reinterpret_cast<float4 *>(dst + 4) =
                make_float4(o[i][j * 4][2 * h + 1], o[i][j * 4 + 1][2 * h + 1], o[i][j * 4 + 2][2 * h + 1], o[i][j * 4 + 3][2 * h + 1]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < COLS / 8; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<float2 *>(&sm.join[warp][i * 16 + h * 8 + g][n * 8 + t * 2]) =
                  make_float2(o[i][j * (COLS / 8) + n][2 * h], o[i][j * (COLS / 8) + n][2 * h + 1]);
        }
      }
      __syncthreads();
      if (mine) {
        if (j == 0) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) big = fmaxf(big, sm.ml[w][row].x);
          const float ref = big == -INFINITY ? 0.f : big;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = sm.ml[w][row];
            f[w] = ex2(x.x - ref);
            sum = fmaf(f[w], x.y, sum);
          }
          if (whole) norm = sum == 0.f ? 0.f : 1.f / sum;
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4 *>(&sm.join[w][row][col]);
          x.x = fmaf(f[w], y.x, x.x);
          x.y = fmaf(f[w], y.y, x.y);
          x.z = fmaf(f[w], y.z, x.z);
          x.w = fmaf(f[w], y.w, x.w);
        }
        x = make_float4(x.x * norm, x.y * norm, x.z * norm, x.w * norm);
        if (whole) store_out((T *)p.out + out_row * kHeadDim + j * COLS + col, x);
        else *reinterpret_cast<float4 *>(part + j * COLS + col) = x;
      }
      __syncthreads();
    }
    if (mine && col == 0) {
      if (!whole) *reinterpret_cast<float2 *>(part + kHeadDim) = make_float2(big, sum);
      else if (p.lse) p.lse[out_row] = sum == 0.f ? -INFINITY : big * kLn2 + logf(sum);
    }
    if (c == q.c0) note = make_int4(q.tok0, q.g, n_rows, q.c1);
  }
  copies_wait<0>();
  if (tid == 0) leave_note(p, note);
  if (status && lane == 0) set_status(p.status, status);
}

template <typename T, int MT, typename C>
cudaError_t launch(const ChunkParams &p, int grid, cudaStream_t s) {
  constexpr int kBytes = sizeof(Shared<T, MT>);
  static_assert(kBytes <= (int)kMaxSmem, "shared memory of a CTA");
  static DeviceFlags done[2];
  cudaError_t e;
  if (p.kv.paged) {
    if ((e = prepare_chunk(few_kernel<T, MT, true, C>, done[1], kBytes, 0)) != cudaSuccess) return e;
    return launch_dependent(few_kernel<T, MT, true, C>, grid, kThr, kBytes, s, p);
  }
  if ((e = prepare_chunk(few_kernel<T, MT, false, C>, done[0], kBytes, 0)) != cudaSuccess) return e;
  return launch_dependent(few_kernel<T, MT, false, C>, grid, kThr, kBytes, s, p);
}

}  // namespace

cudaError_t launch_cross_few(const ChunkParams &p, int rows, bool f32, int grid, cudaStream_t s) {
  if (rows == 16) return f32 ? launch<float, 1, FewF32<16>>(p, grid, s) : launch<uint16_t, 1, FewBf16<16>>(p, grid, s);
  return f32 ? launch<float, 2, FewF32<32>>(p, grid, s) : launch<uint16_t, 2, FewBf16<32>>(p, grid, s);
}

}  // namespace mac
