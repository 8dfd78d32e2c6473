// mac_chunk_f32.cu -- chunk attention in fp32 on the bf16 tensor cores.
//
// For a row with rotated query q at position p, over key tiles of 64:
//   x_j = q . k_j log2(e)/sqrt(d), j <= p;  m the running maximum;
//   l = sum 2^(x_j - m);  o = sum 2^(x_j - m) v_j;
//   out = o / l;  lse = m ln 2 + ln l.
// An fp32 number is the exact sum of three bf16 ones, a = a0 + a1 + a2, eight
// bits of its significand each (cut off, not rounded), so a product is
//   a b = a0 b0 + (a0 b1 + a1 b0) + (a1 b1 + a0 b2 + a2 b0) + what is left out:
// six bf16 products for one in fp32, each exact in the tensor cores' fp32
// sums.  With a1 up to 2^-7 |a| and a2 up to 2^-15 |a|, a1 b2 + a2 b1 is up to
// 2^-21 |a b| (2^-24 on average) and always has the product's sign: leaving it
// out shrinks |a b|.  The small ones are summed first, so that what the sums cut off is
// small against the result, and a tile's P V is added to o in registers
// (rounded to nearest): errors do not pile up over a long context.
//
// One CTA per SM, 128 packed rows (token-major, the G heads of a token
// together), sixteen warps (registers are split by four warps):
//   warps 0-3    softmax, o: a thread owns a row;
//   warps 4-7, 8-11  read K, and V (and Q together), split them and store the
//                parts, swizzled, in shared memory (rows that are not there
//                as zeros), each warp the rows of one page of a tile;
//   warp 12      issues the products: S (64 columns of TMEM) from shared
//                memory, P V (128 columns) with P's parts (96) in TMEM;
//   warp 13      works out the CTA's pieces.
// The roles' loops are kept short: unrolled in full they did not fit the
// instruction cache together, and its misses took two thirds of the time.
// S of the next tile is made while the softmax runs; K is stored while the
// products of the last weights run, V while the scores do.
//
// 4096 tokens, 8 heads of 2 KV heads: 193 to 217 us, 158 to 178 TFLOP/s of fp32
// products (multiply-adds on the CUDA cores: 945 us).  A tile takes 7200 cycles
// whatever its rows, so single tokens are bound by splitting and products, not
// by HBM: four of 32 / 8 heads at 8192 take 95 us (2.8 TB/s).  Of a tile, its 72
// products 4100 (S 48 of 55, reading Q from shared memory, P V 24 of 60), the
// rest waits for K and V to be split, which is 45 instructions per row and
// warp.  Error against 64 bits 3.2e-7 where fp32 matrix products have 5.6e-7.
#include <math.h>

#include "mac_tc.cuh"

namespace mac {
namespace {

constexpr int kRows = ChunkF32::kRows, kKeys = ChunkF32::kKeys;
constexpr int kThr = 512, kConv = kKeys / kPage;    // threads; warps that split K (V): one for each page of a tile
constexpr int kRegsLaunch = 128, kRegsSoft = 232, kRegsSplit = 104, kRegsMma = 72;  // registers per thread
static_assert(kRegsSoft + 2 * kRegsSplit + kRegsMma <= 4 * kRegsLaunch && kThr * kRegsLaunch <= 65536, "the split comes out of the launch's registers");
constexpr int kQPart = kRows * kHeadDim * 2, kKvPart = kKeys * kHeadDim * 2;  // bytes of one bf16 part of a tile
constexpr uint32_t kColS = 0, kColS1 = 64, kColP = 128, kColO = 256;  // TMEM columns: S twice, P, P V
using Plan = ChunkPlan<ChunkF32>;

// A piece of a unit, as the roles see it.
struct Piece {
  int b, g;           // request, KV head
  int tok0, n_tok;    // first token (row of the batch), tokens
  int pos0;           // keys that the first token attends
  int t0, t1;         // key tiles
  int c0, c1;         // a cut unit's first and last CTA; else -1
};

struct Control {
  unsigned long long k_full, k_free, v_full, v_free, q_full, q_free;
  unsigned long long s_full[2], s_free[2], p_full, o_full, o_free, drain;
  uint32_t tmem;
  int abort;
  PieceRing<Piece> pieces;
};
constexpr int kSmemBytes = 3 * kQPart + 6 * kKvPart + (int)sizeof(Control);
static_assert(kSmemBytes <= (int)kMaxSmem && sizeof(Plan) <= 6 * kKvPart, "shared memory of a CTA");

// ---- products ----------------------------------------------------------------
// 128 x 64 (+)= 128 x 128 . 128 x 64 of one part of Q and one of K; 128 x 128
// (+)= 128 x 64 . 64 x 128 of one part of P and one of V.  The whole warp runs
// them and one lane issues.
__device__ __forceinline__ void tc_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
#define MAC_S(AO, BO, P)                                                                                                  \
  "add.u32 x, %1, " AO ";\n\tadd.u32 y, %2, " BO ";\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t"                    \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " P ";\n\t"
  asm volatile(
      "{\n\t.reg .pred q, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t" MAC_S("0", "0", "q") MAC_S("2", "2", "t") MAC_S("4", "4", "t") MAC_S("6", "6", "t")
          MAC_S("1024", "512", "t") MAC_S("1026", "514", "t") MAC_S("1028", "516", "t") MAC_S("1030", "518", "t") "}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc(kKeys, false)), "n"(kDescHi), "r"(add)
      : "memory");
#undef MAC_S
}
static_assert(kQPart / 2 >> 4 == 1024 && kKvPart / 2 >> 4 == 512, "second halves of Q and K tiles");
__device__ __forceinline__ void tc_values(uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
#define MAC_V(AO, BO, P)                                                                     \
  "add.u32 x, %1, " AO ";\n\tadd.u32 y, %2, " BO ";\n\tmov.b64 b, {y, %4};\n\t"              \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, " P ";\n\t"
  asm volatile(
      "{\n\t.reg .pred q, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t" MAC_V("0", "0", "q") MAC_V("8", "128", "t") MAC_V("16", "256", "t")
          MAC_V("24", "384", "t") "}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc(kHeadDim, true)), "n"(kDescHi), "r"(add)
      : "memory");
#undef MAC_V
}

// (part of the first factor | part of the second << 2), 4 bits each, smallest products first: 2 0, 0 2, 1 1, 1 0, 0 1, 0 0
constexpr uint32_t kPairs = 0x2 | 0x8 << 4 | 0x5 << 8 | 0x1 << 12 | 0x4 << 16 | 0x0 << 20;

__device__ void mma_role(const ChunkParams &p, uint32_t qbuf, uint32_t kbuf, uint32_t vbuf, Control *ct, uint32_t tmem) {
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  uint32_t np = 0, nt = 0, ns = 0, nq = 0;  // pieces, tiles of P V, of S, and Q tiles so far
  const uint32_t qd = desc_lo(qbuf, 16), kd = desc_lo(kbuf, 16), vd = desc_lo(vbuf, kKvPart / 2);
  Piece q = {};
  while (ct->pieces.take(wait, np, q)) {
    const int n = q.t1 - q.t0;
    wait(&ct->q_full, nq & 1);
    ++nq;
    for (int j = 0; j <= n; ++j) {
      if (j < n) {  // S of tile j
        const uint32_t buf = ns & 1;
        wait(&ct->k_full, ns & 1);
        wait(&ct->s_free[buf], ((ns >> 1) + 1) & 1);
        ++ns;
        tc_fence_after();
        if (!wait.dead) {
#pragma unroll 1
          for (uint32_t i = 0; i < 6; ++i) {
            const uint32_t w = kPairs >> 4 * i;
            tc_scores(tmem + kColS + buf * kColS1, qd + (w & 3) * (kQPart >> 4), kd + (w >> 2 & 3) * (kKvPart >> 4), i);
          }
          tc_commit(smem_addr(&ct->s_full[buf]));
          tc_commit(smem_addr(&ct->k_free));
          if (j + 1 == n) tc_commit(smem_addr(&ct->q_free));
        }
      }
      if (j > 0) {  // P V of tile j - 1
        wait(&ct->v_full, nt & 1);
        wait(&ct->p_full, nt & 1);
        wait(&ct->o_free, (nt + 1) & 1);
        ++nt;
        tc_fence_after();
        if (!wait.dead) {
#pragma unroll 1
          for (uint32_t i = 0; i < 6; ++i) {
            const uint32_t w = kPairs >> 4 * i;
            tc_values(tmem + kColO, tmem + kColP + (w & 3) * (kKeys / 2), vd + (w >> 2 & 3) * (kKvPart >> 4), i);
          }
          tc_commit(smem_addr(&ct->o_full));
          tc_commit(smem_addr(&ct->v_free));
        }
      }
    }
  }
  // every product has ended before the CTA gives its memory up
  tc_commit(smem_addr(&ct->drain));
  if (!drained(&ct->drain, 0)) {
    *(volatile int *)&ct->abort = 1;
    set_status(p.status, MAC_DEV_WAIT_TIMEOUT);
  }
}

// ---- splitting (warps 4-11) -----------------------------------------------------
// The next parts of four neighbours, packed, and what is left of them (of an
// infinity NaN: a row that attends one is NaN).
__device__ __forceinline__ uint2 split4(float4 &f) {
  const uint32_t a = __float_as_uint(f.x), b = __float_as_uint(f.y), c = __float_as_uint(f.z), d = __float_as_uint(f.w);
  const float2 lo = add2(make_float2(f.x, f.y), make_float2(-__uint_as_float(a & 0xffff0000u), -__uint_as_float(b & 0xffff0000u)));
  const float2 hi = add2(make_float2(f.z, f.w), make_float2(-__uint_as_float(c & 0xffff0000u), -__uint_as_float(d & 0xffff0000u)));
  f = make_float4(lo.x, lo.y, hi.x, hi.y);
  return make_uint2(__byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
}

// Four floats of row r, columns 4 lane .. 4 lane + 3, as three bf16 parts into a tile of ROWS rows.
template <int ROWS>
__device__ __forceinline__ void put_parts(uint8_t *tile, int r, int lane, float4 f) {
  constexpr int kPart = ROWS * kHeadDim * 2;
  const int half = lane >> 4, chunk = lane >> 1 & 7;
  uint8_t *dst = tile + half * (ROWS * 128) + r * 128 + ((chunk ^ (r & 7)) << 4) + (lane & 1) * 8;
  *reinterpret_cast<uint2 *>(dst) = split4(f);
  *reinterpret_cast<uint2 *>(dst + kPart) = split4(f);
  *reinterpret_cast<uint2 *>(dst + 2 * kPart) = split4(f);
}

// Four floats, zeros where !ok; nothing waits for them before they are used.
__device__ __forceinline__ float4 load_if(const float *src, bool ok) {
  float4 f;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
      "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t@p ld.global.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&f"(f.x), "=&f"(f.y), "=&f"(f.z), "=&f"(f.w)
      : "l"(src), "r"((int)ok));
  return f;
}

template <bool PAGED>
__device__ void split_role(const ChunkParams &p, uint8_t *qbuf, uint8_t *kbuf, uint8_t *vbuf, Control *ct) {
  const int lane = threadIdx.x & 31, me_q = (threadIdx.x >> 5) - 4, me = me_q & (kConv - 1);
  const bool is_k = me_q < kConv;  // one copy of the code for both: see above
  const float *src = (const float *)(is_k ? p.kv.k : p.kv.v) + lane * 4;
  unsigned long long *full = is_k ? &ct->k_full : &ct->v_full, *free = is_k ? &ct->k_free : &ct->v_free;
  uint8_t *tile = is_k ? kbuf : vbuf;
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  uint32_t np = 0, nt = 0, nq = 0;  // pieces, tiles and Q tiles so far
  Piece q = {};
  auto hand_over = [&](unsigned long long *bar) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(bar));
  };
  while (ct->pieces.take(wait, np, q)) {
    const int n_rows = q.n_tok * p.G, n_keys = q.pos0 + q.n_tok - 1;
    // this warp's 16 rows of tile t: the element of their first one (-1: no
    // page), and how many of them are keys of the unit
    auto at = [&](int t) -> int64_t {
      if (!PAGED) return (((int64_t)q.b * p.Hkv + q.g) * p.kv.capacity + t * kKeys + me * kPage) * kHeadDim;
      const int k = t * (kKeys / kPage) + me;
      const int id = t < q.t1 && (int64_t)k * kPage < n_keys ? p.kv.page_table[(int64_t)q.b * p.kv.max_pages + k] : -1;
      return id >= 0 && id < p.kv.n_pages ? ((int64_t)id * p.Hkv + q.g) * kPage * kHeadDim : -1;
    };
    float4 f[kPage];
    auto load = [&](int t, int64_t first) {
      const int n = first < 0 ? 0 : n_keys - (t * kKeys + me * kPage);
      const float *row = src + (first < 0 ? 0 : first);
#pragma unroll
      for (int i = 0; i < kPage; ++i) f[i] = load_if(row + i * kHeadDim, i < n);
    };
    load(q.t0, at(q.t0));
    if (wait(&ct->q_free, (nq + 1) & 1)) {
      ++nq;
#pragma unroll 2
      for (int r = me_q; r < kRows; r += 2 * kConv) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_rows)
          x = *reinterpret_cast<const float4 *>((const float *)p.q + ((int64_t)(q.tok0 + r / p.G) * p.Hq + q.g * p.G + r % p.G) * kHeadDim + lane * 4);
        put_parts<kRows>(qbuf, r, lane, x);
      }
      hand_over(&ct->q_full);
    }
    int64_t next = at(q.t0 + 1);  // a tile ahead of its use
    for (int t = q.t0; t < q.t1; ++t, ++nt) {
      if (wait(free, (nt + 1) & 1)) {
#pragma unroll 1
        for (int c = 0; c < kPage; c += kPage / 2) {
#pragma unroll
          for (int i = 0; i < kPage / 2; ++i) put_parts<kKeys>(tile, me * kPage + c + i, lane, f[i]);
#pragma unroll
          for (int i = 0; i < kPage / 2; ++i) f[i] = f[i + kPage / 2];
        }
        if (!is_k || (int)nt != p.withhold) hand_over(full);
      }
      // only now: the fence of the hand-over would wait for loads in flight
      if (t + 1 < q.t1) load(t + 1, next);
      next = at(t + 2);
    }
  }
}

// ---- the walk (warp 13) -----------------------------------------------------------
__device__ void walk_role(const ChunkParams &p, Control *ct, const Plan &plan) {
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  ChunkWalk<ChunkF32> walk;
  walk.start(p, plan);
  for (uint32_t i = 0;; ++i) {
    ChunkPiece x = {};
    const bool more = walk.next(p, x);
    Piece q = {};
    if (more) {
      const ChunkUnit &u = x.u;
      const bool cut = x.cut();
      q = {u.b, u.g, u.tok0, u.n_tok, u.pos0, x.t0, x.t1, cut ? walk.cta_of(u, 0) : -1, cut ? walk.cta_of(u, u.tiles - 1) : -1};
    }
    ct->pieces.post(wait, i, q);
    wait.limit += (long long)(q.t1 - q.t0) << kTileLimitLog;
    if (!more || wait.dead) return;
  }
}

// ---- softmax and output (warps 0-3) -----------------------------------------------
template <bool PAGED>
__device__ void row_role(const ChunkParams &p, Control *ct, uint32_t tmem) {
  const int tid = threadIdx.x, r = tid, lane = tid & 31;
  const uint32_t lanes = (uint32_t)(tid >> 5) << 21;  // this warp's 32 TMEM lanes
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  const float scale = p.q_scale;
  uint32_t np = 0, nt = 0, status = 0;
  int4 note = make_int4(0, 0, 0, 0);
  Piece q = {};
  auto arrive = [&](unsigned long long *bar) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(bar));
  };
  while (ct->pieces.take(wait, np, q)) {
    const int lim = q.pos0 + r / p.G;  // keys [0, lim) are the row's
    const int n = q.t1 - q.t0, n_rows = q.n_tok * p.G, n_keys = q.pos0 + q.n_tok - 1;
    const bool idle = (r & ~31) >= n_rows;  // no row of this warp: it only keeps the order of the tiles
    float m = -INFINITY, l = 0.f, o[kHeadDim];
#pragma unroll
    for (int c = 0; c < kHeadDim; ++c) o[c] = 0.f;
    // o = o corr + P V of the last tile
    auto accumulate = [&](float corr) {
      tc_fence_after();
      if (!idle) {
#pragma unroll
        for (int c = 0; c < kHeadDim; c += 16) {
          float v[16];
          tc_ld16(v, tmem + kColO + c + lanes);
          tc_wait_ld();
          tc_loaded16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[c + j] = fmaf(o[c + j], corr, v[j]);
        }
      }
      arrive(&ct->o_free);
    };
    {
      float corr_before = 0.f;
      for (int j = 0; j < n; ++j, ++nt) {
        const int key0 = (q.t0 + j) * kKeys;
        uint32_t gone = 0;  // pages of the tile that do not exist
        if (PAGED) {
          bool bad = false;
          const int pg = key0 / kPage + lane;
          if (lane < kKeys / kPage && pg * kPage < n_keys) {
            const int id = p.kv.page_table[(int64_t)q.b * p.kv.max_pages + pg];
            bad = id < 0 || id >= p.kv.n_pages;
          }
          gone = __ballot_sync(0xffffffffu, bad);
          if (gone) status |= MAC_DEV_BAD_PAGE;
        }
        // (a barrier for each of the two: both may be there before this warp looks at the first)
        if (!wait(&ct->s_full[nt & 1], nt >> 1 & 1)) continue;
        tc_fence_after();
        const uint32_t s_at = tmem + kColS + (nt & 1) * kColS1 + lanes;
        const int left = key0 + kKeys > q.pos0 ? lim - key0 : kKeys;  // keys of the tile that the row attends
        // 32 scores at a time, those that are not the row's at -inf
        auto scores = [&](float *s, int c0) {
          tc_ld32(s, s_at + c0);
          tc_wait_ld();
          tc_loaded32(s);
          if (left < c0 + 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = c0 + c < left ? s[c] : -INFINITY;
          }
          if (PAGED && gone) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = (gone >> ((c0 + c) / kPage)) & 1 ? -INFINITY : s[c];
          }
        };
        float corr = 0.f, ms = 0.f;
        if (!idle) {
          float top = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            float s[32];
            scores(s, c0);
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 32; c += 4)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[c + e]);
            top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          }
          // the maximum in base 2, rounded once: every weight and the lse go by the same number
          const float mn = fmaxf(m, top * scale);
          ms = mn == -INFINITY ? 0.f : mn;
          corr = ex2(m - ms);
          m = mn;
          l *= corr;
        }
        if (j > 0 && !wait(&ct->o_full, (nt - 1) & 1)) continue;  // the last tile's P has been read
        tc_fence_after();
        if (!idle) {
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            float s[32];
            scores(s, c0);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 x = fma2(make_float2(s[c], s[c + 1]), make_float2(scale, scale), make_float2(-ms, -ms));
              s[c] = ex2(x.x);
              s[c + 1] = ex2(x.y);
              acc[c >> 1 & 1] = add2(acc[c >> 1 & 1], make_float2(s[c], s[c + 1]));
            }
            acc[0] = add2(acc[0], acc[1]);
            l += acc[0].x + acc[0].y;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              uint32_t w[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const uint32_t a = __float_as_uint(s[c]), b = __float_as_uint(s[c + 1]);
                w[c / 2] = __byte_perm(a, b, 0x7632);
                s[c] -= __uint_as_float(a & 0xffff0000u);
                s[c + 1] -= __uint_as_float(b & 0xffff0000u);
              }
              tc_st16(tmem + kColP + part * (kKeys / 2) + c0 / 2 + lanes, w);
            }
          }
          tc_wait_st();
        }
        arrive(&ct->p_full);
        if (lane == 0) mbar_arrive(smem_addr(&ct->s_free[nt & 1]));
        if (j > 0) accumulate(corr_before);
        corr_before = corr;
      }
      if (wait(&ct->o_full, (nt - 1) & 1)) accumulate(corr_before);
    }
    // ---- the piece's rows: a whole unit goes out, a piece of one leaves its state
    const bool whole = q.c0 < 0, keep = !wait.dead && r < n_rows;
    const int c = blockIdx.x;
    if (keep) {
      const int64_t row = (int64_t)(q.tok0 + r / p.G) * p.Hq + q.g * p.G + r % p.G;
      const float f = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      float *part = p.part + ((int64_t)(2 * c + (c == q.c0 ? 1 : 0)) * p.part_rows + r) * kChunkStride;
      float *dst = (whole ? (float *)p.out + row * kHeadDim : part);
#pragma unroll
      for (int e = 0; e < kHeadDim; e += 4) store_out(dst + e, make_float4(o[e] * f, o[e + 1] * f, o[e + 2] * f, o[e + 3] * f));
      if (!whole) *reinterpret_cast<float2 *>(part + kHeadDim) = make_float2(m, l);
      else if (p.lse) p.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
    }
    if (c == q.c0) note = make_int4(q.tok0, q.g, n_rows, q.c1);
  }
  if (tid == 0) leave_note(p, wait.dead ? make_int4(0, 0, 0, 0) : note);
  if (status) set_status(p.status, status);
}

template <bool PAGED>
__global__ void __launch_bounds__(kThr, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  uint8_t *qbuf = smem, *kbuf = smem + 3 * kQPart, *vbuf = kbuf + 3 * kKvPart;
  Control *ct = reinterpret_cast<Control *>(vbuf + 3 * kKvPart);
  if (smem_addr(smem) & 1023) {  // the swizzled tiles need it; dynamic shared memory starts there
    griddep_wait();
    if (threadIdx.x == 0) {
      set_status(p.status, MAC_DEV_BAD_COPY);
      leave_note(p, make_int4(0, 0, 0, 0));
    }
    return;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ct->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&ct->k_full), kConv);
    mbar_init(smem_addr(&ct->v_full), kConv);
    mbar_init(smem_addr(&ct->q_full), 2 * kConv);
    mbar_init(smem_addr(&ct->k_free), 1);
    mbar_init(smem_addr(&ct->v_free), 1);
    mbar_init(smem_addr(&ct->q_free), 1);
    mbar_init(smem_addr(&ct->s_full[0]), 1);
    mbar_init(smem_addr(&ct->s_full[1]), 1);
    mbar_init(smem_addr(&ct->o_full), 1);
    mbar_init(smem_addr(&ct->drain), 1);
    mbar_init(smem_addr(&ct->s_free[0]), 4);
    mbar_init(smem_addr(&ct->s_free[1]), 4);
    mbar_init(smem_addr(&ct->p_full), 4);
    mbar_init(smem_addr(&ct->o_free), 4);
    ct->pieces.init(13);  // warps 0-12
    ct->abort = 0;
    mbar_fence_init();
  }
  griddep_wait();  // from here on the previous kernel's writes are read
  Plan &plan = *reinterpret_cast<Plan *>(kbuf);  // made where the K and V tiles go
  plan.build(p);
  if (plan.any_bad()) chunk_bad_requests<float, Plan>(p);
  const bool work = plan.has_work(p);
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = ct->tmem;
  if (!work) {
    if (threadIdx.x == 0) leave_note(p, make_int4(0, 0, 0, 0));
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    row_role<PAGED>(p, ct, tmem);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSplit));
    split_role<PAGED>(p, qbuf, kbuf, vbuf, ct);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    if (warp == 12) mma_role(p, smem_addr(qbuf), smem_addr(kbuf), smem_addr(vbuf), ct, tmem);
    else if (warp == 13) walk_role(p, ct, plan);
  }
  tc_fence_before();
  block_sync();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <bool PAGED>
cudaError_t launch(const ChunkParams &p, int grid, cudaStream_t s) {
  // with fewer registers at launch the split between the roles would wait forever
  static DeviceFlags done;
  const cudaError_t e = prepare_chunk(chunk_kernel<PAGED>, done, kSmemBytes, kRegsLaunch);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_kernel<PAGED>, grid, kThr, kSmemBytes, s, p);
}

}  // namespace

cudaError_t launch_chunk_f32(const ChunkParams &p, int grid, cudaStream_t s) {
  return p.kv.paged ? launch<true>(p, grid, s) : launch<false>(p, grid, s);
}

}  // namespace mac
