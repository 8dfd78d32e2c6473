// mac_chunk_bf16.cu -- chunk attention in bf16 on the tensor cores.
//
// For a row with rotated query q at position p, over key tiles of 128:
//   S = Q K^T (fp32);  x_j = S_j log2(e)/sqrt(d), j <= p;
//   P_j = 2^(x_j - m) with m a running reference of the row's maximum;
//   l = sum P_j (fp32);  O = sum P_j V_j (P rounded to bf16, sums in fp32);
//   out = O / l;  lse = m ln 2 + ln l.
// P is the one number between the inputs and the output that is held in fewer
// than 32 bits: the product with V takes both factors in bf16, a second part of
// P would make it twice as long (half as much again per tile).  Each weight is
// off by up to 2^-8 of itself, independently, so where the weights are flat the
// output is off by about as much as by its own rounding to bf16: against 64 bits
// 2.1e-3 where the output's rounding alone makes 1.6e-3 (7 tokens at 100), 1.8e-3
// (16384 tokens) and 1.7e-3 (2048 at 32768).  l sums the weights unrounded.
// The reference m moves only when the maximum has grown by more than 8 in
// base 2 (P stays below 2^8, and bf16 keeps the same relative precision
// there), so O is rarely rescaled; any m gives the same quotient.
//
// One CTA per SM, twelve warps:
//   warps 0-3, 4-7  softmax of row tile 0 and 1 (a thread owns a row);
//   warps 8, 11     copy Q and K, and V, by TMA into swizzled shared memory;
//   warp 9          issues the products: S into TMEM from shared memory, and
//                   O += P V with P read back from TMEM;
//   warp 10         works out the CTA's pieces, and clears V rows past the
//                   end of the sequence.
// A unit has up to 256 packed rows (token-major, the G heads of a token
// together), two row tiles of 128.  With 128 rows or fewer both softmax
// groups work on the same rows and take the key tiles in turn.  While one
// group works on its scores the tensor cores work for the other.
//
// TMEM (512 columns): S0, S1, O0, O1, 128 columns each; P overwrites S.
//
// 2048 tokens at 32768, 32 / 8 heads, paged: 640 to 660 us with the merge, 1.65 PFLOP/s
// (up to 752 us in a loop of a second, at the card's power limit).  A pair of
// row tiles and a key tile take 2900 cycles: the products 2048, 2620 with the
// softmax taken out (both operands of S come from shared memory beside the
// copies), the rest is the softmax in the way.  Four single tokens over 131072
// keys: 300 us, 7.1 TB/s of keys and values.
#include <cuda.h>
#include <math.h>

#include "mac_tc.cuh"

namespace mac {
namespace {

constexpr int kTile = 128;                    // rows of a row tile, keys of a key tile
constexpr int kThr = 384;
constexpr int kRegsSoftmax = 208, kRegsOther = 88;  // registers per thread once the roles have split
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThr * 168, "the split comes out of the launch's registers");
constexpr int kStK = 2, kStV = 3, kNSt = kStK + kStV;  // stages of the K ring and of the V ring
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr float kLazy = 8.f;                  // growth of the maximum (base 2) that moves the reference
static_assert(ChunkBf16::kRows == 2 * kTile && ChunkBf16::kKeys == kTile, "tiles");
using Plan = ChunkPlan<ChunkBf16>;

struct Maps {
  CUtensorMap q, k, v;
};

// A piece of a unit, as the roles see it.
struct Piece {
  int b, g;           // request, KV head
  int tok0, n_tok;    // first token (row of the batch), tokens
  int pos0;           // keys that the first token attends
  int t0, t1;         // key tiles
  int end0;           // normal: key tiles of row tile 0 end here (those of row tile 1 at t1)
  int pair;           // both groups on row tile 0, key tiles in turn
  int clear;          // keys of the last tile that exist, if V is to be cleared after them; else kTile
  int c0, c1;         // a cut unit's first and last CTA; else -1
  __device__ int n() const { return t1 - t0; }
  __device__ bool cut() const { return c0 >= 0; }
  // key tiles of group w
  __device__ int count(int w) const { return pair ? (n() - w + 1) >> 1 : w ? t1 - t0 : max(0, end0 - t0); }
};

struct Control {
  unsigned long long full[kNSt], empty[kNSt];
  unsigned long long q_full, q_empty, s_full[2], p_full[2], o_full[2], pair_ml, pair_read, tail, fixed, drain;
  uint32_t tmem;
  int abort;
  PieceRing<Piece> pieces;
  float2 ml[2][kTile];                        // states of the two groups that share rows
};
constexpr int kSmemBytes = (kNSt + 2) * kTileBytes + (int)sizeof(Control);
static_assert(kSmemBytes <= (int)kMaxSmem, "shared memory of a CTA");
static_assert(sizeof(Plan) <= kNSt * kTileBytes, "the plan is made where the stages go");

// ---- products ----------------------------------------------------------------
// The products of a tile, D[128 x 128] (+)= A B in eight steps of depth 16;
// bf16 inputs, fp32 sums.  a, b: low words of shared memory descriptors (a of
// tc_values: TMEM).  The whole warp runs them and one lane issues: with its
// control flow uniform the operands stay in uniform registers, where the
// instruction takes them from.  tc_scores ends with one arrival on `bar`
// once all products issued so far have ended.
__device__ __forceinline__ void tc_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %4, %4;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 1024;\n\tadd.u32 y, %2, 1024;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 1026;\n\tadd.u32 y, %2, 1026;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 1028;\n\tadd.u32 y, %2, 1028;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u32 x, %1, 1030;\n\tadd.u32 y, %2, 1030;\n\tmov.b64 a, {x, %4};\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_values(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred q, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 t, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n\t"
      "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 32;\n\tadd.u32 y, %2, 512;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 40;\n\tadd.u32 y, %2, 640;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 48;\n\tadd.u32 y, %2, 768;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "add.u32 x, %1, 56;\n\tadd.u32 y, %2, 896;\n\tmov.b64 b, {y, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(add)
      : "memory");
}
// ---- TMA -------------------------------------------------------------------
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// 32 bytes: a whole sector at once where dst allows it (rows are 256 bytes
// apart, so all of a launch's do or none).
__device__ __forceinline__ void store32(void *dst, const uint32_t *v) {
  if (((uintptr_t)dst & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<uint4 *>(dst) + 1) = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// ---- copies (warps 8 and 11) ---------------------------------------------------
// One ring's copies: key or value tiles into stages st0 .. st0 + NST - 1, and
// (K) the Q tiles.  A paged tile is 8 pages of two 64-column halves, one copy each.
template <bool PAGED, bool IS_K>
__device__ void load_role(const ChunkParams &p, const Maps &maps, uint32_t stages, uint32_t qbuf, Control *ct) {
  constexpr int NST = IS_K ? kStK : kStV, ST0 = IS_K ? 0 : kStK;
  const CUtensorMap *map = IS_K ? &maps.k : &maps.v;
  const int lane = threadIdx.x & 31, half = lane >> 3 & 1, pg = lane & 7;
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  int use = 0;       // stage uses so far
  uint32_t nq = 0, np = 0;  // Q tiles, pieces so far
  Piece q = {};
  while (ct->pieces.take(wait, np, q)) {
    const int n_pages = (q.pos0 + q.n_tok - 1 + kPage - 1) / kPage;  // of the unit's keys
    auto page = [&](int t) {  // page of this lane's copy; out of range where there is none: the copy fills with zeros
      const int k = t * (kTile / kPage) + pg;
      int id = k < n_pages ? p.kv.page_table[(int64_t)q.b * p.kv.max_pages + k] : -1;
      return bad_page(p, id) ? p.kv.n_pages : id;
    };
    int id = PAGED ? page(q.t0) : 0;
    for (int t = q.t0; t < q.t1; ++t) {
      const int next = PAGED && t + 1 < q.t1 ? page(t + 1) : 0;  // ahead of its use
      const int st = ST0 + use % NST;
      if (wait(&ct->empty[st], (use / NST + 1) & 1)) {  // the first round finds the stages free
        const uint32_t bar = smem_addr(&ct->full[st]), dst = stages + st * kTileBytes;
        if (lane == 0) mbar_expect_tx(bar, kTileBytes);
        __syncwarp();
        if (!IS_K || use != p.withhold) {
          if (PAGED) {
            if (lane < 16) tma_4d(dst + half * (kTileBytes / 2) + pg * (kPage * 128), map, 64 * half, 0, q.g, id, bar);
          } else if (lane < 2) {
            tma_3d(dst + lane * (kTileBytes / 2), map, 64 * lane, t * kTile, q.b * p.Hkv + q.g, bar);
          }
        }
        ++use;
      }
      id = next;
      __syncwarp();
      if (IS_K && t == q.t0 && wait(&ct->q_empty, (nq + 1) & 1)) {
        const uint32_t bar = smem_addr(&ct->q_full);
        const int tiles = q.pair ? 1 : 2;
        if (lane == 0) mbar_expect_tx(bar, tiles * kTileBytes);
        __syncwarp();
        if (lane < 2 * tiles)
          tma_3d(qbuf + lane * (kTileBytes / 2), &maps.q, 64 * (lane & 1), q.g * p.G, q.tok0 + (lane >> 1) * (kTile / p.G), bar);
        ++nq;
        __syncwarp();
      }
    }
  }
  // The last copies of every stage land before the CTA gives its shared memory
  // up.  Where all is well they have; another role may give up (and end the CTA)
  // after this warp is through, so this does not go by ct->abort.
  for (int u = use > NST ? use - NST : 0; u < use; ++u)
    if (!IS_K || u != p.withhold) drained(&ct->full[ST0 + u % NST], (u / NST) & 1);
  if (nq) drained(&ct->q_full, (nq - 1) & 1);
}

// ---- products (warp 9) -----------------------------------------------------------
// The tensor cores work through what is issued in order and hold only a few
// products ahead, so whatever this warp does between the last product of one
// group and the first of the other must be short: waits come where products
// are still running, and one whose phase has already come costs one test.
// A branch between two products costs more than code: both groups' products
// from one rolled copy took 711 us for 2048 tokens at 32768 (32 / 8 heads)
// where this takes 656.  The code that a short prompt fetches for a few tiles
// is what that would have saved (six prompts of up to 900 tokens: 77 -> 71 us).
struct RingPos {
  uint32_t st, phase;  // stage, parity of its next completion
  __device__ void step(uint32_t first, uint32_t n) {
    if (++st == first + n) {
      st = first;
      phase ^= 1;
    }
  }
};

__device__ void mma_role(const ChunkParams &p, uint32_t stages, uint32_t qbuf, Control *ct, uint32_t tmem) {
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  RingPos k = {0, 0}, v = {kStK, 0};
  uint32_t np = 0, q_phase = 0, fix_phase = 0, p_phase[2] = {0, 0};
  Piece q = {};
  auto addr = [&](uint32_t st) { return stages + st * kTileBytes; };
  auto commit = [&](unsigned long long *bar) {
    if (!wait.dead) tc_commit(smem_addr(bar));
  };
  auto scores = [&](uint32_t w, uint32_t qa) {  // S_w = Q K^T, then tell group w
    if (wait.dead) return;
    tc_scores(tmem + w * kTile, desc_lo(qa, 16), desc_lo(addr(k.st), 16), idesc(kTile, false), smem_addr(&ct->s_full[w]));
  };
  auto values = [&](uint32_t w, uint32_t add) {  // O_w (+)= P_w V, once P_w is there (and O_w rescaled)
    wait(&ct->p_full[w], w ? p_phase[1] : p_phase[0]);
    tc_fence_after();
    if (wait.dead) return;
    tc_values(tmem + 2 * kTile + w * kTile, tmem + w * kTile, desc_lo(addr(v.st), kTileBytes / 2), idesc(kTile, true), add);
    if (w) p_phase[1] ^= 1; else p_phase[0] ^= 1;
  };
  auto keys_ready = [&] { wait(&ct->full[k.st], k.phase); };
  auto free_keys = [&] {
    commit(&ct->empty[k.st]);
    k.step(0, kStK);
  };
  auto free_values = [&] {
    commit(&ct->empty[v.st]);
    v.step(kStK, kStV);
  };
  while (ct->pieces.take(wait, np, q)) {
    const int n = q.n();
    const bool fix = q.clear < kTile;  // V rows past the end of the sequence are cleared by warp 10
    auto values_ready = [&](bool last) {
      wait(&ct->full[v.st], v.phase);
      if (last && fix) {
        if (!wait.dead && (threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&ct->tail));  // it has landed
        wait(&ct->fixed, fix_phase);
        fix_phase ^= 1;
      }
    };
    wait(&ct->q_full, q_phase);
    q_phase ^= 1;
    keys_ready();
    if (q.pair) {
      // both groups on the same rows, key tiles in turn
      scores(0, qbuf);
      free_keys();
      if (n > 1) {
        keys_ready();
        scores(1, qbuf);
        free_keys();
      }
      if (n <= 2) commit(&ct->q_empty);
      for (int i = 0; i < n; ++i) {
        const uint32_t w = i & 1;
        values_ready(i + 1 == n);
        values(w, i >= 2);
        free_values();
        if (i + 2 < n) {
          keys_ready();
          scores(w, qbuf);
          free_keys();
          if (i + 3 == n) commit(&ct->q_empty);
        } else {
          commit(&ct->o_full[w]);
        }
      }
      continue;
    }
    // a row tile each; those of row tile 0 may end before those of row tile 1
    const int n0 = q.count(0);
    if (n0 > 0) scores(0, qbuf);
    scores(1, qbuf + kTileBytes);
    free_keys();
    if (n == 1) commit(&ct->q_empty);
    for (int i = 0; i < n; ++i) {
      values_ready(i + 1 == n);
      if (i < n0) {
        values(0, i > 0);
        if (i + 1 < n) keys_ready();
        if (i + 1 < n0) scores(0, qbuf);
        else commit(&ct->o_full[0]);
      } else if (i + 1 < n) {
        keys_ready();
      }
      values(1, i > 0);
      if (i + 1 < n) {
        scores(1, qbuf + kTileBytes);
        if (!wait.dead) tc_commit2(smem_addr(&ct->empty[v.st]), smem_addr(&ct->empty[k.st]));
        v.step(kStK, kStV);
        k.step(0, kStK);
        if (i + 2 == n) commit(&ct->q_empty);
      } else {
        commit(&ct->o_full[1]);
        free_values();
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

// ---- the walk, and V rows past the end (warp 10) ---------------------------------
// Zero weights meet whatever the cache holds past the end of a sequence: it
// may be anything, so those rows are cleared in shared memory before the
// product reads them.  That waits for the products, so it comes one piece
// behind the walk.
__device__ void walk_role(const ChunkParams &p, uint8_t *stages, Control *ct, const Plan &plan) {
  const int lane = threadIdx.x & 31;
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  ChunkWalk<ChunkBf16> walk;
  walk.start(p, plan);
  fence_proxy_async();  // the plan has been read: its place is the stages'
  uint32_t nt = 0, last_v = 0;  // tiles cleared; V uses before the next piece
  int clear = kTile;            // of the piece posted last
  for (uint32_t i = 0;; ++i) {
    ChunkPiece x = {};
    const bool more = walk.next(p, x);
    Piece q = {};
    if (more) {
      const ChunkUnit &u = x.u;
      const bool cut = x.cut();
      q.b = u.b;
      q.g = u.g;
      q.tok0 = u.tok0;
      q.n_tok = u.n_tok;
      q.pos0 = u.pos0;
      q.t0 = x.t0;
      q.t1 = x.t1;
      q.end0 = min(x.t1, (u.pos0 + kTile / p.G - 1 + kTile - 1) / kTile);
      q.pair = u.n_tok * p.G <= kTile;
      q.clear = x.t1 == u.tiles ? min(kTile, u.a + u.n - (x.t1 - 1) * kTile) : kTile;
      q.c0 = cut ? walk.cta_of(u, 0) : -1;
      q.c1 = cut ? walk.cta_of(u, u.tiles - 1) : -1;
    }
    ct->pieces.post(wait, i, q);
    wait.limit += (long long)(q.t1 - q.t0) << kTileLimitLog;
    if (clear < kTile && wait(&ct->tail, nt & 1)) {
      ++nt;
      uint8_t *v = stages + (kStK + (last_v + kStV - 1) % kStV) * kTileBytes;
      for (int e = clear * 8 + lane; e < kTile * 8; e += 32) {
        *reinterpret_cast<uint4 *>(v + e * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(v + kTileBytes / 2 + e * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ct->fixed));
    }
    if (!more || wait.dead) return;
    clear = q.clear;
    last_v = (last_v + q.n()) % kStV;
  }
}

// ---- softmax, output (warps 0-7) --------------------------------------------------
template <bool PAGED>
__device__ void softmax_role(const ChunkParams &p, Control *ct, uint32_t tmem) {
  const int tid = threadIdx.x, w = tid >> 7, r = tid & 127, lane = tid & 31;
  const uint32_t lanes = (uint32_t)((tid >> 5) & 3) << 21;  // this warp's 32 TMEM lanes
  const uint32_t s_at = tmem + w * kTile + lanes;
  Waiter wait{&ct->abort, p.status, p.wait_limit, false};
  const float scale = p.q_scale, lazy = kLazy / scale;
  const float2 scale2 = make_float2(scale, scale);
  int4 note = make_int4(0, 0, 0, 0);
  uint32_t np = 0, ns = 0, no = 0, n_pair = 0;  // pieces, scores, outputs taken, shared row tiles
  uint32_t status = 0;
  Piece q = {};
  while (ct->pieces.take(wait, np, q)) {
    const int tok = ((q.pair ? 0 : w * kTile) + r) / p.G;   // token of this row
    const int lim = q.pos0 + tok;                         // it attends keys [0, lim)
    const int mine = q.count(w), step = q.pair ? 2 : 1, first = q.t0 + (q.pair ? w : 0);
    const int n_keys = q.pos0 + q.n_tok - 1;
    const int n_rows = q.n_tok * p.G;
    // a warp without a row of the unit only keeps the order of the tiles:
    // its weights are whatever TMEM holds, and so are its rows of O
    const bool idle = (q.pair ? 0 : w * kTile) + (r & ~31) >= n_rows;
    float m = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f);
    for (int i = 0; i < mine; ++i) {
      const int key0 = (first + i * step) * kTile;
      uint32_t gone = 0;  // pages of the tile that do not exist
      if (PAGED) {
        bool bad = false;
        const int pg = key0 / kPage + lane;
        if (lane < kTile / kPage && pg * kPage < n_keys)
          bad = bad_page(p, p.kv.page_table[(int64_t)q.b * p.kv.max_pages + pg]);
        gone = __ballot_sync(0xffffffffu, bad);
      }
      if (!wait(&ct->s_full[w], ns & 1)) continue;
      ++ns;
      tc_fence_after();
      if (idle) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ct->p_full[w]));
        continue;
      }
      float s[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tc_ld32(s + c, s_at + c);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tc_loaded32(s + c);
      if (key0 + kTile > q.pos0 || (PAGED && gone)) {  // some row of the unit does not attend the whole tile (one mask for
        // both reasons: with two the loop's code took 668 us for 2048 tokens at 32768, now 656)
        if (PAGED && gone) status |= MAC_DEV_BAD_PAGE;
        const int left = lim - key0;
#pragma unroll
        for (int pg = 0; pg < kTile / kPage; ++pg) {
          const int of_page = PAGED && (gone >> pg & 1) ? 0 : left;  // keys attended end here
#pragma unroll
          for (int c = pg * kPage; c < (pg + 1) * kPage; ++c) s[c] = c < of_page ? s[c] : -INFINITY;
        }
      }
      float mx[4] = {fmaxf(s[0], s[4]), fmaxf(s[1], s[5]), fmaxf(s[2], s[6]), fmaxf(s[3], s[7])};
#pragma unroll
      for (int c = 8; c < kTile; c += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], fmaxf(s[c + j], s[c + 4 + j]));  // three-input maximum
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (__any_sync(0xffffffffu, top > m + lazy)) {
        const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.f : mn;
        const float corr = ex2((m - ms) * scale);
        m = mn;
        l2.x *= corr;
        l2.y *= corr;
        if (i > 0) {  // the last product into O_w has ended: S_w was issued after it
          const uint32_t o_at = tmem + 2 * kTile + w * kTile + lanes;
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            tc_ld32(o, o_at + c);
            tc_wait_ld();
            tc_loaded32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= corr;
            tc_st32(o_at + c, reinterpret_cast<uint32_t *>(o));
          }
        }
      }
      const float ms = m == -INFINITY ? 0.f : m;
      const float2 neg = make_float2(-ms * scale, -ms * scale);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < kTile; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float2 x = fma2(make_float2(s[c + 2 * j], s[c + 2 * j + 1]), scale2, neg);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          acc[j & 1] = add2(acc[j & 1], x);
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk[j]) : "f"(x.y), "f"(x.x));  // to bf16: see above
        }
        tc_st16(s_at + c / 2, pk);
      }
      l2 = add2(l2, add2(acc[0], acc[1]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ct->p_full[w]));
    }
    // ---- the piece's rows
    float l = l2.x + l2.y;
    // this group's products have ended; in a pair the barrier below says so of the other's
    bool live = true;
    if (mine > 0) {
      live = wait(&ct->o_full[w], no & 1);
      ++no;
    }
    float f[2] = {1.f, 1.f};  // factors of O_w and (pair) of the other group's
    if (q.pair) {
      // (bounded waits instead of a block barrier: a group may give up)
      ct->ml[w][r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ct->pair_ml));
      live &= wait(&ct->pair_ml, n_pair & 1);
      const float2 other = ct->ml[w ^ 1][r];
      const float mn = fmaxf(m, other.x), ms = mn == -INFINITY ? 0.f : mn;
      f[0] = ex2((m - ms) * scale);
      f[1] = ex2((other.x - ms) * scale);
      l = w == 0 ? fmaf(f[0], l, f[1] * other.y) : fmaf(f[1], other.y, f[0] * l);
      m = mn;
    }
    live = live && !wait.dead;
    tc_fence_after();
    const int row = (q.pair ? 0 : w * kTile) + r;
    const bool whole = !q.cut(), keep = live && row < n_rows;
    const int c = blockIdx.x;
    float *part = p.part + ((int64_t)(2 * c + (c == q.c0 ? 1 : 0)) * p.part_rows + row) * kChunkStride;
    const int64_t out_row = (int64_t)(q.tok0 + row / p.G) * p.Hq + q.g * p.G + row % p.G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    // a pair's groups take half of the columns each
#pragma unroll 1
    for (int cc = q.pair ? w * 64 : 0; cc < (q.pair ? w * 64 + 64 : kHeadDim); cc += 32) {
      float o[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0.f;
      if (live) {
        if (mine > 0) {
          tc_ld32(o, tmem + 2 * kTile + w * kTile + lanes + cc);
          tc_wait_ld();
          tc_loaded32(o);
        }
        if (q.pair) {
          float o2[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) o2[j] = 0.f;
          if (q.count(w ^ 1) > 0) {
            tc_ld32(o2, tmem + 2 * kTile + (w ^ 1) * kTile + lanes + cc);
            tc_wait_ld();
            tc_loaded32(o2);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = w == 0 ? fmaf(f[0], o[j], f[1] * o2[j]) : fmaf(f[1], o2[j], f[0] * o[j]);
        }
      }
      if (!keep) continue;
      if (whole) {
        uint16_t *dst = (uint16_t *)p.out + out_row * kHeadDim + cc;
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[e]) : "f"(o[j + 2 * e + 1] * inv), "f"(o[j + 2 * e] * inv));
          store32(dst + j, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 8) store32(part + cc + j, reinterpret_cast<const uint32_t *>(o + j));
      }
    }
    if (keep && !(q.pair && w == 1)) {
      if (!whole) *reinterpret_cast<float2 *>(part + kHeadDim) = make_float2(m * scale, l);  // base 2, as the merge takes it
      else if (p.lse) p.lse[out_row] = l == 0.f ? -INFINITY : m * scale * kLn2 + logf(l);
    }
    if (q.pair) {  // go on once O has been read by both groups
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ct->pair_read));
      wait(&ct->pair_read, n_pair & 1);
      ++n_pair;
    }
    if (c == q.c0) note = make_int4(q.tok0, q.g, n_rows, q.c1);
  }
  if (tid == 0) leave_note(p, wait.dead ? make_int4(0, 0, 0, 0) : note);
  if (status) set_status(p.status, status);
}

template <bool PAGED>
__global__ void __launch_bounds__(kThr, 1) chunk_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  uint8_t *qbuf = smem + kNSt * kTileBytes;
  Control *ct = reinterpret_cast<Control *>(qbuf + 2 * kTileBytes);
  if (smem_addr(smem) & 1023) {  // the swizzled tiles need it; dynamic shared memory starts there
    griddep_wait();
    if (threadIdx.x == 0) {
      set_status(p.status, MAC_DEV_BAD_COPY);
      leave_note(p, make_int4(0, 0, 0, 0));
    }
    return;
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ct->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNSt; ++i) {
      mbar_init(smem_addr(&ct->full[i]), 1);
      mbar_init(smem_addr(&ct->empty[i]), 1);
    }
    mbar_init(smem_addr(&ct->q_full), 1);
    mbar_init(smem_addr(&ct->q_empty), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&ct->s_full[w]), 1);
      mbar_init(smem_addr(&ct->p_full[w]), 4);
      mbar_init(smem_addr(&ct->o_full[w]), 1);
    }
    mbar_init(smem_addr(&ct->pair_ml), 8);
    mbar_init(smem_addr(&ct->pair_read), 8);
    ct->pieces.init(11);  // warps 0-9 and 11
    mbar_init(smem_addr(&ct->tail), 1);
    mbar_init(smem_addr(&ct->fixed), 1);
    mbar_init(smem_addr(&ct->drain), 1);
    ct->abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x == 32) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  griddep_wait();  // from here on the previous kernel's writes are read
  // this CTA's part of the work, the plan made where the stages go
  Plan &plan = *reinterpret_cast<Plan *>(smem);
  plan.build(p);
  if (plan.any_bad()) chunk_bad_requests<uint16_t, Plan>(p);
  const bool work = plan.has_work(p);
  fence_proxy_async();  // copies into the stages come after this
  tc_fence_before();
  block_sync();
  tc_fence_after();
  const uint32_t tmem = ct->tmem;
  if (!work) {
    if (threadIdx.x == 0) leave_note(p, make_int4(0, 0, 0, 0));
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_role<PAGED>(p, ct, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) load_role<PAGED, true>(p, maps, smem_addr(smem), smem_addr(qbuf), ct);
    else if (warp == 11) load_role<PAGED, false>(p, maps, smem_addr(smem), smem_addr(qbuf), ct);
    else if (warp == 9) {
      mma_role(p, smem_addr(smem), smem_addr(qbuf), ct, tmem);
    } else walk_role(p, smem, ct, plan);
  }
  tc_fence_before();
  block_sync();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---- host ---------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeFn)f;
  }();
  return fn;
}

// Tensor map of bf16 elements, boxes 64 elements (128 bytes, swizzled) wide.
bool encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
  const cuuint32_t unit[4] = {1, 1, 1, 1};
  EncodeFn fn = encode_fn();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAGED>
cudaError_t launch(const ChunkParams &p, const Maps &maps, int grid, cudaStream_t s) {
  // with fewer registers at launch the split between the roles would wait forever
  static DeviceFlags done;
  const cudaError_t e = prepare_chunk(chunk_kernel<PAGED>, done, kSmemBytes, (256 * kRegsSoftmax + 128 * kRegsOther) / kThr);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_kernel<PAGED>, grid, kThr, kSmemBytes, s, p, maps);
}

}  // namespace

cudaError_t launch_chunk_bf16(const ChunkParams &p, int grid, cudaStream_t s) {
  Maps maps;
  const cuuint64_t row = kHeadDim * 2;
  const cuuint32_t G = p.G;
  {
    const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)p.Hq, (cuuint64_t)p.T}, strides[2] = {row, row * p.Hq};
    const cuuint32_t box[3] = {64, G, kTile / G};
    if (!encode(&maps.q, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    CUtensorMap *m = i ? &maps.v : &maps.k;
    const void *base = i ? p.kv.v : p.kv.k;
    if (p.kv.paged) {
      const cuuint64_t dims[4] = {kHeadDim, kPage, (cuuint64_t)p.Hkv, (cuuint64_t)p.kv.n_pages};
      const cuuint64_t strides[3] = {row, row * kPage, row * kPage * p.Hkv};
      const cuuint32_t box[4] = {64, kPage, 1, 1};
      if (!encode(m, base, 4, dims, strides, box)) return cudaErrorInvalidValue;
    } else {
      const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)p.kv.capacity, (cuuint64_t)p.B * p.Hkv};
      const cuuint64_t strides[2] = {row, row * p.kv.capacity};
      const cuuint32_t box[3] = {64, kTile, 1};
      if (!encode(m, base, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
  }
  return p.kv.paged ? launch<true>(p, maps, grid, s) : launch<false>(p, maps, grid, s);
}

}  // namespace mac
