// mac_beam_select.cu -- beam search's selection over beams and vocabulary.
//
// For the beams j of a group, with their scores c_j and logits x_jv:
//   L_j = ln sum_v exp x_jv;   s_jv = c_j + x_jv - L_j;
// the n_out largest s of the group, ties to the lowest (j, v).
//
// One kernel.  Its CTAs read every logit once, a CTA a piece of a row: its threads
// keep running sums of exponentials and their largest logit.  Within a row the
// order of s is that of x, so a piece's n_out best by (x, lowest v) are all that
// can be chosen of it.  They are found by a threshold: the n_out-th largest of the
// maxima of 32 groups of threads is a lower bound that few logits pass.  The
// logits of the few threads whose largest one passes are read again, by all
// threads (by themselves they took half of all instructions, as nearly every
// warp has such a thread); what passes is ranked by counting.  The last of a
// group's CTAs joins the pieces and ranks the beams' candidates against one another.
//
// Across beams the order depends on L.  The sums are in fp32, so L is known to
// kSlack only; where that leaves the order of a candidate that counts open
// (two beams' scores within twice that: once in some thousand groups), the
// beams in question are summed again to 2^-38 and the candidates ranked anew.
// So the choice is that of the exact scores, however the card adds.
//
// In a graph (us; floor: bytes at 6.7 TB/s): 4 beams of 32000 bf16 logits 6.7 (0.04);
// 64 of 128000 9.4 from L2, 10.9 from HBM (2.4); 256 of 50001 fp32 logits, 16 of
// each 8 beams, 13.4 and 16.5 (7.6).  Bound by barriers, trips to L2 and code that is
// fetched for the first time (about 3 us of a scan, 3.5 of a choice), then by the
// scan's CTAs, which end together: their thresholds and rankings overlap nothing.
// All CTAs run at once, four to an SM at most: with a fifth as many again 12.2 and
// 14.8 of 9.4 and 13.4, with three per SM 9.4 and 13.2, with two 11.3 and 13.3.  With
// the choice a kernel of its own, whose CTAs start ahead, 7.0, 9.6 and 15.8 where this
// took 6.8, 9.4 and 14.9, and 13.8, 15.8 and 20.8 where this took 11.1, 13.0 and 19.4 of
// calls one after another from Python.  A beam summed again takes its group's CTA 12 us
// of 32000 logits, 65 of 128000 (instructions: some 100 for each logit).
#include <cuda_bf16.h>
#include <math.h>

#include "mac_beam.cuh"
#include "mac_tc.cuh"

namespace mac {
namespace {

constexpr int kThr = kScanThreads, kWarps = kThr / 32, kGroups8 = kThr / 8;
static_assert(kGroups8 == 32 && kMaxPicks <= kGroups8, "a lane holds a group's maximum; the threshold is one of them");
constexpr int kRoom = 1024;  // candidates that are ranked at once
// Bound of the error of L, relative to the sum.  An exponent (x - ref) log2 e is
// off by 2.3 2^-24 of itself (the difference, the product, the constant), and the
// mean of ref - x under the softmax is at most ln V + 1 <= 14.9: 2.0e-6.  ex2 is
// off by 2^-22: of a term, of the moves of its reference (1.6 with every move by
// e^-1 or less), of the joins in a CTA and of the pieces: 1.1e-6.  Sums round 7, 8 and
// 7 times by 2^-24 (a thread's batches are added with their rounded parts): 1.3e-6.
// The logarithm 2^-22 ln 2.  4.6e-6 in all.
constexpr double kSlack = 5.0 / (1 << 20);
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ unsigned long long key_of(float x, int v) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 and 0 are one value
  return (unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)v);
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int token_of(unsigned long long key) { return (int)(0xffffffffu - (uint32_t)key); }

// Leaves the n-th largest of 32 values in *nth (1 <= n <= 32): eight threads rank a value.
__device__ __forceinline__ void find_nth(const float *values, int n, float *nth) {
  const int k = threadIdx.x >> 3, part = threadIdx.x & 7;
  const float g = values[k];
  const float4 o = reinterpret_cast<const float4 *>(values)[part];
  int above = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = j == 0 ? o.x : j == 1 ? o.y : j == 2 ? o.z : o.w;
    above += x > g || (x == g && part * 4 + j < k);
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) above += __shfl_xor_sync(0xffffffffu, above, d);
  if (part == 0 && above == n - 1) *nth = g;
}

// put(i, rank of i) for each of c things, four threads to one; above(i, j): j goes before i.
template <typename A, typename P>
__device__ __forceinline__ void rank_all(int c, A above, P put) {
  for (int i0 = 0; i0 < c; i0 += kThr / 4) {
    const int i = i0 + (threadIdx.x >> 2);
    int rank = 0;
    if (i < c)
      for (int j = threadIdx.x & 3; j < c; j += 4) rank += above(i, j);
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (i < c && (threadIdx.x & 3) == 0) put(i, rank);
  }
}

// Whether a beam has next tokens at all: not finished, with a finite score.
__device__ __forceinline__ bool goes_on(const SelectParams &p, int b) {
  const float c = p.scores[b];
  return !(p.done && p.done[b] != 0) && c > -INFINITY && c < INFINITY;
}

// The logits of a row: `head` elements up to a 16-byte boundary, `full` vectors of 16 bytes, a tail.
template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T *at;
  int head, full, tail0, V;
  __device__ Row(const SelectParams &p, int b) {
    at = (const T *)p.logits + b * p.stride;
    V = p.V;
    const int behind = (int)(((uintptr_t)at & 15) / sizeof(T));
    head = behind ? min(VEC - behind, V) : 0;
    full = (V - head) / VEC;
    tail0 = head + full * VEC;
  }
  __device__ int token(int i) const { return head + i * VEC; }  // of vector i's first element
  __device__ const uint4 *vec(int i) const { return reinterpret_cast<const uint4 *>(at + token(i)); }
  // Element k of the head and the tail, -1: there is none.
  __device__ int loose(int k) const {
    const int v = k < head ? k : tail0 + k - head;
    return k < head + V - tail0 ? v : -1;
  }
};

// A running sum of exponentials, sh + sl relative to e^ref.  The reference moves
// only when a logit is above it by more than 1, so that what a move rounds
// counts for less with every later one.
struct Running {
  float ref = -INFINITY, sh = 0.f, sl = 0.f, mx = -INFINITY;
  __device__ __forceinline__ void reach(float top) {
    mx = fmaxf(mx, top);
    if (top > ref + 1.f) {
      const float f = ex2((ref - top) * kLog2e);
      sh *= f;
      sl *= f;
      ref = top;
    }
  }
  __device__ __forceinline__ float origin() const { return ref == -INFINITY ? 0.f : ref; }
  __device__ __forceinline__ void add(float x) {  // rounded parts kept
    const float a = sh + x, b = a - sh;
    sl += (sh - (a - b)) + (x - b);
    sh = a;
  }
};

__device__ __forceinline__ float top_of(const uint4 &u, uint16_t) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top_of(const uint4 &u, float) {
  return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}

struct ScanShared {
  __align__(16) float gmax[kGroups8];
  float wsum[kWarps], nth;
  unsigned long long room[kRoom];
  unsigned long long wbest[kWarps];
  uint8_t passed[kThr];
  int count, n_passed;
};

// Piece `seg` of beam b's row; U vectors of a thread at a time, the next ones on
// their way meanwhile.
template <typename T, int U>
__device__ __forceinline__ void scan_piece(const SelectParams &p, ScanShared &sm, int seg, int b) {
  constexpr int VEC = Row<T>::VEC;
  constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<T> row(p, b);
  // A thread's place among the vectors of a step.  Where they are too few for twice
  // n_out groups of eight neighbours, neighbours are in groups of their own (32 beams of
  // 218 logits, 16 of each 16: 13.3 -> 10.6; of full steps, which they read apart, + 0.5).
  const bool spread = U == 1 && row.full - seg * kThr < min(16 * p.n_out, kThr);
  const int turn = spread ? (tid & 7) << 5 | tid >> 3 : tid;
  const int i0 = seg * p.steps * kThr + turn;
  if (tid == 0) sm.count = sm.n_passed = 0;

  Running r;
  uint4 cur[U], next[U];
  auto load = [&](uint4 *x, int k) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (k + u) * kThr;
      x[u] = make_uint4(kNone, kNone, kNone, kNone);
      if (k + u < p.steps && i < row.full) x[u] = *row.vec(i);
    }
  };
  load(cur, 0);
  const int extra = seg == p.segs - 1 ? row.loose(turn) : -1;  // the last piece takes the row's ends
  const float loose = extra >= 0 ? elem_f32<T>(row.at, extra) : -INFINITY;
  for (int k = 0; k < p.steps; k += U) {
    if (k + U < p.steps) load(next, k + U);
    float top = top_of(cur[0], T());
#pragma unroll
    for (int u = 1; u < U; ++u) top = fmaxf(top, top_of(cur[u], T()));
    r.reach(top);
    const float o = -r.origin();
    float2 acc[4] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[VEC];
      unpack16<T>(cur[u], f);
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const float2 t = fma2(add2(make_float2(f[e], f[e + 1]), make_float2(o, o)), make_float2(kLog2e, kLog2e), make_float2(0.f, 0.f));
        acc[e / 2 & 3] = add2(acc[e / 2 & 3], make_float2(ex2(t.x), ex2(t.y)));
      }
    }
    const float2 s = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
    r.add(s.x + s.y);
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = next[u];
  }
  if (extra >= 0) {
    r.reach(loose);
    r.add(ex2((loose - r.origin()) * kLog2e));
  }
  const float mx = r.mx;
  float g = mx;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  if ((lane & 7) == 0) sm.gmax[tid >> 3] = g;
  __syncthreads();
  find_nth(sm.gmax, p.n_out, &sm.nth);
  g = sm.gmax[lane];
#pragma unroll
  for (int d = 16; d; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  const float m = g;
  // NaN and +inf among the logits make the sum NaN
  float s = r.sh + r.sl;
  if (m > -INFINITY) s *= ex2((r.ref - m) * kLog2e);
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) sm.wsum[warp] = s;
  __syncthreads();
  const float least = sm.nth;
  // the threads whose logits may pass, looked through by all of them
  if (mx >= least && mx > -INFINITY) sm.passed[atomicAdd(&sm.n_passed, 1)] = (uint8_t)turn;
  __syncthreads();
  auto take = [&](float x, int v) {
    if (x >= least && x > -INFINITY) {
      const int at = atomicAdd(&sm.count, 1);
      if (at < kRoom) sm.room[at] = key_of(x, v);
    }
  };
  const int n_vecs = sm.n_passed * p.steps;
  for (int q = tid; q < n_vecs; q += kThr) {
    const int k = q / sm.n_passed, i = (seg * p.steps + k) * kThr + sm.passed[q - k * sm.n_passed];
    if (i >= row.full) continue;
    const uint4 u = *row.vec(i);
    float x[VEC];
    unpack16<T>(u, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) take(x[e], row.token(i) + e);
  }
  if (extra >= 0) take(loose, extra);
  __syncthreads();
  const int c = sm.count;
  unsigned long long *out = p.keys + (int64_t)b * p.n_out * p.segs + seg;  // its r-th best at out[r * segs]
  if (tid == 0) {
    float all = (sm.wsum[0] + sm.wsum[1]) + (sm.wsum[2] + sm.wsum[3]);
    all += (sm.wsum[4] + sm.wsum[5]) + (sm.wsum[6] + sm.wsum[7]);
    p.ml[(int64_t)b * p.segs + seg] = make_float2(m, all);
  }
  if (c <= kRoom) {
    rank_all(c, [&](int i, int j) { return sm.room[j] > sm.room[i]; }, [&](int i, int rank) {
      if (rank < p.n_out) out[rank * p.segs] = sm.room[i];
    });
    for (int i = c + tid; i < p.n_out; i += kThr) out[i * p.segs] = 0;
    return;
  }
  // more logits of one value than there is room for: one at a time, the best below the last
  // f(value, token) of this thread's logits, read again
  auto each = [&](auto f) {
#pragma unroll 1
    for (int k = 0; k < p.steps; ++k) {
      const int i = i0 + k * kThr;
      if (i >= row.full) break;
      const uint4 u = *row.vec(i);
      float x[VEC];
      unpack16<T>(u, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(x[e], row.token(i) + e);
    }
    if (extra >= 0) f(loose, extra);
  };
  unsigned long long last = ~0ull;
  for (int q = 0; q < p.n_out; ++q) {
    unsigned long long best = 0;
    each([&](float x, int v) {
      if (x > -INFINITY) {
        const unsigned long long k = key_of(x, v);
        if (k < last && k > best) best = k;
      }
    });
#pragma unroll
    for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
    __syncthreads();  // the last round's have been read
    if (lane == 0) sm.wbest[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = max(best, sm.wbest[w]);
    if (tid == 0) out[q * p.segs] = best;
    last = best;
  }
}
static_assert(kWarps == 8, "the sum over the warps");

// ---- the sum again, to 2^-38 ----------------------------------------------------
// exp d for d <= 0 as an unevaluated sum of two floats, by the table method (P. T. P.
// Tang, "Table-driven implementation of the exponential function", 1989):
// d = k ln2 / 64 + r, exp d = 2^(k / 64) (1 + r + r^2 / 2 + r^3 / 6 + r^4 / 24), with
// |r| < 0.0055, r and the powers of two held in two floats each.  What is left
// out is below r^5 / 120 < 2^-44; the terms from r^2 on are rounded once, 2^-24 of
// at most 2^-16.
struct Precise {
  float2 power[64];  // 2^(j / 64)
};

__device__ __forceinline__ float2 exp2f2(const Precise &t, float x, float m) {
  const float d = x - m, bb = d - x;
  const float dh = fmaxf(d, -80.f);  // no branch: a thread's logits are worked on together
  const float dl = (x - (d - bb)) + (-m - bb);  // x - m = d + dl exactly
  const float k = rintf(dh * 92.332482616893657f);  // 64 / ln 2
  // ln 2 / 64 = c0 + c1 + c2; c0 and c1 have 9 bits, so k c0 and k c1 are exact for |k| < 2^13
  constexpr float c0 = 0.010833740234375f, c1 = -3.3155083656311035e-06f, c2 = -2.976022343684012e-11f;
  float rh = fmaf(-k, c0, dh);          // exact: dh and k c0 are close
  const float q = -k * c1;
  const float s = rh + q;
  float rl = (rh - (s - (s - rh))) + (q - (s - rh));
  rh = s;
  rl += dl - k * c2;
  const int j = (int)k;
  const float2 T = t.power[j & 63];
  const float lo = rl + rh * rh * fmaf(rh, fmaf(rh, 1.f / 24.f, 1.f / 6.f), 0.5f);
  const float h = T.x * rh, e = fmaf(T.x, rh, -h);
  const float sh = T.x + h;
  const float sl = (h - (sh - T.x)) + (e + (T.y + (T.x * lo + T.y * rh)));
  if (!(d > -80.f)) return make_float2(0.f, 0.f);  // below 2^-115
  const float scale = __uint_as_float((uint32_t)((j >> 6) + 127) << 23);
  return make_float2(sh * scale, sl * scale);
}

// Logits of a thread that are loaded and worked on at a time (all four beams of 32000:
// 56 us; 60 with 8, 69 with 4).
constexpr int kAhead = 16;
template <typename T>
__device__ double precise_sum(const SelectParams &p, int b, float m, const Precise &t, double *wsum) {
  const T *row = (const T *)p.logits + b * p.stride;
  float sh = 0.f, sl = 0.f;
  for (int v0 = threadIdx.x; v0 < p.V; v0 += kAhead * kThr) {
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = v0 + u * kThr < p.V ? elem_f32<T>(row, v0 + u * kThr) : -INFINITY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float2 y = exp2f2(t, x[u], m);
      const float a = sh + y.x, bb = a - sh;
      sl += ((sh - (a - bb)) + (y.x - bb)) + y.y;
      sh = a;
    }
  }
  double s = (double)sh + (double)sl;
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) wsum[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kWarps; ++w) s += wsum[w];
  return s;
}

// ---- the beams against one another -------------------------------------------------
// fp64 is slow here (a warp's instruction takes 16 cycles of an SM), so
// scores are compared as whole numbers, and the candidates that come into
// question are found by their scores in fp32, less what those may be off by.
__device__ __forceinline__ unsigned long long ordered(double s) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(s + 0.0);  // -0 and 0 are one score
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double of_ordered(unsigned long long u) {
  return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}
// A candidate: its score, ordered, and its place (beam << 20 | token).
struct Pick {
  unsigned long long s;
  uint32_t at;
  __device__ int beam() const { return (int)(at >> 20); }
  __device__ int token() const { return (int)(at & (kMaxVocab - 1)); }
};
static_assert(kMaxVocab == 1 << 20 && kMaxBeams <= 1 << 11, "a place in 32 bits");
// x before y
__device__ __forceinline__ bool before(const Pick &x, const Pick &y) { return x.s > y.s || (x.s == y.s && x.at < y.at); }

// A load that is issued where it stands (the compiler moves others to their use).
__device__ __forceinline__ float2 load_now(const float2 *at) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(at) : "memory");
  return v;
}

constexpr int kHeld = 2048;  // keys of a group that are held

struct PickShared {
  double base[kMaxBeams];                   // c - L + its largest logit; of a finished beam c
  float base_f[kMaxBeams], top[kMaxBeams];  // base in fp32; its largest logit
  float2 sum[kMaxBeams];                    // L, as a power of two and the rest
  float score[kMaxBeams];                   // c
  int kind[kMaxBeams];                      // 0: no candidates, 1: its tokens, 2: finished
  float wmax[kWarps][32];
  __align__(16) float gmax[32];
  double wsum[kWarps];
  Pick room[kRoom];
  __align__(16) unsigned long long keys[kHeld + 2];  // the group's, from the 16-byte boundary before them
  Pick best[kMaxPicks], wbest[kWarps];
  uint16_t sorted[kRoom];                   // places in `room`, best first
  Precise precise;
  float nth;
  int count, open;                          // candidates in `room`; beams whose L is not known well enough
};

// The choice of a group; its pieces were written by other CTAs too.
template <typename T>
__device__ __forceinline__ void pick(const SelectParams &p, PickShared &sm, int group) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, first = group * p.n;
  uint32_t status = 0;
  // The group's keys lie end to end.  They are on their way before anything else is
  // waited for, past L1, which may hold what they were when a neighbour was read.
  const int per_beam = p.n_out * p.segs, n_keys = p.n * per_beam;
  const unsigned long long *keys = p.keys + (int64_t)first * per_beam;
  const int odd = (int)((uintptr_t)keys >> 3 & 1);
  for (int i = 2 * tid - odd; i < min(n_keys, kHeld); i += 2 * kThr)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(sm.keys + odd + i)), "l"(keys + i) : "memory");
  for (int j = warp; j < p.n; j += kWarps) {
    const float2 *ml = p.ml + (int64_t)(first + j) * p.segs;
    // whatever it is worth: no wait for the score
    const float2 mine = lane < p.segs ? load_now(ml + lane) : make_float2(-INFINITY, 0.f);
    const float c = p.scores[first + j];
    int what = goes_on(p, first + j) ? 1 : 0;
    if (!what && c == c && c < INFINITY && c > -INFINITY) what = 2;
    else if (!what && c != -INFINITY) status |= MAC_DEV_NONFINITE_LOGIT;
    float m = -INFINITY, log2 = 0.f, rest = 0.f;  // L = (log2 + rest) ln 2
    if (what == 1) {
      m = mine.x;
      for (int i = lane + 32; i < p.segs; i += 32) m = fmaxf(m, __ldcg(ml + i).x);
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      // an empty piece has sum 0, or NaN
      auto share = [&](float2 x) { return x.x == -INFINITY ? x.y : x.y * ex2((x.x - m) * kLog2e); };
      float sum = share(mine);
      for (int i = lane + 32; i < p.segs; i += 32) sum += share(__ldcg(ml + i));
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (!(sum < 1e30f) || m == INFINITY) {  // NaN or +inf among the logits
        what = 0;
        status |= MAC_DEV_NONFINITE_LOGIT;
      } else if (m == -INFINITY) {
        what = 0;
      } else {  // 1 <= sum <= 2^20
        const int e = (int)(__float_as_uint(sum) >> 23) - 127;
        log2 = (float)e;
        rest = lg2_approx(sum * __uint_as_float((uint32_t)(127 - e) << 23));
      }
    }
    if (lane == 0) {
      sm.kind[j] = what;
      sm.sum[j] = make_float2(log2, rest);
      sm.score[j] = c;
      sm.base_f[j] = c - (log2 + rest) * 0.69314718f;
      sm.top[j] = m;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // f(beam, key) of this thread's candidates; a finished beam's key is that of its
  // end.  Lanes are turned by 5 with every 32 keys, so that neither the best of all
  // pieces nor all of one piece meet in few of them.  (A loop that is not unrolled:
  // what a choice waits for is code that has not been fetched yet.)
  auto candidates = [&](auto f) {
#pragma unroll 1
    for (int i = tid; (i & ~31) < n_keys; i += kThr) {
      const int at = (i & ~31) | ((i + 5 * (i >> 5)) & 31);
      if (at >= n_keys) continue;
      const unsigned long long k = at < kHeld ? sm.keys[odd + at] : __ldcg(keys + at);
      const int beam = (int)((unsigned long long)at * p.beam_inv >> 40);
      if (k != 0 && sm.kind[beam] == 1) f(beam, k);
    }
    if (tid < p.n && sm.kind[tid] == 2) f(tid, 1ull);
  };
  auto rough = [&](int beam, unsigned long long k) { return sm.kind[beam] == 2 ? sm.base_f[beam] : sm.base_f[beam] + (value_of(k) - sm.top[beam]); };
  auto exactly = [&](int beam, unsigned long long k) {
    Pick x;
    const bool end = sm.kind[beam] == 2;
    x.s = ordered(end ? sm.base[beam] : sm.base[beam] + ((double)value_of(k) - (double)sm.top[beam]));
    x.at = (uint32_t)beam << 20 | (uint32_t)(end ? p.end : token_of(k));
    return x;
  };
  for (int pass = 0; pass < 2; ++pass) {
    if (tid == 0) sm.count = sm.open = 0;
    __syncthreads();
    // a lower bound of the n_out-th best, from the maxima of 32 groups of threads, those of a lane
    float g = -INFINITY;
    candidates([&](int beam, unsigned long long k) { g = fmaxf(g, rough(beam, k)); });
    sm.wmax[warp][lane] = g;
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kWarps; ++w) g = fmaxf(g, sm.wmax[w][lane]);
      sm.gmax[lane] = g;
    } else if (warp == 1 && pass == 0 && lane < p.n) {
      sm.base[lane] = (double)sm.score[lane] - ((double)sm.sum[lane].x + (double)sm.sum[lane].y) * 0.6931471805599453;
    }
    __syncthreads();
    find_nth(sm.gmax, p.n_out, &sm.nth);
    float widest = 0.f;
    for (int j = 0; j < p.n; ++j)
      if (sm.kind[j]) widest = fmaxf(widest, fabsf(sm.base_f[j]));
    __syncthreads();
    // rough scores are off by 2^-24 of the base, of the difference and of the sum, 2^-22 (|base| + |s|)
    // in all, and by L's product and sum in fp32, less than kSlack / 2; twice
    const float least = sm.nth == -INFINITY ? sm.nth : sm.nth - (4.f * (float)kSlack + (widest + fabsf(sm.nth)) * (1.f / (1 << 20)));
    candidates([&](int beam, unsigned long long k) {
      if (rough(beam, k) >= least) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kRoom) sm.room[at] = exactly(beam, k);
      }
    });
    __syncthreads();
    const int c = sm.count;
    if (c <= kRoom) {
      rank_all(c, [&](int i, int j) { return before(sm.room[j], sm.room[i]); }, [&](int i, int rank) {
        sm.sorted[rank] = (uint16_t)i;
        if (rank < p.n_out) sm.best[rank] = sm.room[i];
      });
      __syncthreads();
      if (pass == 1) break;
      // Neighbours of two beams whose order is open, down to where no candidate that counts is in question
      for (int i = tid; i + 1 < c; i += kThr) {
        const Pick x = sm.room[sm.sorted[i]], y = sm.room[sm.sorted[i + 1]];
        if (x.beam() == y.beam() || (sm.kind[x.beam()] == 2 && sm.kind[y.beam()] == 2)) continue;
        const double s = of_ordered(x.s);
        if (s - of_ordered(y.s) <= 2 * kSlack && (i < p.n_out || of_ordered(sm.best[p.n_out - 1].s) - s <= 2 * kSlack))
          atomicOr(&sm.open, 1 << x.beam() | 1 << y.beam());
      }
      __syncthreads();
      if (sm.open == 0) break;
    } else if (pass == 0) {
      if (tid == 0) sm.open = (1 << p.n) - 1;
      __syncthreads();
    } else {  // too many of one score: one at a time
      for (int r = 0; r < p.n_out; ++r) {
        Pick x = {0, ~0u};
        candidates([&](int beam, unsigned long long k) {
          const Pick y = exactly(beam, k);
          if (before(y, x) && (r == 0 || before(sm.best[r - 1], y))) x = y;
        });
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          Pick y;
          y.s = __shfl_xor_sync(0xffffffffu, x.s, d);
          y.at = __shfl_xor_sync(0xffffffffu, x.at, d);
          if (before(y, x)) x = y;
        }
        if (lane == 0) sm.wbest[warp] = x;
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kWarps; ++w)
            if (before(sm.wbest[w], x)) x = sm.wbest[w];
          sm.best[r] = x;
        }
        __syncthreads();
      }
      break;
    }
    // the open beams' sums again
    if (tid < 64) {
      int k = tid;
      asm volatile("" : "+r"(k));  // here, not ahead of the loop: in fp64 it takes 1.5 us
      const double v = exp2((double)k / 64);
      const float hi = (float)v;
      sm.precise.power[tid] = make_float2(hi, (float)(v - (double)hi));
    }
    const int redo = sm.open;
    __syncthreads();
    for (int j = 0; j < p.n; ++j) {
      if (!(redo >> j & 1) || sm.kind[j] != 1) continue;
      const double sum = precise_sum<T>(p, first + j, sm.top[j], sm.precise, sm.wsum);
      if (tid == 0) {
        sm.base[j] = (double)p.scores[first + j] - log(sum);
        sm.base_f[j] = (float)sm.base[j];
      }
    }
    __syncthreads();
  }
  const int found = min(sm.count, p.n_out);
  if (status && lane == 0) set_status(p.status, status);
  if (warp > 0) return;
  // results: lane i has the i-th best
  float score = -INFINITY;
  int beam = -1, token = -1;
  if (lane < found) {
    const Pick x = sm.best[lane];
    score = (float)of_ordered(x.s);
    beam = x.beam();
    token = x.token();
  }
  const int over = lane >= found || token == p.end || sm.kind[max(beam, 0)] == 2;
  int at = lane;
  if (p.placed) {  // the best child of a surviving parent goes to the parent's slot, the others fill up in order
    bool eldest = lane < found;
    for (int i = 0; i < p.n; ++i) {
      const int o = __shfl_sync(0xffffffffu, beam, i);
      if (i < lane && o == beam) eldest = false;
    }
    const uint32_t taken = __reduce_or_sync(0xffffffffu, eldest ? 1u << beam : 0u);
    const uint32_t rest = __ballot_sync(0xffffffffu, !eldest && lane < p.n);
    int k = __popc(rest & ((1u << lane) - 1));
    if (eldest) at = beam;
    else
      for (at = 0; at < 31; ++at)
        if (!(taken >> at & 1) && k-- == 0) break;
  }
  if (lane < p.n_out) {
    const int64_t o = (int64_t)group * p.n_out + at;
    p.scores_out[o] = score;
    p.parent[o] = beam;
    p.token[o] = token;
    if (p.done_out) p.done_out[o] = over;
  }
}

template <typename T, int U>
__global__ void __launch_bounds__(kThr, 4) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ union Shared {
    ScanShared scan;
    PickShared pick;
    __device__ Shared() {}
  } sm;
  __shared__ bool last;
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.y, group = b / p.n;
  if (goes_on(p, b)) scan_piece<T, U>(p, sm.scan, blockIdx.x, b);
  // Whoever is the last of a group's CTAs chooses.  What a CTA wrote ahead of the
  // barrier that thread 0 has come through is seen by whoever finds it counted.
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.counts + group) : "memory");
    last = before + 1 == (uint32_t)p.n * gridDim.x;
    if (last) p.counts[group] = 0;  // for the next call
  }
  __syncthreads();
  if (last) pick<T>(p, sm.pick, group);
}

template <typename T>
cudaError_t launch(const SelectParams &p, cudaStream_t s) {
  const dim3 grid(p.segs, p.S);
  return p.steps == 1 ? launch_dependent(select_kernel<T, 1>, grid, kThr, 0, s, p) : launch_dependent(select_kernel<T, 4>, grid, kThr, 0, s, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams &p, int dtype, cudaStream_t s) {
  return dtype == MAC_F32 ? launch<float>(p, s) : launch<uint16_t>(p, s);
}

}  // namespace mac
