// mac_beam_select.cu -- beam search's selection over beams and vocabulary.
//
// For the beams j of a group, with their scores c_j and logits x_jv:
//   L_j = ln sum_v exp x_jv;   s_jv = c_j + x_jv - L_j;
// the n_out largest s of the group, ties to the lowest (j, v).
//
// scan_kernel reads every logit once: a CTA holds a piece of a row in
// registers, so the piece's maximum, its sum of exponentials and its best
// logits come from one trip to memory.  Within a row the order of s is that
// of x, so a piece's n_out best by (x, lowest v) are all that can be chosen of
// it.  They are found by a threshold: the n_out-th largest of the maxima of
// 32 groups of threads is a lower bound that few logits pass; those are
// ranked by counting.  pick_kernel, a CTA per group, joins the pieces and
// ranks the beams' candidates against one another.
//
// Across beams the order depends on L.  The sums are in fp32, so L is known to
// kSlack only; where that leaves the order of a candidate that counts open
// (two beams' scores within twice that: once in some thousand groups), the
// beams in question are summed again to 2^-38 and the candidates ranked anew.
// So the choice is that of the exact scores, however the card adds.
#include <math.h>

#include "mac_beam.cuh"

namespace mac {
namespace {

constexpr int kThr = kScanThreads, kWarps = kThr / 32, kGroups8 = kThr / 8;
static_assert(kGroups8 == 32 && kMaxPicks <= kGroups8, "a lane holds a group's maximum; the threshold is one of them");
constexpr int kRoom = 1024;  // candidates that are ranked at once
// Bound of the error of L.  An exponent t = (x - m) log2 e is off by 3 2^-24 |t|
// (the difference, the product, the constant), and the mean of (m - x) under the
// softmax is at most ln V <= 13.9: 2.5e-6 of the sum.  ex2 adds 2^-22, twice; a
// thread's sum 10 2^-24, a CTA's 8 2^-24, the logarithm 2^-23: 4.2e-6 in all.
constexpr double kSlack = 1.0 / (1 << 17);
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

// The n-th largest of the lanes' values (1 <= n <= 32).
template <typename F>
__device__ __forceinline__ F nth_largest(F g, int n) {
  const int lane = threadIdx.x & 31;
  int above = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const F o = __shfl_sync(0xffffffffu, g, j);
    above += o > g || (o == g && j < lane);
  }
  return __shfl_sync(0xffffffffu, g, __ffs(__ballot_sync(0xffffffffu, above == n - 1)) - 1);
}

// Whether a beam has next tokens at all: not finished, with a finite score.
__device__ __forceinline__ bool goes_on(const SelectParams &p, int b) {
  const float c = p.scores[b];
  return !(p.done && p.done[b] != 0) && c > -INFINITY && c < INFINITY;
}

template <typename T, int PER>
__global__ void __launch_bounds__(kThr) scan_kernel(const __grid_constant__ SelectParams p) {
  constexpr int VEC = 16 / (int)sizeof(T), NV = PER / VEC;
  __shared__ float gmax[kGroups8], wsum[kWarps];
  __shared__ unsigned long long room[kRoom];
  __shared__ unsigned long long wbest[kWarps];
  __shared__ int count;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seg = blockIdx.x, b = blockIdx.y;
  if (!goes_on(p, b)) return;
  const T *row = (const T *)p.logits + b * p.stride;
  // pieces start on 16-byte boundaries: the row starts `shift` elements behind one
  const int shift = (int)(((uintptr_t)row & 15) / sizeof(T));
  const int v0 = seg * (kThr * PER) + tid * VEC - shift;
  uint4 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * kThr * VEC;
    constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
    raw[i] = make_uint4(kNone, kNone, kNone, kNone);
    if (v >= 0 && v + VEC <= p.V) {
      raw[i] = __ldcs(reinterpret_cast<const uint4 *>(row + v));
    } else if (v < p.V && v + VEC > 0) {  // the row's ends
      uint32_t *w = &raw[i].x;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (v + e >= 0 && v + e < p.V) {
          if (sizeof(T) == 4) w[e] = reinterpret_cast<const uint32_t *>(row)[v + e];
          else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (uint32_t)row[v + e] << 16 : (w[e / 2] & 0xffff0000u) | (uint32_t)row[v + e];
        }
    }
  }
  if (tid == 0) count = 0;
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[VEC];
    unpack16<T>(raw[i], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) mx = fmaxf(mx, f[e]);
  }
  float g = mx;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  if ((lane & 7) == 0) gmax[tid >> 3] = g;
  __syncthreads();
  g = gmax[lane];
  const float least = nth_largest(g, p.n_out);
#pragma unroll
  for (int d = 16; d; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  const float m = g, ref = m == -INFINITY ? 0.f : m;
  // the sum; NaN and +inf make it NaN
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[VEC];
    unpack16<T>(raw[i], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e & 3] += ex2((f[e] - ref) * kLog2e);
  }
  float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) wsum[warp] = s;
  if (mx >= least && mx > -INFINITY) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[VEC];
      unpack16<T>(raw[i], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (f[e] >= least && f[e] > -INFINITY) {
          const int at = atomicAdd(&count, 1);
          if (at < kRoom) room[at] = key_of(f[e], v0 + i * kThr * VEC + e);
        }
    }
  }
  __syncthreads();
  const int c = count;
  const int64_t piece = (int64_t)b * p.segs + seg;
  unsigned long long *out = p.keys + piece * p.n_out;
  if (tid == 0) {
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += wsum[w];
    p.ml[piece] = make_float2(m, all);
  }
  if (c <= kRoom) {
    for (int i = tid; i < c; i += kThr) {
      const unsigned long long k = room[i];
      int rank = 0;
      for (int j = 0; j < c; ++j) rank += room[j] > k;
      if (rank < p.n_out) out[rank] = k;
    }
    for (int i = c + tid; i < p.n_out; i += kThr) out[i] = 0;
    return;
  }
  // more logits of one value than there is room for: one at a time, the best below the last
  unsigned long long last = ~0ull;
  for (int r = 0; r < p.n_out; ++r) {
    unsigned long long best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[VEC];
      unpack16<T>(raw[i], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (f[e] > -INFINITY) {
          const unsigned long long k = key_of(f[e], v0 + i * kThr * VEC + e);
          if (k < last && k > best) best = k;
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
    __syncthreads();  // the last round's have been read
    if (lane == 0) wbest[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = max(best, wbest[w]);
    if (tid == 0) out[r] = best;
    last = best;
  }
}

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
  float dh = x - m;
  const float bb = dh - x;
  const float dl = (x - (dh - bb)) + (-m - bb);  // x - m = dh + dl exactly
  if (!(dh > -80.f)) return make_float2(0.f, 0.f);  // below 2^-115
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
  const float scale = __uint_as_float((uint32_t)((j >> 6) + 127) << 23);
  return make_float2(sh * scale, sl * scale);
}

template <typename T>
__device__ double precise_sum(const SelectParams &p, int b, float m, const Precise &t, double *wsum) {
  const T *row = (const T *)p.logits + b * p.stride;
  float sh = 0.f, sl = 0.f;
#pragma unroll 4
  for (int v = threadIdx.x; v < p.V; v += kThr) {
    const float2 x = exp2f2(t, elem_f32<T>(row, v), m);
    const float a = sh + x.x, bb = a - sh;
    sl += ((sh - (a - bb)) + (x.x - bb)) + x.y;
    sh = a;
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
struct Pick {
  double s;
  int beam, token;
};
// x before y
__device__ __forceinline__ bool before(const Pick &x, const Pick &y) {
  return x.s > y.s || (x.s == y.s && (x.beam < y.beam || (x.beam == y.beam && x.token < y.token)));
}

template <typename T>
__global__ void __launch_bounds__(kThr) pick_kernel(const __grid_constant__ SelectParams p) {
  __shared__ double base[kMaxBeams];      // c - L + its largest logit; of a finished beam c
  __shared__ float top[kMaxBeams];        // its largest logit
  __shared__ int kind[kMaxBeams];         // 0: no candidates, 1: its tokens, 2: finished
  __shared__ double gmax[kGroups8], wsum[kWarps];
  __shared__ Pick room[kRoom];
  __shared__ Pick best[kMaxPicks], wbest[kWarps];
  __shared__ Precise precise;
  __shared__ int count, open;             // candidates in `room`; beams whose L is not known well enough
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, first = blockIdx.x * p.n;
  uint32_t status = 0;
  for (int j = warp; j < p.n; j += kWarps) {
    const float c = p.scores[first + j];
    int what = goes_on(p, first + j) ? 1 : 0;
    if (!what && c == c && c < INFINITY && c > -INFINITY) what = 2;
    else if (!what && c != -INFINITY) status |= MAC_DEV_NONFINITE_LOGIT;
    double l = 0.0;
    float m = -INFINITY;
    if (what == 1) {
      const float2 *ml = p.ml + (int64_t)(first + j) * p.segs;
      for (int i = lane; i < p.segs; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      double sum = 0.0;
      for (int i = lane; i < p.segs; i += 32) sum += (double)ml[i].y * (double)(ml[i].x == -INFINITY ? (ml[i].y == 0.f ? 0.f : ml[i].y) : ex2((ml[i].x - m) * kLog2e));
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (!(sum < 1e30) || m == INFINITY) {  // NaN or +inf among the logits
        what = 0;
        status |= MAC_DEV_NONFINITE_LOGIT;
      } else if (m == -INFINITY) {
        what = 0;
      } else {
        const float f = (float)sum;  // 1 <= sum <= 2^20
        const int e = (int)(__float_as_uint(f) >> 23) - 127;
        l = e * 0.6931471805599453 + (double)logf(f * __uint_as_float((uint32_t)(127 - e) << 23));
      }
    }
    if (lane == 0) {
      kind[j] = what;
      base[j] = (double)c - l;
      top[j] = m;
    }
  }
  const int per_beam = p.segs * p.n_out, n_keys = p.n * per_beam;
  const unsigned long long *keys = p.keys + (int64_t)first * per_beam;
  // candidate i of the group; false: there is none
  auto candidate = [&](int i, Pick &c) {
    if (i >= n_keys) {  // a finished beam goes on as it is
      c.beam = i - n_keys;
      c.token = p.end;
      c.s = base[c.beam];
      return kind[c.beam] == 2;
    }
    c.beam = i / per_beam;
    if (kind[c.beam] != 1) return false;
    const unsigned long long k = keys[i];
    c.token = token_of(k);
    c.s = base[c.beam] + ((double)value_of(k) - (double)top[c.beam]);
    return k != 0;
  };
  for (int pass = 0; pass < 2; ++pass) {
    if (tid == 0) count = open = 0;
    __syncthreads();
    // a lower bound of the n_out-th best, from the maxima of groups of threads
    double g = -INFINITY;
    for (int i = tid; i < n_keys + p.n; i += kThr) {
      Pick c;
      if (candidate(i, c)) g = fmax(g, c.s);
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) g = fmax(g, __shfl_xor_sync(0xffffffffu, g, d));
    if ((lane & 7) == 0) gmax[tid >> 3] = g;
    __syncthreads();
    const double least = nth_largest(gmax[lane], p.n_out) - 2 * kSlack;
    for (int i = tid; i < n_keys + p.n; i += kThr) {
      Pick c;
      if (candidate(i, c) && c.s >= least) {
        const int at = atomicAdd(&count, 1);
        if (at < kRoom) room[at] = c;
      }
    }
    __syncthreads();
    const int c = count;
    if (c <= kRoom) {
      for (int i = tid; i < c; i += kThr) {
        const Pick x = room[i];
        int rank = 0, near = 0;
        for (int j = 0; j < c; ++j) {
          const Pick y = room[j];
          rank += before(y, x);
          if (y.beam != x.beam && fabs(y.s - x.s) <= 2 * kSlack && (kind[x.beam] == 1 || kind[y.beam] == 1))
            near |= 1 << x.beam | 1 << y.beam;
        }
        if (rank < p.n_out) {
          best[rank] = x;
          if (near) atomicOr(&open, near);
        }
      }
      __syncthreads();
      if (pass == 1 || open == 0) break;
    } else if (pass == 0) {
      if (tid == 0) open = (1 << p.n) - 1;
      __syncthreads();
    } else {  // too many of one score: one at a time
      for (int r = 0; r < p.n_out; ++r) {
        Pick x = {-INFINITY, kMaxBeams, 0};
        for (int i = tid; i < n_keys + p.n; i += kThr) {
          Pick y;
          if (candidate(i, y) && before(y, x) && (r == 0 || before(best[r - 1], y))) x = y;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          Pick y;
          y.s = __shfl_xor_sync(0xffffffffu, x.s, d);
          y.beam = __shfl_xor_sync(0xffffffffu, x.beam, d);
          y.token = __shfl_xor_sync(0xffffffffu, x.token, d);
          if (before(y, x)) x = y;
        }
        if (lane == 0) wbest[warp] = x;
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kWarps; ++w)
            if (before(wbest[w], x)) x = wbest[w];
          best[r] = x;
        }
        __syncthreads();
      }
      break;
    }
    // the open beams' sums again
    if (tid < 64) {
      const double v = exp2((double)tid / 64);
      const float hi = (float)v;
      precise.power[tid] = make_float2(hi, (float)(v - (double)hi));
    }
    const int redo = open;
    __syncthreads();
    for (int j = 0; j < p.n; ++j) {
      if (!(redo >> j & 1) || kind[j] != 1) continue;
      const double sum = precise_sum<T>(p, first + j, top[j], precise, wsum);
      if (tid == 0) base[j] = (double)p.scores[first + j] - log(sum);
    }
    __syncthreads();
  }
  const int found = min(count, p.n_out);
  if (status && lane == 0) set_status(p.status, status);
  if (warp > 0) return;
  // results: lane i has the i-th best
  Pick x = {-INFINITY, -1, -1};
  if (lane < found) x = best[lane];
  int over = lane >= found || x.token == p.end;
  if (lane < found && kind[x.beam] == 2) over = 1;
  int at = lane;
  if (p.placed) {  // the best child of a surviving parent goes to the parent's slot, the others fill up in order
    const bool live = lane < found;
    bool eldest = live;
    for (int i = 0; i < p.n; ++i) {
      const int o = __shfl_sync(0xffffffffu, x.beam, i);
      if (i < lane && o == x.beam) eldest = false;
    }
    const uint32_t taken = __reduce_or_sync(0xffffffffu, eldest ? 1u << x.beam : 0u);
    const uint32_t rest = __ballot_sync(0xffffffffu, !eldest && lane < p.n);
    int k = __popc(rest & ((1u << lane) - 1));
    if (eldest) at = x.beam;
    else
      for (at = 0; at < 31; ++at)
        if (!(taken >> at & 1) && k-- == 0) break;
  }
  if (lane < p.n_out) {
    const int64_t o = (int64_t)blockIdx.x * p.n_out + at;
    p.scores_out[o] = (float)x.s;
    p.parent[o] = x.beam;
    p.token[o] = x.token;
    if (p.done_out) p.done_out[o] = over;
  }
}

template <typename T>
cudaError_t launch(const SelectParams &p, cudaStream_t s) {
  const dim3 grid(p.segs, p.S);
  cudaError_t e = p.per == 32   ? launch_dependent(scan_kernel<T, 32>, grid, kThr, 0, s, p)
                  : p.per == 16 ? launch_dependent(scan_kernel<T, 16>, grid, kThr, 0, s, p)
                                : launch_dependent(scan_kernel<T, 8>, grid, kThr, 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(pick_kernel<T>, p.S / p.n, kThr, 0, s, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams &p, int dtype, cudaStream_t s) {
  return dtype == MAC_F32 ? launch<float>(p, s) : launch<uint16_t>(p, s);
}

}  // namespace mac
