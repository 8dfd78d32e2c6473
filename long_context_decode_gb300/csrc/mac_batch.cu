// mac_batch.cu -- what a batch of new tokens needs before it is attended:
// the pages, rows and slots of its tokens (tables_kernel), and its rotated
// keys and its values in the cache (write_kernel).
#include "mac_batch.cuh"

namespace mac {

// ---------------------------------------------------------------------------
// page tables, rows and slots
// ---------------------------------------------------------------------------
// One cluster.  Every CTA loads the B <= 1024 requests (one per thread) and
// scans them itself, so the requests' pages, rows and places in the stack of
// free pages are in its shared memory after two block scans; then pages,
// flattened over the requests, are dealt to all threads of the cluster
// (a binary search over the B + 1 starts finds an item's request).  The
// cluster barrier orders what the arguments may alias and what depends on
// the stack: inputs are read before any output is written, and pages given
// back are on the stack before any page is taken.
// Rows: in a single CTA (up to kOneCta rows) a thread finds each row's page
// for itself (16 requests of one token: 3.3 us).  In the cluster they go a
// page's worth at a time: a lane finds its page (the search, the load of the
// id), then the warp writes the rows of its 32 pages, two pages at once.  A
// search per row, 100 instructions, made 104K rows of 128 requests take 18.3
// us on the cluster's eight SMs; this way the call takes 10 to 12 (and the 16 requests 4.4).
// Pages given back are dealt like pages taken, so with few rows it is a single
// CTA's threads that search, load and store them: 7 of 16 requests of up to
// 131072 tokens reset (33K pages) take 52 us, 31 of 128 of up to 65536 (62K
// pages) 121 us, where the calls without resets take 3.3 and 3.9.
constexpr int kTablesCluster = 8, kOneCta = 1024;

__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();  // aligned: the warp arrives as one
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive scans of three values over the block's threads (all call it; whole
// warps, two at least); `tot` holds one entry per warp.
__device__ __forceinline__ void block_scan3(long long v[3], long long (*tot)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, v[i], d);
      if (lane >= d) v[i] += o;
    }
  __syncthreads();  // the last scan's totals have been read
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) tot[warp][i] = v[i];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      long long t = lane < n_warps ? tot[lane][i] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += o;
      }
      if (lane < n_warps) tot[lane][i] = t;
    }
  }
  __syncthreads();
  if (warp > 0)
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += tot[warp - 1][i];
}

// The request whose [start[b], start[b+1]) holds x (start[0] <= x < start[B]).
template <typename N>
__device__ __forceinline__ int request_of(const N *start, int B, N x) {
  int lo = 0, hi = B;  // start[lo] <= x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

struct TablesShared {
  int row[kMaxUnits + 1];          // first row of request b
  int base[kMaxUnits];             // tokens it holds before the new ones
  int take[kMaxUnits + 1];         // new pages asked for before it
  int give[kMaxUnits + 1];         // pages given back before it
  int block[kMaxUnits + 1];        // pages that new tokens before its own lie on
  long long tot[32][3];
};

__global__ void __launch_bounds__(1024) tables_kernel(const __grid_constant__ TablesParams p) {
  __shared__ TablesShared sm;
  griddep_launch_dependents();
  griddep_wait();
  const int b = threadIdx.x;
  const bool has = b < p.B;
  uint32_t status = 0;

  const int n_ctas = gridDim.x, stride = n_ctas * blockDim.x;
  const int first = blockIdx.x * blockDim.x + threadIdx.x;

  // the request's demand
  long long len = 0, add = 0;
  bool flag = false;
  if (has) {
    len = p.len_in[b];
    add = p.new_len[b];
    flag = p.flags && p.flags[b] != 0;
  }
  long long n_free = 0;
  if (p.paged) {
    n_free = *p.n_free_in;
    if (n_free < 0 || n_free > p.n_pages) {
      status |= MAC_DEV_BAD_PAGE;
      n_free = n_free < 0 ? 0 : p.n_pages;
    }
  }
  const bool len_ok = len >= 0 && len <= p.limit;
  const long long base = flag && len_ok ? 0 : len;
  const bool ok = len_ok && add >= 0 && base + add <= p.limit;
  if (has && !ok) status |= MAC_DEV_BAD_SEQ_LEN;
  const long long have = (base + kPage - 1) / kPage;
  const long long want = has && ok && add > 0 ? add : 0;
  const long long need = p.paged && want ? (base + add + kPage - 1) / kPage - have : 0;
  const long long back = p.paged && has && flag && len_ok ? (len + kPage - 1) / kPage : 0;

  long long v[3] = {want, need, back};
  block_scan3(v, sm.tot);
  if (has) sm.give[b] = (int)min(v[2] - back, (long long)p.n_pages);
  if (b == p.B - 1) sm.give[p.B] = (int)min(v[2], (long long)p.n_pages);
  __syncthreads();
  long long n_back = sm.give[p.B];
  if (p.paged && n_free + n_back > p.n_pages) {  // more given back than the pool has
    status |= MAC_DEV_BAD_PAGE;
    n_back = p.n_pages - n_free;
  }
  const long long n_avail = n_free + n_back;
  const bool in = want > 0 && v[0] <= p.T && (need == 0 || v[1] <= n_avail);
  if (want > 0 && !in) status |= MAC_DEV_NO_ROOM;
  long long w[3] = {in ? want : 0, in ? need : 0, in ? (base + want - 1) / kPage - base / kPage + 1 : 0};
  const long long rows = w[0], pages = w[1], blocks = w[2];
  block_scan3(w, sm.tot);
  if (has) {
    sm.row[b] = (int)(w[0] - rows);
    sm.take[b] = (int)(w[1] - pages);
    sm.block[b] = (int)(w[2] - blocks);
    sm.base[b] = (int)base;
    if (b == p.B - 1) {
      sm.row[p.B] = (int)w[0];
      sm.take[p.B] = (int)w[1];
      sm.block[p.B] = (int)w[2];
    }
  }
  __syncthreads();

  // pages of reset requests go back on the stack
  for (long long x = first; x < n_back; x += stride) {
    const int r = request_of(sm.give, p.B, (int)x);
    const int32_t id = p.table[(int64_t)r * p.max_pages + (x - sm.give[r])];
    if (id < 0 || id >= p.n_pages) status |= MAC_DEV_BAD_PAGE;
    p.free_pages[n_free + x] = id;
  }
  cluster_sync_all();

  if (blockIdx.x == 0) {
    if (has) {
      p.len_out[b] = (int32_t)(in ? base + add : base);
      p.q_start[b] = sm.row[b];
      if (b == p.B - 1) {
        p.q_start[p.B] = sm.row[p.B];
        if (p.paged) *p.n_free_out = (int32_t)(n_avail - sm.take[p.B]);
      }
    }
  }
  const int n_take = sm.take[p.B], n_rows = sm.row[p.B];
  for (int x = first; x < n_take; x += stride) {
    const int r = request_of(sm.take, p.B, x);
    int32_t id = __ldcg(p.free_pages + (n_avail - 1 - x));
    if (id < 0 || id >= p.n_pages) {
      status |= MAC_DEV_BAD_PAGE;
      id = -1;
    }
    p.table[(int64_t)r * p.max_pages + (sm.base[r] + kPage - 1) / kPage + (x - sm.take[r])] = id;
  }
  // page k of request r's tokens, or r itself for a contiguous cache: the slot of its first token
  auto first_slot = [&](int r, int k) -> long long {
    if (!p.paged) return (int64_t)r * p.capacity + (int64_t)k * kPage;
    const int held = (sm.base[r] + kPage - 1) / kPage;
    const int32_t id = k < held ? p.table[(int64_t)r * p.max_pages + k] : __ldcg(p.free_pages + (n_avail - 1 - (sm.take[r] + k - held)));
    if (id >= 0 && id < p.n_pages) return (int64_t)id * kPage;
    status |= MAC_DEV_BAD_PAGE;
    return -1;
  };
  const int n_blocks = p.T > kOneCta ? sm.block[p.B] : 0, lane = threadIdx.x & 31;
  if (p.T <= kOneCta)
    for (int t = first; t < n_rows; t += stride) {
      const int r = request_of(sm.row, p.B, t), at = sm.base[r] + (t - sm.row[r]);
      const long long s0 = first_slot(r, at / kPage);
      p.pos[t] = at + 1;
      p.slot[t] = s0 < 0 ? -1 : s0 + at % kPage;
    }
  for (int x0 = first - lane; x0 < n_blocks; x0 += stride) {
    const int x = x0 + lane;
    int lo = 0, hi = 0, shift = 0;  // positions - 1 of this page's new tokens; row of a token minus its position
    long long slot0 = -1;           // slot of the page's first token
    if (x < n_blocks) {
      const int r = request_of(sm.block, p.B, x);
      const int base = sm.base[r], k = base / kPage + (x - sm.block[r]), n = sm.row[r + 1] - sm.row[r];
      lo = max(base, k * kPage);
      hi = (int)min((long long)base + n, (long long)(k + 1) * kPage);
      shift = sm.row[r] - base;
      slot0 = first_slot(r, k);
    }
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int src = 2 * i + (lane >> 4);
      const int l = __shfl_sync(0xffffffffu, lo, src), h = __shfl_sync(0xffffffffu, hi, src);
      const int sh = __shfl_sync(0xffffffffu, shift, src);
      const long long s0 = __shfl_sync(0xffffffffu, slot0, src);
      const int at = l / kPage * kPage + (lane & 15);
      if (at >= l && at < h) {
        p.pos[at + sh] = at + 1;
        p.slot[at + sh] = s0 < 0 ? -1 : s0 + (lane & 15);
      }
    }
  }
  for (long long t = (long long)n_rows + first; t < p.T; t += stride) {
    p.pos[t] = 0;
    p.slot[t] = -1;
  }
  if (status) set_status(p.status, status);
}

cudaError_t launch_tables(const TablesParams &p, cudaStream_t s) {
  // one thread per request at least
  if (p.T <= kOneCta) return launch_dependent(tables_kernel, 1, p.B <= 256 ? 256 : (p.B + 31) / 32 * 32, 0, s, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kTablesCluster);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kTablesCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tables_kernel, p);
}

// ---------------------------------------------------------------------------
// rotated keys and values into the cache
// ---------------------------------------------------------------------------
// A CTA takes TOK rows.  First its threads work out the rows' 64 angles
// (shared by all heads of a row) and the rows' places in the cache; then a
// thread owns 2 x 16 bytes of a head, the two halves of its rotation pairs
// (j, j + 64 for half-split pairs; neighbours for interleaved ones), and
// walks the row's heads with the sines and cosines in registers.  Bound by
// HBM: every element is read and written once.
constexpr int kWriteThreads = 128;

template <typename T>
__device__ __forceinline__ uint4 pack16(const float *f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float *f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {  // rounded to nearest even
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <>
__device__ __forceinline__ uint4 pack16<uint16_t>(const float *f) {
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

template <typename T, int ROPE, int TOK>
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int PER = 16 / (int)sizeof(T);           // elements per 16 bytes
  constexpr int ITEMS = kHeadDim / (2 * PER);        // threads per head
  constexpr int LANES = kWriteThreads / (ITEMS * TOK);  // heads of a row in flight
  __shared__ float cs[TOK][kHeadDim / 2], sn[TOK][kHeadDim / 2];
  __shared__ int64_t place[TOK], step[TOK];          // element of head 0's row in the cache (-1: skip), and between heads
  const int t0 = blockIdx.x * TOK;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < TOK) {
    const int t = t0 + threadIdx.x;
    int64_t at = -1, st = 0;
    if (t < p.T) {
      const int64_t slot = p.slot[t];
      if (slot >= p.n_slots) set_status(p.status, MAC_DEV_BAD_PAGE);
      else if (slot >= 0 && p.pos[t] < 1) set_status(p.status, MAC_DEV_BAD_SEQ_LEN);
      else if (slot >= 0) {
        const int64_t unit = p.paged ? kPage : p.capacity;
        const int64_t blk = p.paged ? slot / kPage : slot / p.capacity;
        at = (blk * p.Hkv * unit + (slot - blk * unit)) * kHeadDim;
        st = unit * kHeadDim;
      }
    }
    place[threadIdx.x] = at;
    step[threadIdx.x] = st;
  }
  if (ROPE != MAC_ROPE_NONE) {
    for (int i = threadIdx.x; i < TOK * (kHeadDim / 2); i += kWriteThreads) {
      const int t = t0 + i / (kHeadDim / 2), j = i % (kHeadDim / 2);
      const int64_t pos = t < p.T ? p.pos[t] : 1;
      // the angle's fraction of a turn, exact modulo 2^64 (see rope_angle);
      // sincospif is good to fp32, which the rows' many heads pay for once
      const unsigned long long turn = (unsigned long long)(pos - 1) * p.rope_f[j];
      sincospif((float)(long long)turn * 1.0842021724855044e-19f, &sn[i / (kHeadDim / 2)][j], &cs[i / (kHeadDim / 2)][j]);  // 2^-63
    }
  }
  __syncthreads();
  const int tok = threadIdx.x / (ITEMS * LANES), lane = threadIdx.x / ITEMS % LANES, item = threadIdx.x % ITEMS;
  const int64_t at = place[tok];
  if (at < 0) return;
  const int64_t t = t0 + tok;
  float c[PER], s[PER];
  if (ROPE != MAC_ROPE_NONE) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = cs[tok][item * PER + i];
      s[i] = sn[tok][item * PER + i];
    }
  }
  // 16-byte chunks of this thread within a head
  const int c0 = ROPE == MAC_ROPE_INTERLEAVED ? 2 * item : item;
  const int c1 = ROPE == MAC_ROPE_INTERLEAVED ? 2 * item + 1 : item + ITEMS;
  const int n_q = p.q ? p.Hq : 0, n = n_q + 2 * p.Hkv;
  for (int h0 = lane; h0 < n; h0 += 4 * LANES) {
    uint4 x0[4], x1[4];
    uint4 *to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int h = h0 + u * LANES;
      to[u] = nullptr;
      if (h < n) {
        const T *src;
        T *dst;
        if (h < n_q) {
          src = (const T *)p.q + t * p.q_stride + h * kHeadDim;
          dst = (T *)p.q_out + (t * p.Hq + h) * kHeadDim;
        } else if (h < n_q + p.Hkv) {
          src = (const T *)p.k + t * p.k_stride + (h - n_q) * kHeadDim;
          dst = (T *)p.cache_k + at + (h - n_q) * step[tok];
        } else {
          src = (const T *)p.v + t * p.v_stride + (h - n_q - p.Hkv) * kHeadDim;
          dst = (T *)p.cache_v + at + (h - n_q - p.Hkv) * step[tok];
        }
        to[u] = reinterpret_cast<uint4 *>(dst);
        x0[u] = reinterpret_cast<const uint4 *>(src)[c0];
        x1[u] = reinterpret_cast<const uint4 *>(src)[c1];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!to[u]) continue;
      if (ROPE != MAC_ROPE_NONE && h0 + u * LANES < n_q + p.Hkv) {
        float f[2 * PER], g[2 * PER];
        unpack16<T>(x0[u], f);
        unpack16<T>(x1[u], f + PER);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int ia = ROPE == MAC_ROPE_INTERLEAVED ? 2 * i : i, ib = ROPE == MAC_ROPE_INTERLEAVED ? 2 * i + 1 : PER + i;
          g[ia] = f[ia] * c[i] - f[ib] * s[i];
          g[ib] = f[ib] * c[i] + f[ia] * s[i];
        }
        x0[u] = pack16<T>(g);
        x1[u] = pack16<T>(g + PER);
      }
      to[u][c0] = x0[u];
      to[u][c1] = x1[u];
    }
  }
}

template <typename T, int TOK>
static cudaError_t launch_write_t(const WriteParams &p, cudaStream_t s) {
  const int grid = (p.T + TOK - 1) / TOK;
  if (p.rope_mode == MAC_ROPE_HALF) return launch_dependent(write_kernel<T, MAC_ROPE_HALF, TOK>, grid, kWriteThreads, 0, s, p);
  if (p.rope_mode == MAC_ROPE_INTERLEAVED) return launch_dependent(write_kernel<T, MAC_ROPE_INTERLEAVED, TOK>, grid, kWriteThreads, 0, s, p);
  return launch_dependent(write_kernel<T, MAC_ROPE_NONE, TOK>, grid, kWriteThreads, 0, s, p);
}

cudaError_t launch_write(const WriteParams &p, int dtype, cudaStream_t s) {
  // Eight heads of a row in flight: two bf16 rows per CTA, one fp32 row.
  // 8679 rows of 32 + 2 x 8 bf16 heads: 34.8 us (6.1 TB/s); with four rows of
  // 256 threads 36.4, two rows of 256 threads 39.5, one row of 256 threads 53.
  // 2160 rows of 32 + 2 x 4 fp32 heads: 15.9 us; two rows per CTA 17.0.
  // Fewer bf16 rows take a CTA each, whatever their heads, as the number of
  // CTAs in flight decides (us, one and two rows per CTA): 32 + 2 x 8 heads, 600
  // rows 4.1 and 5.7, 1200 5.7 and 6.4, 1800 6.8 and 6.5; 8 + 2 x 2 heads, 600
  // rows 2.9 and 3.4, 1200 3.9 and 3.8, 1800 4.4 and 3.8; 1 + 2 heads, 600 rows
  // 2.4 and 2.7, 1800 3.9 and 2.9.  Many rows of few heads are bound by the CTAs
  // too: 8000 rows of 8 + 2 x 2 bf16 heads take 10.1 us (four rows per CTA 8.1;
  // 32 + 2 x 8 heads 31.8 and 32.1), of fp32 heads 16.8 (13.1 and 12.8; 59, 60.6 and 62.5).
  if (dtype == MAC_F32) return launch_write_t<float, 1>(p, s);
  return p.T <= 2048 ? launch_write_t<uint16_t, 1>(p, s) : launch_write_t<uint16_t, 2>(p, s);
}

}  // namespace mac
