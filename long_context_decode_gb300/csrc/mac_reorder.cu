// mac_reorder.cu -- slots go on from their parents' histories: page tables,
// lengths and common positions (reorder_kernel), and what a layer keeps per
// slot (state_kernel).
#include "mac_beam.cuh"

namespace mac {
namespace {

// ---------------------------------------------------------------------------
// page tables
// ---------------------------------------------------------------------------
// A column is one place of a group's page tables: n ids, those of its n slots.
// What happens to a column depends on itself alone, so a thread reads it,
// writes the children's ids over it, and counts the ids that no slot holds any
// more.  Slots that have their first positions in common have their first pages
// in common: columns before the first place where a slot that changes differs
// from its parent are not looked at.  Pages go back in order of (group, column,
// slot), for which a column needs the count of all columns before it: a CTA
// takes a run of columns, counts, and writes once it knows the others' counts.
// One cluster; where a single CTA's threads have a column each at most, or
// nothing goes back, its CTAs do not wait for one another before they write.
// Bound by its chain of trips to L2 (lengths and parents, common positions, ids,
// the stack) and the barriers between: a step of 16 groups of 4 slots takes
// 6.0 us, beams opened on 16 prompts of up to 32768 tokens (8 slots each, 120K
// table entries) 11.9, most of it the instructions of 17K columns on eight SMs.
constexpr int kKeeps = (int)0x80000000;  // no id: nothing to write
constexpr int kLeastThr = 512, kMostThr = 1024, kCluster = 8;

__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();  // aligned: the warp arrives as one
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Its halves: what this CTA has read may be written once all have come to the first.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ long long read_cta(const long long *at, int rank) {  // the same place in another CTA's shared memory
  uint32_t there;
  long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_addr(at)), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(there) : "memory");
  return v;
}

// Inclusive scan over the block's threads (all call it); *all: the sum.
template <typename N>
__device__ __forceinline__ N block_scan(N v, long long *tot, N *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const N o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the last scan's totals have been read
  if (lane == 31) tot[warp] = v;
  __syncthreads();
  N t = lane < blockDim.x >> 5 ? (N)tot[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const N o = __shfl_up_sync(0xffffffffu, t, d);
    if (lane >= d) t += o;
  }
  const N before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
  if (warp > 0) v += before;
  *all = __shfl_sync(0xffffffffu, t, 31);
  return v;
}

struct ReorderShared {
  int up[kMaxUnits];               // slot whose history a slot goes on from; -1: none
  int len[kMaxUnits];              // tokens it held
  int low[kMaxUnits];              // per group: first column that may change
  int top[kMaxUnits];              // columns held
  uint32_t kids[kMaxUnits];        // slots of the group that have children
  int bad[kMaxUnits];              // a length out of range
  uint8_t out[kMaxUnits];          // slot without a page for its part
  long long first[kMaxUnits + 1];  // columns of the groups before it
  long long tot[32];
  long long back;                  // pages given back by this CTA's columns
};

__device__ __forceinline__ int pages_of(int n) { return (int)(((long long)n + kPage - 1) / kPage); }

template <int NB>
__global__ void __launch_bounds__(kMostThr) reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ ReorderShared sm;
  griddep_launch_dependents();
  griddep_wait();
  const int t = threadIdx.x, threads = blockDim.x, n = p.n, groups = p.S / n, g_t = t / n, base_t = g_t * n;
  const bool has = t < p.S;
  const int n_ctas = gridDim.x, rank = blockIdx.x;
  uint32_t status = 0;
  long long n_free = 0;

  // who goes on from whom
  int parent = -1, len_old = 0;
  if (has) {
    len_old = p.len_in[t];
    parent = p.parent[t];
  }
  if (p.paged) {
    n_free = *p.n_free_in;
    if (n_free < 0 || n_free > p.n_pages) {
      status |= MAC_DEV_BAD_PAGE;
      n_free = n_free < 0 ? 0 : p.n_pages;
    }
  }
  if (t < groups) {
    sm.low[t] = 0x7fffffff;
    sm.top[t] = 0;
    sm.kids[t] = 0;
    sm.bad[t] = 0;
  }
  __syncthreads();
  if (has) {
    sm.len[t] = len_old;
    if (len_old < 0 || len_old > p.limit) {
      sm.bad[g_t] = 1;
      status |= MAC_DEV_BAD_SEQ_LEN;
    }
  }
  __syncthreads();
  const bool skip = has && sm.bad[g_t];  // the group is passed over
  int up = -1, common = 0;
  if (has) {
    up = base_t + parent;
    if (skip) up = t;
    else if (parent == -1) up = -1;
    else if (parent < -1 || parent >= n) {
      status |= MAC_DEV_BAD_PARENT;
      up = t;
    }
    sm.up[t] = up;
    if (up >= 0) {
      atomicOr(&sm.kids[g_t], 1u << (up - base_t));
      if (up != t) common = p.shared_in[(int64_t)t * n + up - base_t];
    }
  }
  __syncthreads();
  const int len_new = up >= 0 ? sm.len[up] : 0;
  const bool moved = has && up != t;
  bool parted = false;
  int keeper = t;  // has the last page of the history that this slot goes on from
  if (moved && up >= 0) {
    common = min(max(common, 0), min(len_new, len_old));
    keeper = up;
    if (sm.up[up] != up)
      for (keeper = base_t; sm.up[keeper] != up; ++keeper) {
      }
    parted = p.paged && len_new % kPage != 0 && keeper != t;
  }
  bool gives = false;  // some page of this slot may go back
  if (p.paged && has && !skip) {
    if (moved) atomicMin(&sm.low[g_t], common / kPage);
    atomicMax(&sm.top[g_t], pages_of(len_old));
    gives = moved && pages_of(len_old) > common / kPage;
  }
  const bool any_gives = __syncthreads_or(gives);
  {
    long long all;
    const long long cols = t < groups ? max(0, sm.top[t] - min(sm.low[t], sm.top[t])) : 0;
    const long long end = block_scan(cols, sm.tot, &all);
    if (t < groups) sm.first[t] = end - cols;
    if (t == 0) sm.first[groups] = all;
  }
  int n_parted;
  const int part_at = block_scan((int)parted, sm.tot, &n_parted) - parted;
  // (the scan's barriers stand between the writes of `first` and its use)
  const long long total = sm.first[groups];
  // Every CTA has read the arguments by now; the outputs, which may be the same
  // arrays, are written when all have.
  cluster_arrive();
  const bool alone = total <= threads;  // one CTA's threads do
  if (alone && rank != 0) return;
  if (!alone) cluster_wait();
  const long long run = alone ? total : (total + n_ctas - 1) / n_ctas;
  const long long x0 = alone ? 0 : min(total, rank * run), x1 = min(total, x0 + run);

  int got[NB], ids[NB];  // ids that a column's slots get, and that they have
  uint32_t gone = 0;   // slots whose id goes back
  int base = 0, col = 0;
  auto id_of = [&](int slot) { return p.table[(int64_t)slot * p.max_pages + col]; };
  auto column = [&](long long x) {
    int g = 0, hi = groups;
    while (hi - g > 1) {
      const int mid = (g + hi) >> 1;
      if (sm.first[mid] <= x) g = mid; else hi = mid;
    }
    base = g * n;
    col = sm.low[g] + (int)(x - sm.first[g]);
    gone = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = i < n ? sm.up[base + i] : -1;
      got[i] = u >= 0 && u != base + i && col < pages_of(sm.len[u]) ? id_of(u) : kKeeps;
    }
    if (!any_gives) return;
#pragma unroll
    for (int j = 0; j < NB; ++j) ids[j] = j < n && col < pages_of(sm.len[base + j]) ? id_of(base + j) : kKeeps;
    const uint32_t kids = sm.kids[g];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (ids[j] == kKeeps) continue;
      if (ids[j] < 0 || ids[j] >= p.n_pages) {
        status |= MAC_DEV_BAD_PAGE;
        continue;
      }
      bool stays = false;
#pragma unroll
      for (int i = 0; i < NB; ++i) stays |= ids[i] == ids[j] && (i < j || (kids >> i & 1));
      if (!stays) gone |= 1u << j;
    }
  };

  long long n_back = 0, at = 0;
  bool known = false;  // this thread's column has been read
  if (any_gives && total > 0) {
    int mine = 0;
    for (long long x = x0 + t; x < x1; x += threads) {
      column(x);
      mine += __popc(gone);
    }
    known = x1 - x0 <= threads;
    int all;
    const int end = block_scan(mine, sm.tot, &all);
    if (alone) {
      n_back = all;
    } else {
      if (t == 0) sm.back = all;
      cluster_sync_all();
      for (int r = 0; r < n_ctas; ++r) {
        const long long b = read_cta(&sm.back, r);
        if (r < rank) at += b;
        n_back += b;
      }
    }
    if (known) at += end - mine;  // of this thread's column
    if (n_free + n_back > p.n_pages) {  // more given back than the pool has
      status |= MAC_DEV_BAD_PAGE;
      n_back = p.n_pages - n_free;
    }
  }
  for (long long xb = x0; xb < x1; xb += threads) {
    const long long x = xb + t;
    if (!known) gone = 0;
    if (x < x1) {
      if (!known) column(x);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (got[i] != kKeeps) p.table[(int64_t)(base + i) * p.max_pages + col] = got[i];
    }
    if (!any_gives) continue;
    long long w = at;
    if (!known) {
      int all;
      const int k = __popc(gone), end = block_scan(k, sm.tot, &all);
      w += end - k;
      at += all;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (gone >> j & 1) {
        if (w < n_back) p.free_pages[n_free + w] = ids[j];
        ++w;
      }
  }
  // the stack and the tables are written
  if (alone) {
    __syncthreads();
    cluster_wait();
  } else {
    cluster_sync_all();
  }
  if (rank != 0) {
    if (status) set_status(p.status, status);
    return;
  }

  // lengths, common positions, moves; a page of its own for every history that parts within one
  const long long n_avail = n_free + n_back;
  const bool room = !parted || part_at < n_avail;
  if (has) sm.out[t] = !room;
  int from = -1, to = -1;
  if (parted && room) {
    from = __ldcg(p.table + (int64_t)keeper * p.max_pages + len_new / kPage);
    to = __ldcg(p.free_pages + (n_avail - 1 - part_at));
  }
  __syncthreads();
  int row[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    row[j] = 0;
    if (!has || j >= n || up < 0 || !room) continue;
    const int o = base_t + j, uo = sm.up[o];
    if (o == t) row[j] = len_new;
    else if (uo < 0 || sm.out[o]) row[j] = 0;
    else if (uo == up) row[j] = max(len_new - 1, 0);
    else row[j] = p.shared_in[(int64_t)up * n + uo - base_t];
  }
  __syncthreads();  // shared_out and len_out may be the inputs
  if (has) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (j < n) p.shared_out[(int64_t)t * n + j] = row[j];
    p.len_out[t] = room ? len_new : 0;
    Move m = {-1, 0, 0, 0, -1, -1, 0, 0};
    if (moved && up >= 0 && room) {
      m.src = up;
      m.first = common + 1;
      m.last = max(len_new, len_old);
      m.len = len_new;
      if (parted) {
        if (to < 0 || to >= p.n_pages) to = -1;
        if (to < 0 || from < 0 || from >= p.n_pages) status |= MAC_DEV_BAD_PAGE;
        m.page_from = from;
        m.page_to = to;
        m.rows = len_new % kPage;
        p.table[(int64_t)t * p.max_pages + len_new / kPage] = to;
      }
    }
    int4 *out = reinterpret_cast<int4 *>(p.moves + t);
    out[0] = make_int4(m.src, m.first, m.last, m.len);
    out[1] = make_int4(m.page_from, m.page_to, m.rows, 0);
    if (!room) status |= MAC_DEV_NO_ROOM;
  }
  if (p.paged && t == 0) *p.n_free_out = (int32_t)(n_avail - min((long long)n_parted, n_avail));
  if (status) set_status(p.status, status);
}

template <int NB>
cudaError_t launch(const ReorderParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int64_t most = p.paged ? (int64_t)(p.S / p.n) * p.max_pages : 0;  // columns
  const int threads = p.S <= kLeastThr ? kLeastThr : (p.S + 31) / 32 * 32;
  // without pages, or where the tables have no more columns than threads, there is work for one CTA
  cfg.gridDim = dim3(most <= threads ? 1 : kCluster);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, reorder_kernel<NB>, p);
}

// ---------------------------------------------------------------------------
// a layer's state
// ---------------------------------------------------------------------------
// In place, without a second copy: a thread has the same 16 bytes of all slots
// of a group (an element of a ring entry or of a cache row), reads what the
// slots' parents hold there, and then writes.  Nobody else touches them, so
// slots may change places.  A warp takes an entry of a head (its query and
// summary) or a row of a KV head (key and value).  Only positions that a slot
// does not share with its parent are moved.
// A step (32 slots, 12 positions apart at most, 32 / 8 bf16 heads, paged): 3.5 us,
// its launch and three trips to memory.  Beams opened on two prompts (8 slots of
// 8 / 2 fp32 heads, 59 MB written, 20 MB of parents' state read, by three children
// each): 14.8 us from L2, 19.6 from HBM, 1.7 times the bytes' time there.  With
// four CTAs per SM, and so 64 registers, they took 5.9 and 22.6 of 3.8 and 15.6, with
// three 4.4 and 15.6.  Groups of two slots have less on its way per thread, and room
// for four CTAs: 16 of 418 positions at most, 128 in the ring, copied whole (110 MB)
// 29.2, 48.7 with two.
constexpr int kStateThr = 256;

struct StateShared {
  int4 move[kMaxUnits];            // source (-1: none), first and last position, length
  long long rings[kMaxUnits + 1];  // ring positions of the groups before it
  long long rows[kMaxUnits + 1];   // cache rows of the groups (paged: slots) before it
  int ring_first[kMaxUnits], row_first[kMaxUnits];
  long long tot[2][kStateThr / 32];
};

// What of a slot's move can be used; *rows: rows of its parted page.
__device__ __forceinline__ int4 checked_move(const StateParams &p, int slot, int *rows, uint32_t *status) {
  const int4 *in = reinterpret_cast<const int4 *>(p.moves + slot);
  int4 m = in[0];
  const int4 page = in[1];  // from, to, rows
  *rows = 0;
  if (m.x == -1) return m;
  if (m.x < 0 || m.x >= p.S || m.x / p.n != slot / p.n) {
    *status |= MAC_DEV_BAD_PARENT;
    m.x = -1;
    return m;
  }
  const long long most = p.k && !p.paged ? p.capacity : 0x7ffffffe;
  if (m.y < 1 || m.z < 0 || m.z > 0x7ffffffe || m.w < 0 || m.w > most) {
    *status |= MAC_DEV_BAD_SEQ_LEN;
    m.x = -1;
    return m;
  }
  if (page.z > 0 && p.paged && p.k) {
    if (page.x < 0 || page.x >= p.n_pages || page.y < 0 || page.y >= p.n_pages || page.z > kPage) *status |= MAC_DEV_BAD_PAGE;
    else *rows = page.z;
  }
  return m;
}

__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 ? div_s64(a, b) : (uint32_t)a / (uint32_t)b;
}

// NB slots of a group's 16 bytes in registers; CTAS of them on an SM.
template <int NB, int CTAS>
__global__ void __launch_bounds__(kStateThr, CTAS) state_kernel(const __grid_constant__ StateParams p) {
  __shared__ StateShared sm;
  griddep_launch_dependents();
  griddep_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = p.n, groups = p.S / n;
  const bool by_slot = p.paged != 0;
  uint32_t status = 0;
  for (int s = t; s < p.S; s += kStateThr) {
    int rows;
    sm.move[s] = checked_move(p, s, &rows, &status);
    if (by_slot) sm.rows[s + 1] = rows;
  }
  if (status && blockIdx.x == 0) set_status(p.status, status);
  if (t == 0) sm.rings[0] = sm.rows[0] = 0;
  __syncthreads();
  // positions and rows of every group (paged: rows of every slot)
  for (int g0 = 0; g0 < (by_slot ? p.S : groups); g0 += kStateThr) {
    const int g = g0 + t;
    long long v[2] = {0, 0};
    if (g < groups) {
      int first = 0x7fffffff, last = 0, len = 0;
      for (int i = 0; i < n; ++i) {
        const int4 m = sm.move[g * n + i];
        if (m.x < 0) continue;
        first = min(first, m.y);
        last = max(last, m.z);
        len = max(len, m.w);
      }
      if (last >= first) {
        sm.ring_first[g] = max(first, last - p.K + 1);
        if (p.pos) v[0] = last - sm.ring_first[g] + 1;
      }
      if (!by_slot && p.k && len >= first) {
        sm.row_first[g] = first;
        v[1] = len - first + 1;
      }
    }
    if (by_slot && g < p.S) v[1] = sm.rows[g + 1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v[i], d);
        if (lane >= d) v[i] += o;
      }
      if (lane == 31) sm.tot[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      long long *to = i ? sm.rows : sm.rings;
      if (g >= (i && by_slot ? p.S : groups)) continue;
      long long before = to[g0];
      for (int w = 0; w < warp; ++w) before += sm.tot[i][w];
      to[g + 1] = before + v[i];
    }
    __syncthreads();
  }
  const long long n_rings = sm.rings[groups] * p.Hq, n_rows = sm.rows[by_slot ? p.S : groups] * p.Hkv;
  auto find = [](const long long *start, int count, long long x) {
    int lo = 0, hi = count;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  const long long step = (long long)gridDim.x * (kStateThr / 32);
  const int units = kHeadDim * p.es / 16;  // of a row: 16 (bf16, half a warp) or 32
  for (long long item = (long long)blockIdx.x * (kStateThr / 32) + warp; item < n_rings + n_rows; item += step) {
    if (item < n_rings) {
      const long long line = quotient(item, p.Hq);
      const int h = (int)(item - line * p.Hq), g = find(sm.rings, groups, line), base = g * n;
      const int pos = sm.ring_first[g] + (int)(line - sm.rings[g]), c = pos % p.K;
      // slots that take this entry, and from whom
      const int4 m = lane < n ? sm.move[base + lane] : make_int4(-1, 0, 0, 0);
      const int ahead = m.z % p.K - c, back = ahead < 0 ? ahead + p.K : ahead;  // of the slot's last position, to this entry's
      const uint32_t take = __ballot_sync(0xffffffffu, m.x >= 0 && m.z - back >= m.y);
      if (!take) continue;
      const int64_t entry = (int64_t)h * p.K + c, slots = (int64_t)p.Hq * p.K;
      uint4 o[NB], q[NB];
      uint32_t w[NB];  // lane 0: the entry's lse; lane 1, of the first head: its position
      const bool with_w = lane == 0 || (lane == 1 && h == 0);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int src = __shfl_sync(0xffffffffu, m.x, i);
        if (!(take >> i & 1)) continue;
        const int64_t e = src * slots + entry;
        o[i] = reinterpret_cast<const uint4 *>(p.o + e * kHeadDim)[lane];
        if (lane < units) q[i] = reinterpret_cast<const uint4 *>(p.q + e * kHeadDim * p.es)[lane];
        if (with_w) w[i] = lane ? (uint32_t)p.pos[(int64_t)src * p.K + c] : __float_as_uint(p.lse[e]);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (!(take >> i & 1)) continue;
        const int64_t e = (base + i) * slots + entry;
        reinterpret_cast<uint4 *>(p.o + e * kHeadDim)[lane] = o[i];
        if (lane < units) reinterpret_cast<uint4 *>(p.q + e * kHeadDim * p.es)[lane] = q[i];
        if (lane == 0) p.lse[e] = __uint_as_float(w[i]);
        else if (with_w) p.pos[(int64_t)(base + i) * p.K + c] = (int32_t)w[i];
      }
      continue;
    }
    const long long line = quotient(item - n_rings, p.Hkv);
    const int h = (int)(item - n_rings - line * p.Hkv);
    // bf16: half a warp for the key, half for the value; fp32: one after the other
    if (by_slot) {
      const int slot = find(sm.rows, p.S, line), r = (int)(line - sm.rows[slot]);
      const int4 page = reinterpret_cast<const int4 *>(p.moves + slot)[1];
      const int64_t row = (int64_t)kHeadDim * p.es;
      const int64_t from = (((int64_t)page.x * p.Hkv + h) * kPage + r) * row, to = (((int64_t)page.y * p.Hkv + h) * kPage + r) * row;
      for (int u = lane; u < 2 * units; u += 32) {
        uint8_t *cache = u < units ? p.k : p.v;
        const int at = (u & (units - 1)) * 16;
        *reinterpret_cast<uint4 *>(cache + to + at) = *reinterpret_cast<const uint4 *>(cache + from + at);
      }
      continue;
    }
    const int g = find(sm.rows, groups, line), base = g * n;
    const int pos = sm.row_first[g] + (int)(line - sm.rows[g]);
    const int4 m = lane < n ? sm.move[base + lane] : make_int4(-1, 0, 0, 0);
    const uint32_t take = __ballot_sync(0xffffffffu, m.x >= 0 && pos >= m.y && pos <= m.w);
    for (int u = lane; u < 2 * units; u += 32) {
      uint8_t *cache = u < units ? p.k : p.v;
      const int at = (u & (units - 1)) * 16;
      auto place = [&](int slot) {
        return reinterpret_cast<uint4 *>(cache + (((int64_t)slot * p.Hkv + h) * p.capacity + pos - 1) * kHeadDim * p.es + at);
      };
      uint4 x[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int src = __shfl_sync(0xffffffffu, m.x, i);
        if (take >> i & 1) x[i] = *place(src);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (take >> i & 1) *place(base + i) = x[i];
    }
  }
}

}  // namespace

cudaError_t launch_reorder(const ReorderParams &p, cudaStream_t s) {
  if (p.n <= 4) return launch<4>(p, s);
  return p.n <= 8 ? launch<8>(p, s) : launch<16>(p, s);
}

cudaError_t launch_state(const StateParams &p, int sms, cudaStream_t s) {
  if (p.n <= 2) return launch_dependent(state_kernel<2, 4>, sms * 4, kStateThr, 0, s, p);
  if (p.n <= 4) return launch_dependent(state_kernel<4, 2>, sms * 2, kStateThr, 0, s, p);
  return p.n <= 8 ? launch_dependent(state_kernel<8, 2>, sms * 2, kStateThr, 0, s, p) : launch_dependent(state_kernel<16, 1>, sms, kStateThr, 0, s, p);
}

}  // namespace mac
