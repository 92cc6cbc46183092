// Page bookkeeping of the paged caches (fork, reserve, release, compact), page copies and the
// append of new rows into pages.
//
// The state is three int32 arrays: the page table [B, max_pages], the reference counts
// [n_pages] and the sequence lengths [B].  Every result is a function of the state and the
// arguments alone (the lowest free pages are taken, in sequence order), so the kernels use
// scans where order matters and atomics only for counts, whose sums do not depend on it.
//
// Measured on a B200 (a graph of one launch between two events).  Serving-size book, 256
// or 128 sequences, 8,192 pages: fork 6.3 us, reserve 14.0, release 5.9, compact 13.9: chains of a few
// dependent reads each, so each is one launch of one block (reserve), a block per row, or one cluster
// (compact).  Page copies: 2,000 pages of 256 KB in 169 us, 0.97 of the measured copy rate; 180 in 18
// us.  Append of 25,000 rows of 8 heads 39-41 us (5.2 TB/s), of 64 rows 7.4.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"
#include "paged.cuh"

namespace cg = cooperative_groups;

namespace jssa {
namespace {

__device__ __forceinline__ int warp_inclusive_scan(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Exclusive scan over a block of 1024 threads; *total gets the sum.  `part`: 33 ints.  The
// caller must pass a barrier between two uses of `part` (both calls end with one).
__device__ __forceinline__ int block_exclusive_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inc = warp_inclusive_scan(v);
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = part[lane];
    const int s = warp_inclusive_scan(w);
    part[lane] = s - w;
    if (lane == 31) part[32] = s;
  }
  __syncthreads();
  const int r = part[warp] + inc - v;
  *total = part[32];
  __syncthreads();
  return r;
}

// Sequence length clamped to what the table row can hold.
__device__ __forceinline__ int clamp_len(int len, const PageBook& k, bool* bad) {
  const int64_t cap = static_cast<int64_t>(k.max_pages) * k.page_size;
  *bad = len < 0 || len > cap;
  return len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
}

// A table entry past its sequence's length (a sequence that gave tokens back) still counts as a holder of its page;
// before fork or reserve writes over it, the page is given up.  A page that is counted free already keeps its count, and
// the entry, which cannot be right, is cleared.
__device__ __forceinline__ void give_up(const PageBook& k, int32_t* entry, int p) {  // p: the entry's page
  if (p < 0 || p >= k.n_pages) return;
  if (atomicSub(k.ref + p, 1) <= 0) {
    atomicAdd(k.ref + p, 1);
    *entry = -1;
    flag_error(k.status, DEVFLAG_BAD_INDEX);
  }
}

// ------------------------------------------------------------------ fork
// One block per entry: validates it against the whole list, then copies the table row and
// counts its pages.  Rows that are forked to are neither read nor written by other entries.
__global__ void __launch_bounds__(256) pages_fork_kernel(PageBook k, const int32_t* src, const int32_t* dst, int n) {
  const int i = blockIdx.x;
  const int s = src[i], t = dst[i];
  if (s < 0) return;
  bool bad = s >= k.B || t < 0 || t >= k.B || s == t;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int sj = src[j], tj = dst[j];
    if (sj < 0) continue;
    bad |= (j < i && tj == t) || sj == t || tj == s;
  }
  if (!bad) bad = k.seq_lens[t] != 0;
  bad = __syncthreads_or(bad) != 0;
  if (bad) {
    if (threadIdx.x == 0) flag_error(k.status, DEVFLAG_BAD_INDEX);
    return;
  }
  bool bad_len;
  const int len = clamp_len(k.seq_lens[s], k, &bad_len);
  const int used = static_cast<int>(ceil_div(len, k.page_size));
  const int32_t* from = k.table + static_cast<int64_t>(s) * k.max_pages;
  int32_t* to = k.table + static_cast<int64_t>(t) * k.max_pages;
  bool bad_page = false;
  for (int j = threadIdx.x; j < k.max_pages; j += blockDim.x) {
    const int held = to[j];
    int p = j < used ? from[j] : -1;
    if (p >= k.n_pages) {
      bad_page = true;
      p = -1;
    }
    if (p >= 0) atomicAdd(k.ref + p, 1);
    give_up(k, to + j, held);
    to[j] = p < 0 ? -1 : p;
  }
  if (bad_page) flag_error(k.status, DEVFLAG_BAD_INDEX);
  if (threadIdx.x == 0) {
    k.seq_lens[t] = len;
    if (bad_len) flag_error(k.status, DEVFLAG_BAD_SEQ_LEN);
  }
}

// ------------------------------------------------------------------ reserve
// One block; thread b plans sequence b (B <= 1024).  A shared partly filled page with count r
// and m growers is given up by every grower but, when m = r, the last one (sequence by
// sequence, each that leaves lowers the count, and the last finds itself alone): m and the
// highest grower come from two atomics per page in `growers`, cleared before them.
// Entries that will be written are given up first (by their sequence's thread where they are one or two, by a warp
// otherwise), so that pages that a sequence holds past its length serve it again; when the call
// fails they are taken back.
// The free pages are listed in ascending order until enough are found: a pass takes 16 x 1024
// counts, a ballot per 32 of them, and one scan over the 512 ballots ranks them all.  The first
// 4096 stay in shared memory.  Then a warp per sequence writes the entries.
constexpr int kReservePer = 16, kReserveNear = 4096;
__global__ void __launch_bounds__(1024) pages_reserve_kernel(PageBook k, const int32_t* n_new, int32_t* copy_src,
                                                             int32_t* copy_dst, int32_t* growers, int32_t* free_list) {
  __shared__ int part[33];
  __shared__ int lo_s[1024], cnt_s[1024], off_s[1024], votes_s[kReservePer * 32], near_s[kReserveNear];
  __shared__ int past_s[1024], many_s[1024];
  const int b = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ps = k.page_size;
  int len = 0, add = 0, last = -1, past = 0, n_past = 0;  // entries from the length's end on that will be written
  bool fail = false, part_page = false;
  if (b < k.B) {
    bool bad;
    len = clamp_len(k.seq_lens[b], k, &bad);
    add = n_new[b];
    if (bad || add < 0) {
      flag_error(k.status, DEVFLAG_BAD_SEQ_LEN);
      add = 0;
    }
    if (static_cast<int64_t>(len) + add > static_cast<int64_t>(k.max_pages) * ps) fail = true;
    if (add > 0 && !fail) {
      past = static_cast<int>(ceil_div(len, ps));
      n_past = static_cast<int>(ceil_div(static_cast<int64_t>(len) + add, ps)) - past;
    }
    past_s[b] = past;
    many_s[b] = n_past > 2 ? n_past : 0;
    part_page = add > 0 && len % ps != 0;
    if (part_page) {
      last = k.table[static_cast<int64_t>(b) * k.max_pages + len / ps];
      if (last < 0 || last >= k.n_pages) {
        fail = true;
        part_page = false;
      }
    }
  }
  if (part_page) {
    growers[2 * static_cast<int64_t>(last)] = 0;
    growers[2 * static_cast<int64_t>(last) + 1] = 0;
  }
  auto past_entries = [&](auto each) {
    if (n_past <= 2)
      for (int j = 0; j < n_past; ++j) each(k.table + static_cast<int64_t>(b) * k.max_pages + past + j);
    for (int q = warp; q < k.B; q += 32)
      for (int j = lane; j < many_s[q]; j += 32) each(k.table + static_cast<int64_t>(q) * k.max_pages + past_s[q] + j);
  };
  __threadfence_block();
  fail = __syncthreads_or(fail) != 0;
  if (!fail) past_entries([&](int32_t* e) { give_up(k, e, *e); });
  if (!fail && part_page) {
    atomicAdd(growers + 2 * static_cast<int64_t>(last), 1);
    atomicMax(growers + 2 * static_cast<int64_t>(last) + 1, b + 1);
  }
  __threadfence_block();
  __syncthreads();
  bool split = false;
  if (!fail && part_page) {
    const int r = __ldcg(k.ref + last);
    const int m = __ldcg(growers + 2 * static_cast<int64_t>(last));
    const int top = __ldcg(growers + 2 * static_cast<int64_t>(last) + 1);
    split = r > 1 && (m < r || top != b + 1);
  }
  int lo = 0, cnt = 0;
  if (!fail && add > 0) {
    lo = split ? len / ps : static_cast<int>(ceil_div(len, ps));
    cnt = static_cast<int>(ceil_div(static_cast<int64_t>(len) + add, ps)) - lo;
  }
  int total;
  const int off = block_exclusive_scan(cnt, part, &total);  // <= B * max_pages < 2^31? checked by the host
  lo_s[b] = lo;
  cnt_s[b] = cnt;
  off_s[b] = off;
  int found = 0;
  for (int64_t base = 0; !fail && base < k.n_pages && found < total; base += 1024 * kReservePer) {
    uint32_t votes[kReservePer];
    int ref[kReservePer];
#pragma unroll
    for (int u = 0; u < kReservePer; ++u) {
      const int64_t page = base + u * 1024 + threadIdx.x;
      ref[u] = page < k.n_pages ? __ldcg(k.ref + page) : 1;
    }
#pragma unroll
    for (int u = 0; u < kReservePer; ++u) {
      votes[u] = __ballot_sync(0xFFFFFFFFu, ref[u] <= 0);
      if (lane == 0) votes_s[u * 32 + warp] = __popc(votes[u]);
    }
    __syncthreads();
    int here;
    const int at = found + block_exclusive_scan(threadIdx.x < kReservePer * 32 ? votes_s[threadIdx.x] : 0, part, &here);
    if (threadIdx.x < kReservePer * 32) votes_s[threadIdx.x] = at;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kReservePer; ++u) {
      const int rank = votes_s[u * 32 + warp] + __popc(votes[u] & ((1u << lane) - 1u));
      if (((votes[u] >> lane) & 1) && rank < total) {
        const int page = static_cast<int>(base) + u * 1024 + static_cast<int>(threadIdx.x);
        if (rank < kReserveNear) near_s[rank] = page;
        else free_list[rank] = page;
      }
    }
    found += here;
    __syncthreads();
  }
  auto nth_free = [&](int rank) { return rank < kReserveNear ? near_s[rank] : __ldcg(free_list + rank); };
  if (!fail && found < total) {
    past_entries([&](int32_t* e) {
      if (*e >= 0 && *e < k.n_pages) atomicAdd(k.ref + *e, 1);
    });
    fail = true;
  }
  if (fail) {
    if (b < k.B) copy_src[b] = copy_dst[b] = -1;
    if (b == 0) flag_error(k.status, DEVFLAG_NO_PAGES);
    return;
  }
  __threadfence_block();
  __syncthreads();
  for (int q = warp; q < k.B; q += 32) {
    int32_t* row = k.table + static_cast<int64_t>(q) * k.max_pages + lo_s[q];
    for (int j = lane; j < cnt_s[q]; j += 32) {
      const int p = nth_free(off_s[q] + j);
      row[j] = p;
      k.ref[p] = 1;
    }
  }
  if (b < k.B) {
    copy_src[b] = split ? last : -1;
    copy_dst[b] = split ? nth_free(off) : -1;
    if (split) atomicSub(k.ref + last, 1);
    if (add > 0) k.seq_lens[b] = len + add;
  }
}

// ------------------------------------------------------------------ release
__global__ void __launch_bounds__(256) pages_release_kernel(PageBook k, const int32_t* ended, int window,
                                                            int n_sinks) {
  const int b = blockIdx.x;
  bool bad_len, bad_page = false;
  const int len = clamp_len(k.seq_lens[b], k, &bad_len);
  const bool all = ended != nullptr && ended[b] != 0;
  __syncthreads();  // every thread has read the length before it is cleared
  const int64_t ps = k.page_size;
  int32_t* row = k.table + static_cast<int64_t>(b) * k.max_pages;
  if (all || window > 0) {
    for (int j = threadIdx.x; j < k.max_pages; j += blockDim.x) {
      const int p = row[j];
      if (p == -1) continue;
      if (!all && !(j * ps >= n_sinks && (j + 1) * ps <= static_cast<int64_t>(len) - window)) continue;
      row[j] = -1;
      if (p < 0 || p >= k.n_pages) {
        bad_page = true;
      } else if (atomicSub(k.ref + p, 1) <= 0) {  // already free: the count stays
        atomicAdd(k.ref + p, 1);
        bad_page = true;
      }
    }
  }
  if (bad_page) flag_error(k.status, DEVFLAG_BAD_INDEX);
  if (threadIdx.x == 0) {
    if (all) k.seq_lens[b] = 0;
    if (bad_len) flag_error(k.status, DEVFLAG_BAD_SEQ_LEN);
  }
}

// ------------------------------------------------------------------ compact
// One cluster of 8 blocks; block c takes a contiguous slice of the pages.  Pass 1 counts the
// pages in use: m = their number.  Pass 2 counts those below m; the holes below m and the
// pages in use at or above m are equally many.  Pass 3 ranks and lists both.  Then the counts
// move, and the table is rewritten through map[page] = rank of its move: by the same launch
// where the table has few entries, by a second one over the whole GPU otherwise.
constexpr int kCompactBlocks = 8;
constexpr int64_t kCompactEntries = 1 << 16;  // 8 passes of the cluster's threads
__device__ __forceinline__ void remap_entries(const PageBook& k, const int32_t* dst, const int32_t* map, int m,
                                              int64_t i0, int64_t step) {
  const int64_t n = static_cast<int64_t>(k.B) * k.max_pages;
  for (int64_t i = i0; i < n; i += step) {
    const int p = k.table[i];
    if (p >= m && p < k.n_pages) {
      const int r = __ldcg(map + p);
      if (r >= 0) k.table[i] = __ldcg(dst + r);
    }
  }
}
__global__ void __launch_bounds__(1024) __cluster_dims__(kCompactBlocks, 1, 1)
    pages_compact_kernel(PageBook k, int32_t* src, int32_t* dst, int max_moves, int32_t* n_moves, int32_t* map,
                         bool remap) {
  __shared__ int part[33];
  __shared__ int live_s, low_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int c = static_cast<int>(cluster.block_rank());
  const int per = static_cast<int>(ceil_div(ceil_div(k.n_pages, kCompactBlocks), 1024)) * 1024;
  const int64_t lo = static_cast<int64_t>(c) * per, hi = min64(k.n_pages, lo + per);
  int n = 0;
  for (int64_t p = lo + threadIdx.x; p < hi; p += 1024) n += k.ref[p] > 0;
  int total;
  block_exclusive_scan(n, part, &total);
  if (threadIdx.x == 0) live_s = total;
  cluster.sync();
  int m = 0;
  for (int q = 0; q < kCompactBlocks; ++q) m += *cluster.map_shared_rank(&live_s, q);
  n = 0;
  for (int64_t p = lo + threadIdx.x; p < min64(hi, m); p += 1024) n += k.ref[p] > 0;
  block_exclusive_scan(n, part, &total);
  if (threadIdx.x == 0) low_s = total;
  cluster.sync();
  int low = 0, before = 0;  // pages in use below m; pages in use in the slices before this one
  for (int q = 0; q < kCompactBlocks; ++q) {
    low += *cluster.map_shared_rank(&low_s, q);
    if (q < c) before += *cluster.map_shared_rank(&live_s, q);
  }
  const int moves = min(m - low, max_moves);
  for (int64_t base = lo; base < hi; base += 1024) {
    const int64_t p = base + threadIdx.x;
    const int live = p < hi && k.ref[p] > 0;
    const int rank = before + block_exclusive_scan(live, part, &total);  // pages in use below p
    before += total;
    if (p < hi) {
      if (p < m) {
        const int hole = static_cast<int>(p) - rank;
        if (!live && hole < moves) dst[hole] = static_cast<int>(p);
      } else {
        const int mover = rank - low;
        map[p] = live && mover < moves ? mover : -1;
        if (live && mover < moves) src[mover] = static_cast<int>(p);
      }
    }
  }
  for (int64_t i = moves + static_cast<int64_t>(c) * 1024 + threadIdx.x; i < max_moves; i += kCompactBlocks * 1024)
    src[i] = dst[i] = -1;
  if (c == 0 && threadIdx.x == 0) {
    n_moves[0] = moves;
    map[k.n_pages] = m;
  }
  __threadfence();
  cluster.sync();  // both lists are complete, and no block reads the counts any more
  for (int i = c * 1024 + threadIdx.x; i < moves; i += kCompactBlocks * 1024) {
    const int s = __ldcg(src + i), t = __ldcg(dst + i);
    k.ref[t] = k.ref[s];
    k.ref[s] = 0;
  }
  if (remap) remap_entries(k, dst, map, m, c * 1024 + static_cast<int>(threadIdx.x), kCompactBlocks * 1024);
}

__global__ void __launch_bounds__(256) pages_remap_kernel(PageBook k, const int32_t* dst, const int32_t* map) {
  remap_entries(k, dst, map, map[k.n_pages], static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// ------------------------------------------------------------------ copy and append
// Offset, in 16-byte vectors, of vector v of a page seen as [head][row][d / 8].
__device__ __forceinline__ int64_t pool_vec(const int64_t (&st)[3], int page_size, int cpr, int v) {
  const int ch = v % cpr, hr = v / cpr;
  return (hr / page_size) * (st[1] >> 3) + (hr % page_size) * (st[2] >> 3) + ch;
}

// A block takes chunks of 256 x kCopyPer vectors of one pool of one pair; every thread's loads are
// issued before its stores.
constexpr int kCopyPer = 4;
__global__ void __launch_bounds__(256) pages_copy_kernel(PagePool p, const int32_t* src, const int32_t* dst, int n,
                                                         const int32_t* count, int* status) {
  if (count) n = max(0, min(n, count[0]));
  const int cpr = p.d / 8;
  const int vecs = p.Hkv * p.page_size * cpr;  // per page and pool (< 2^31, checked by the host)
  const int chunks = (vecs - 1) / (256 * kCopyPer) + 1;  // every vector's number stays below 2^31
  const int64_t items = static_cast<int64_t>(n) * 2 * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t pair = it / (2 * chunks);
    const int rest = static_cast<int>(it - pair * (2 * chunks));
    const int s = src[pair], t = dst[pair];
    if (s < 0 || t < 0) continue;
    if (s >= p.n_pages || t >= p.n_pages) {
      if (rest == 0 && threadIdx.x == 0) flag_error(status, DEVFLAG_BAD_INDEX);
      continue;
    }
    const bool is_v = rest >= chunks;
    const int64_t(&st)[3] = is_v ? p.vs : p.ks;
    uint4* pool = reinterpret_cast<uint4*>(is_v ? p.V : p.K);
    const uint4* from = pool + s * (st[0] >> 3);
    uint4* to = pool + t * (st[0] >> 3);
    const int v0 = (is_v ? rest - chunks : rest) * 256 * kCopyPer + threadIdx.x;
    uint4 x[kCopyPer];
    int64_t o[kCopyPer];
#pragma unroll
    for (int u = 0; u < kCopyPer; ++u) {
      const int v = v0 + u * 256;
      if (v < vecs) {
        o[u] = pool_vec(st, p.page_size, cpr, v);
        x[u] = __ldcs(from + o[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kCopyPer; ++u)
      if (v0 + u * 256 < vecs) to[o[u]] = x[u];
  }
}

// Row and page of new token `i` (packed), or page -1 if it is not written.
__device__ __forceinline__ int append_place(const PagedAppendArgs& a, int64_t i, int* row) {
  const int b = sequence_of(a.q_begin, a.B, i);
  const NewTokens r = new_tokens(a.q_begin, a.seq_lens, b, static_cast<int64_t>(a.max_pages) * a.pool.page_size,
                                 a.n_tokens, a.n_tokens, a.status);
  if (i < r.q0 || i >= r.q0 + r.nq) return -1;
  const int64_t t = r.len - r.nq + (i - r.q0);
  const int p = a.table[static_cast<int64_t>(b) * a.max_pages + t / a.pool.page_size];
  *row = static_cast<int>(t % a.pool.page_size);
  if (p < 0 || p >= a.pool.n_pages) {
    flag_error(a.status, DEVFLAG_BAD_INDEX);
    return -1;
  }
  return p;
}

// A block takes kAppendTokens tokens: their places first, then their vectors, four loads of a
// thread under way before its first store.  The last block has none: it looks at every sequence, because one in
// disorder may have no token that would come upon it.
constexpr int kAppendTokens = 8, kAppendPer = 4;
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a) {
  __shared__ int page_s[kAppendTokens], row_s[kAppendTokens];
  if (blockIdx.x == gridDim.x - 1) {
    for (int b = threadIdx.x; b < a.B; b += blockDim.x)
      new_tokens(a.q_begin, a.seq_lens, b, static_cast<int64_t>(a.max_pages) * a.pool.page_size, a.n_tokens, a.n_tokens,
                 a.status);
    return;
  }
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kAppendTokens;
  if (threadIdx.x < kAppendTokens) {
    int row = 0;
    page_s[threadIdx.x] = i0 + threadIdx.x < a.n_tokens ? append_place(a, i0 + threadIdx.x, &row) : -1;
    row_s[threadIdx.x] = row;
  }
  __syncthreads();
  const int cpr = a.pool.d / 8, per = a.pool.Hkv * cpr;  // 16-byte vectors of a row, of a token's K or V rows
  const int total = kAppendTokens * 2 * per;
  for (int v0 = threadIdx.x; v0 < total; v0 += 256 * kAppendPer) {
    uint4 x[kAppendPer];
    uint4* to[kAppendPer];
#pragma unroll
    for (int u = 0; u < kAppendPer; ++u) {
      const int v = v0 + u * 256;
      const int j = v / (2 * per), rest = v - j * 2 * per;
      to[u] = nullptr;
      if (v >= total || page_s[j] < 0) continue;
      const bool is_v = rest >= per;
      const int e = is_v ? rest - per : rest;
      const int64_t(&st)[3] = is_v ? a.pool.vs : a.pool.ks;
      x[u] = __ldcs(reinterpret_cast<const uint4*>(is_v ? a.V_new : a.K_new) + (i0 + j) * (a.new_stride >> 3) + e);
      to[u] = reinterpret_cast<uint4*>(is_v ? a.pool.V : a.pool.K) + page_s[j] * (st[0] >> 3) +
              (e / cpr) * (st[1] >> 3) + row_s[j] * (st[2] >> 3) + e % cpr;
    }
#pragma unroll
    for (int u = 0; u < kAppendPer; ++u)
      if (to[u]) *to[u] = x[u];
  }
}

}  // namespace

cudaError_t launch_pages_fork(const PageBook& k, const int32_t* src, const int32_t* dst, int n, cudaStream_t s) {
  return launch_ex(pages_fork_kernel, dim3(n), dim3(256), 0, s, 0, k, src, dst, n);
}

cudaError_t launch_pages_reserve(const PageBook& k, const int32_t* n_new, int32_t* copy_src, int32_t* copy_dst,
                                 int32_t* growers, int32_t* free_list, cudaStream_t s) {
  return launch_ex(pages_reserve_kernel, dim3(1), dim3(1024), 0, s, 0, k, n_new, copy_src, copy_dst, growers,
                   free_list);
}

cudaError_t launch_pages_release(const PageBook& k, const int32_t* ended, int window, int n_sinks, cudaStream_t s) {
  return launch_ex(pages_release_kernel, dim3(k.B), dim3(256), 0, s, 0, k, ended, window, n_sinks);
}

cudaError_t launch_pages_compact(const PageBook& k, int32_t* src, int32_t* dst, int max_moves, int32_t* n_moves,
                                 int32_t* map, cudaStream_t s) {
  const int64_t entries = static_cast<int64_t>(k.B) * k.max_pages;
  const bool remap = entries <= kCompactEntries;
  cudaError_t e = launch_ex(pages_compact_kernel, dim3(kCompactBlocks), dim3(1024), 0, s, 0, k, src, dst, max_moves,
                            n_moves, map, remap);
  if (e != cudaSuccess || remap) return e;
  const int64_t blocks = ceil_div(entries, 256);
  return launch_ex(pages_remap_kernel, dim3(static_cast<unsigned>(min64(blocks, 1024))), dim3(256), 0, s, 0, k,
                   static_cast<const int32_t*>(dst), static_cast<const int32_t*>(map));
}

cudaError_t launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int n, const int32_t* count,
                              int* status, int num_sms, cudaStream_t s) {
  const int64_t chunks = ceil_div(static_cast<int64_t>(p.Hkv) * p.page_size * (p.d / 8), 256 * kCopyPer);
  const int64_t blocks = min64(static_cast<int64_t>(n) * 2 * chunks, static_cast<int64_t>(num_sms) * 64);
  return launch_ex(pages_copy_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, 0, p, src, dst, n, count,
                   status);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  const int64_t blocks = ceil_div(a.n_tokens, kAppendTokens) + 1;
  return launch_ex(paged_append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, 0, a);
}

}  // namespace jssa
