// The work of the attention kernels over a paged cache, cut into pieces: items, the line that they
// form, the walk over a CTA's pieces, the boxes of a tile, and the merge of cut items.
//
// A kernel's constants come as a class C: kD (head dim), kTile (keys per tile), kWG (query tiles of an
// item side by side), kDB = kD / 64, kSoftmax (threads that merge), kThreads, kItemUnits (what a piece
// costs beside its tiles), kQueryMap (queries come by TMA).
#pragma once

#include <cuda.h>

#include "launch.h"
#include "paged.cuh"

namespace jssa {

constexpr int kPaPieces = 4;    // pieces published at once
constexpr int kPaBadRing = 16;  // tiles whose missing pages are remembered
constexpr float kLog2e = 1.4426950408889634f;

struct PaParams {
  CUtensorMap q, k, v;
  PagedAttnArgs a;
  int G, tpt;      // query heads per KV head; tokens per query tile
  int box, nbox;   // rows of a TMA box (a power of two); boxes per tile
  int tile_pages, tile_rows;  // a tile's length in pages and rows
  float scale_log2;
};

// One item: its tokens and the list of its keys.  Place v of the list holds token v below s_al
// and token v + shift from there on; z0 <= v < z1 and v >= nv are seen by no query.
struct Item {
  int tok0, ntok, pf;
  int s_al, shift, z0, z1, nv, ntiles;
  bool solo;  // one query tile
  bool few;   // and all of its sequence's new tokens
};

template <class C>
__device__ __forceinline__ Item item_at(const PaParams& p, int nq, int len, int j) {
  Item it;
  const int tpi = p.tpt * C::kWG;
  it.tok0 = j * tpi;
  it.ntok = min(tpi, nq - it.tok0);
  it.pf = len - nq + it.tok0;
  const int hi = it.pf + it.ntok;
  it.s_al = it.shift = it.z0 = it.z1 = 0;
  if (p.a.window > 0) {
    const int lo = max(0, it.pf + 1 - p.a.window), lo_al = lo & ~(p.box - 1);
    it.z0 = min(p.a.n_sinks, lo);
    const int s_al = (it.z0 + p.box - 1) & ~(p.box - 1);
    if (s_al < lo_al) {
      it.s_al = s_al;
      it.shift = lo_al - s_al;
    }
    it.z1 = lo - it.shift;
  }
  it.nv = hi - it.shift;
  it.ntiles = (it.nv + C::kTile - 1) / C::kTile;
  it.solo = C::kWG == 1 || it.ntok <= p.tpt;
  it.few = nq <= p.tpt;
  return it;
}

// Cut items of more than a warp's rows, each row whole in one accumulator, are merged by a launch of their own
// over the whole GPU; the others by the CTA that finishes them last.
template <class C>
__device__ __forceinline__ bool tall_item(const Item& it, int G) {
  return (!it.solo || C::kWG == 1) && it.ntok * G > 32;
}

// An item's length on the line: a tile of two query tiles counts twice, and what a piece costs
// before its first tile and after its last stands at the front.
template <class C>
__device__ __forceinline__ int64_t item_units(const Item& it) {
  return C::kItemUnits + (it.solo ? it.ntiles : 2 * static_cast<int64_t>(it.ntiles));
}

// Quotient of non-negative numbers, on the 32-bit path where both fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The cuts of the line: CTA c has [start(c), start(c + 1)).
struct Cuts {
  int64_t len, more;  // `more` CTAs have len + 1 units
  __device__ Cuts(int64_t total, int n) : len(quotient(total, n)), more(total - len * n) {}
  __device__ int64_t start(int c) const { return c * len + min64(c, more); }
  __device__ int owner(int64_t x) const {  // of place x
    const int64_t y = x - more * (len + 1);
    return static_cast<int>(y < 0 ? quotient(x, len + 1) : more + quotient(y, len));
  }
};

// A CTA's share of one item: tiles [t0, t1); t1 = 0 ends the CTA's work.  CTAs c_first to c_last share the item.
struct Piece {
  Item it;
  int64_t q0;  // first token's row
  int b, h, t0, t1, c_first, c_last;
};

// Where a CTA's stretch of the line begins.
struct Start {
  Cuts cuts;
  int64_t at;  // start of the item (b, h, j)
  int b, h, j;
  bool idle;
};

// Walks the pieces that fall to this CTA, in order.
template <class C>
struct Walk {
  const PaParams& p;
  Cuts cuts;
  int64_t u, u0, u1, q0;
  int b, h, j, nq, len;

  __device__ Walk(const PaParams& pp, const Start& s) : p(pp), cuts(s.cuts), u(s.at), b(s.b), h(s.h), j(s.j) {
    u0 = cuts.start(blockIdx.x);
    u1 = cuts.start(blockIdx.x + 1);
    load();
    if (s.idle) u = u1 = 0;
  }
  __device__ void load() {
    const NewTokens t = new_tokens(p.a.q_begin, p.a.seq_lens, b,
                                   static_cast<int64_t>(p.a.max_pages) * p.a.pool.page_size, p.a.n_tokens,
                                   p.a.max_q_len, nullptr);
    q0 = t.q0, nq = t.nq, len = t.len;
  }
  __device__ Piece next() {
    Piece c;
    c.t1 = 0;
    while (u < u1) {
      c.it = item_at<C>(p, nq, len, j);
      const int w = c.it.solo ? 1 : 2;
      const int64_t at = u + C::kItemUnits;  // tile i belongs to the CTA that has place at + w i
      c.t0 = at >= u0 ? 0 : static_cast<int>((u0 - at + w - 1) / w);
      c.t1 = at >= u1 ? 0 : static_cast<int>(min64(c.it.ntiles, (u1 - at + w - 1) / w));
      c.b = b, c.h = h, c.q0 = q0 + c.it.tok0;
      u += item_units<C>(c.it);
      ++j;
      if (c.it.tok0 + c.it.ntok == nq) {
        j = 0;
        if (++h == p.a.pool.Hkv) {
          h = 0;
          do {
            if (++b == p.a.B) break;
            load();
          } while (nq == 0);
        }
      }
      if (c.t0 < c.t1) {
        c.c_first = at >= u0 ? static_cast<int>(blockIdx.x) : cuts.owner(at);
        c.c_last = c.t1 == c.it.ntiles ? static_cast<int>(blockIdx.x)
                                       : cuts.owner(at + static_cast<int64_t>(w) * (c.it.ntiles - 1));
        return c;
      }
      c.t1 = 0;
    }
    return c;
  }
};

// Each sequence's length on the line (per KV head), and the largest product of an item's length and
// what one more piece of it costs, into 12 KB of shared memory: by every thread of the CTA.
template <class C>
__device__ __forceinline__ void line_lengths(const PaParams& p, int64_t* seq_units) {
  float* seq_merge = reinterpret_cast<float*>(seq_units + 1024);
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.pool.page_size;
  // a warp per sequence where sequences may have many items, a thread otherwise
  const int tpi = p.tpt * C::kWG;
  const bool wide = a.max_q_len > 8 * tpi;
  const int step = wide ? C::kThreads / 32 : C::kThreads;
  for (int b = wide ? warp : tid; b < a.B; b += step) {
    const NewTokens t = new_tokens(a.q_begin, a.seq_lens, b, cap, a.n_tokens, a.max_q_len,
                                   blockIdx.x == 0 ? a.status : nullptr);
    int64_t n = 0;
    float merge = 0.f;  // the largest product of an item's length and what one more piece of it costs, in units
    for (int j = wide ? lane : 0; j * static_cast<int64_t>(tpi) < t.nq; j += wide ? 32 : 1) {
      const Item it = item_at<C>(p, t.nq, t.len, j);
      const int64_t u = item_units<C>(it);
      n += u;
      // What one more piece of an item adds to its merge, in units (a tile of one query tile is one: about 1 us).  Rows
      // merged by a CTA: a unit for 8,192 values.  A quarter and four times that: one token of 16-head groups over 40K
      // 28.0 us -> 29.9 and 33.4; 100 tokens of one head over 40K 70.3 -> 74.4 and 91.1.  Rows merged by the second launch:
      // 0.15.  None and four times that: 500 tokens of one head over 40K 41.7 -> 44.5 and 43.4; 64 with
      // d = 256 over 20K 28.4 -> 38.1 and 32.9.
      const float cost = tall_item<C>(it, p.G) ? 0.15f : it.ntok * p.G * (C::kD / 8192.f);
      merge = fmaxf(merge, u * cost);
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        merge = fmaxf(merge, __shfl_xor_sync(0xFFFFFFFFu, merge, o));
      }
    }
    if (!wide || lane == 0) {
      seq_units[b] = n;
      seq_merge[b] = merge;
    }
  }
}

// The line's length, and the item that this CTA's stretch of it begins in: by one warp.
template <class C>
__device__ __forceinline__ Start line_start(const PaParams& p, const int64_t* seq_units) {
  const float* seq_merge = reinterpret_cast<const float*>(seq_units + 1024);
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.pool.page_size;
  // the line's length, and the item that this CTA's stretch of it begins in
  const int per = (a.B + 31) / 32;
  int64_t mine = 0;
  float merge = 0.f;
  for (int e = 0; e < per && lane * per + e < a.B; ++e) {
    mine += seq_units[lane * per + e] * a.pool.Hkv;
    merge = fmaxf(merge, seq_merge[lane * per + e]);
  }
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += v;
  }
  const int64_t total = __shfl_sync(0xFFFFFFFFu, before, 31);
  before -= mine;
  // A CTA has two units at least, so that each cut piece has a whole tile, and no less than balances an
  // item's time in pieces of u units, u, against the time to merge them, cost * length / u.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) merge = fmaxf(merge, __shfl_xor_sync(0xFFFFFFFFu, merge, o));
  const int64_t least = max64(2, static_cast<int64_t>(sqrtf(merge)));
  const int nact = static_cast<int>(min64(gridDim.x, max64(1, quotient(total, least))));
  const Cuts cuts(total, nact);
  const bool idle = total == 0 || static_cast<int>(blockIdx.x) >= nact;
  int64_t at = 0;
  int b0 = 0, h0 = 0, j0 = 0;
  if (!idle) {
    const int64_t u0 = cuts.start(blockIdx.x);
    const uint32_t owner = __ballot_sync(0xFFFFFFFFu, u0 >= before && u0 < before + mine);
    const int from = __ffs(owner) - 1;
    at = before;
    b0 = lane * per;
    if (lane == from)
      while (u0 >= at + seq_units[b0] * a.pool.Hkv) at += seq_units[b0++] * a.pool.Hkv;
    at = __shfl_sync(0xFFFFFFFFu, at, from);
    b0 = __shfl_sync(0xFFFFFFFFu, b0, from);
    const int64_t per_head = seq_units[b0];
    h0 = static_cast<int>(quotient(u0 - at, per_head));
    at += h0 * per_head;
    int64_t rem = u0 - at;
    const NewTokens t = new_tokens(a.q_begin, a.seq_lens, b0, cap, a.n_tokens, a.max_q_len, nullptr);
    for (;; j0 += 32) {
      const int64_t tok = (j0 + lane) * static_cast<int64_t>(p.tpt * C::kWG);
      const int64_t n = tok < t.nq ? item_units<C>(item_at<C>(p, t.nq, t.len, j0 + lane)) : 0;
      int64_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, sum > rem);
      if (past) {
        const int l0 = __ffs(past) - 1;
        j0 += l0;
        at += __shfl_sync(0xFFFFFFFFu, sum - n, l0);
        break;
      }
      const int64_t all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      rem -= all;
      at += all;
    }
  }
  return {cuts, at, b0, h0, j0, idle};
}

// The bounded waits of a CTA.  After a timeout the outputs of the call are undefined.
struct Waiter {
  volatile int* dead;
  int* status;
  // The hint lets a waiting warp sleep in the barrier unit; the clock is read every 64 wake-ups, because
  // waiting warps share the issue slots with the ones at work.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    uint64_t t0 = 0;
    for (uint32_t n = 0;; ++n) {
      uint32_t done;
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
          " selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(done)
          : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
          : "memory");
      if (done) return true;
      if (*dead) return false;
      if (n % 64 == 63) {
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
          flag_error(status, DEVFLAG_TIMEOUT);
          *dead = 1;
          return false;
        }
      }
    }
  }
};

// The armed test of the waits (common.cuh): one warp of the first CTA reads the request while the line is worked out, and
// withholds something that other warps wait for.  Their waits give up after their own limit (a shorter one for this
// CTA would have to be read at every wait).
__device__ __forceinline__ int wait_test_armed(const PagedAttnArgs& a) {
  int armed = 0;
  if (blockIdx.x == 0 && (threadIdx.x & 31) == 0)  // volatile: the load is not to be moved to where it is looked at
    asm volatile("ld.global.cg.b32 %0, [%1];" : "=r"(armed) : "l"(a.status + 1));
  return armed;
}

// In a CTA that has given up: the copies into the stages in `used`, which end a phase of their barriers, land.  One of
// a barrier's two phases has always ended, and the wait for the other is short where no copy will end it (a
// copy lands within microseconds).
__device__ __forceinline__ void drain_copies(uint64_t* bars, int n, uint32_t used, int* status) {
  for (int i = 0; i < n; ++i)
    if ((used >> i) & 1)
      for (int t = 0; t < 2; ++t) mbar_wait_bounded(&bars[i], t, status, 1000000);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bits [0, n) of a word, n clamped to [0, 32].
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// One box of an item's tiles, from tile to tile: its page-table entry and row within the page.
template <class C>
struct BoxWalk {
  int v, slot, row;
  __device__ void place(const PaParams& p, const Item& it) {
    const int t = v < it.s_al ? v : v + it.shift;
    slot = t / p.a.pool.page_size;
    row = t - slot * p.a.pool.page_size;
  }
  __device__ BoxWalk(const PaParams& p, const Piece& s, int box) : v(s.t0 * C::kTile + box * p.box) {
    place(p, s.it);
  }
  // Page of the box: -2 where the item has no keys, -1 where the table names no page.
  __device__ int page(const PaParams& p, const Piece& s, bool on) const {
    if (!on || v >= s.it.nv) return -2;
    const int pg = __ldg(p.a.table + static_cast<int64_t>(s.b) * p.a.max_pages + slot);
    return pg < 0 || pg >= p.a.pool.n_pages ? -1 : pg;
  }
  __device__ void step(const PaParams& p, const Item& it) {
    const bool sink = v < it.s_al;
    v += C::kTile;
    if (sink && v >= it.s_al) {
      place(p, it);
    } else {
      slot += p.tile_pages;
      row += p.tile_rows;
      if (row >= p.a.pool.page_size) row -= p.a.pool.page_size, ++slot;
    }
  }
};

// Whether tile i holds rows that no query of the item sees.
template <class C>
__device__ __forceinline__ bool edge_tile(const Item& it, int i) {
  const int v0 = i * C::kTile, v1 = v0 + C::kTile;
  return v1 > it.nv || (it.z0 < it.z1 && v0 < it.z1 && v1 > it.z0);
}

// Stores 32 consecutive outputs of a row.
template <bool F32>
__device__ __forceinline__ void store_out32(void* O, int64_t at, const float (&v)[32]) {
  if constexpr (F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(O) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(O) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                        pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
  }
}

// Merges the pieces of a cut item in their order: the softmax threads of the CTA that finishes it
// last.  A thread takes kWords 16-byte words of rows at a time and kParts partials of each at once;
// with fewer words than threads, 2^sh neighbouring lanes share a word's partials.
template <class C, bool F32, int kWords, int kParts>
__device__ __forceinline__ void merge_words(const PaParams& p, const Piece& s, int words, int sh) {
  const PagedAttnArgs& a = p.a;
  const int n = s.c_last - s.c_first + 1, part = threadIdx.x & ((1 << sh) - 1), wstep = C::kSoftmax >> sh;
  for (int w0 = 0; w0 < words; w0 += kWords * wstep) {
    float4 o[kWords];
    float M[kWords], L[kWords];
    int row[kWords], col[kWords];
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      const int idx = w0 + x * wstep + (threadIdx.x >> sh);
      row[x] = idx < words ? idx / (C::kD / 4) : -1;
      col[x] = idx % (C::kD / 4);
      o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      M[x] = -INFINITY;
      L[x] = 0.f;
    }
    for (int k0 = part; k0 < n; k0 += kParts << sh) {
      float2 ml[kWords][kParts];
      float4 v[kWords][kParts];
#pragma unroll
      for (int x = 0; x < kWords; ++x)
#pragma unroll
        for (int y = 0; y < kParts; ++y) {
          const int k = k0 + (y << sh);
          ml[x][y] = make_float2(-INFINITY, 0.f);
          v[x][y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row[x] < 0 || k >= n) continue;
          // an item's first piece is the last of its CTA, the others the first of theirs
          const int64_t at = static_cast<int64_t>(2 * (s.c_first + k) + (k == 0 ? 1 : 0)) * a.rows_cap + row[x];
          ml[x][y] = __ldcg(&a.part_ml[at]);
          v[x][y] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * C::kD) + col[x]);
        }
#pragma unroll
      for (int x = 0; x < kWords; ++x) {
        float mn = M[x];
#pragma unroll
        for (int y = 0; y < kParts; ++y) mn = fmaxf(mn, ml[x][y].x);  // a piece without keys has m = -infinity
        const float z = mn == -INFINITY ? 0.f : mn * p.scale_log2;
        const float w = exp2_approx(fmaf(M[x], p.scale_log2, -z));
        M[x] = mn;
        L[x] *= w;
        o[x].x *= w, o[x].y *= w, o[x].z *= w, o[x].w *= w;
#pragma unroll
        for (int y = 0; y < kParts; ++y) {
          const float u = exp2_approx(fmaf(ml[x][y].x, p.scale_log2, -z));
          L[x] = fmaf(u, ml[x][y].y, L[x]);
          o[x].x = fmaf(u, v[x][y].x, o[x].x), o[x].y = fmaf(u, v[x][y].y, o[x].y);
          o[x].z = fmaf(u, v[x][y].z, o[x].z), o[x].w = fmaf(u, v[x][y].w, o[x].w);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      for (int y = 1; y < 1 << sh; y <<= 1) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, M[x], y), l2 = __shfl_xor_sync(0xFFFFFFFFu, L[x], y);
        const float mn = fmaxf(M[x], m2), z = mn == -INFINITY ? 0.f : mn * p.scale_log2;
        const float w1 = exp2_approx(fmaf(M[x], p.scale_log2, -z)), w2 = exp2_approx(fmaf(m2, p.scale_log2, -z));
        M[x] = mn;
        L[x] = w1 * L[x] + w2 * l2;
        o[x].x = w1 * o[x].x + w2 * __shfl_xor_sync(0xFFFFFFFFu, o[x].x, y);
        o[x].y = w1 * o[x].y + w2 * __shfl_xor_sync(0xFFFFFFFFu, o[x].y, y);
        o[x].z = w1 * o[x].z + w2 * __shfl_xor_sync(0xFFFFFFFFu, o[x].z, y);
        o[x].w = w1 * o[x].w + w2 * __shfl_xor_sync(0xFFFFFFFFu, o[x].w, y);
      }
      if (part != 0 || row[x] < 0) continue;
      const float g = L[x] > 0.f ? 1.f / L[x] : 0.f;
      o[x].x *= g, o[x].y *= g, o[x].z *= g, o[x].w *= g;
      const int64_t to = (s.q0 + row[x] / p.G) * a.Hq + s.h * p.G + row[x] % p.G;
      if constexpr (F32)
        reinterpret_cast<float4*>(static_cast<float*>(a.O) + to * C::kD)[col[x]] = o[x];
      else
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + to * C::kD)[col[x]] =
            make_uint2(pack_bf16x2(o[x].x, o[x].y), pack_bf16x2(o[x].z, o[x].w));
      if (col[x] == 0 && a.lse) a.lse[to] = L[x] > 0.f ? M[x] * a.sm_scale + logf(L[x]) : -INFINITY;
    }
  }
}

template <class C, bool F32>
__device__ __forceinline__ void merge_pieces(const PaParams& p, const Piece& s) {
  const int words = s.it.ntok * p.G * (C::kD / 4);
  int sh = 0;
  while (sh < 5 && (words << (sh + 1)) <= C::kSoftmax) ++sh;
  if (words > C::kSoftmax && s.c_last - s.c_first < 8) merge_words<C, F32, 4, 2>(p, s, words, 0);
  else merge_words<C, F32, 1, 8>(p, s, words, sh);
}

// 16-byte word w of a two-query-tile piece's rows in the workspace: row after row.
__device__ __forceinline__ float4* part_word(const PagedAttnArgs& a, int d, int slot, int w) {
  return reinterpret_cast<float4*>(a.part_o) + (static_cast<int64_t>(slot) * (d / 4) + w) * a.rows_cap;
}

// ------------------------------------------------------------------ host
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Map of a bf16 tensor whose innermost extent is d (boxes of 64 of them, 128-byte swizzle).  The
// stride of an extent of 1 is never used and set to a row's, which the encoder accepts.
inline bool encode(CUtensorMap* m, const void* base, int rank, const int64_t* extent, const int64_t* stride,
                   const int* box) {
  cuuint64_t dims[5], strides[4];
  cuuint32_t boxes[5], ones[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    dims[i] = static_cast<cuuint64_t>(extent[i]);
    boxes[i] = static_cast<cuuint32_t>(box[i]);
    if (i > 0) strides[i - 1] = static_cast<cuuint64_t>(extent[i] > 1 ? stride[i] : extent[0]) * 2;
  }
  const EncodeTiled fn = encode_tiled();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims,
                  strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Parameters of a launch whose query tiles hold tpt tokens.
template <class C>
inline bool paged_params(const PagedAttnArgs& a, int tpt, PaParams* p) {
  p->a = a;
  p->G = a.Hq / a.pool.Hkv;
  p->tpt = tpt;
  p->box = 16;  // the largest power of two that divides a page, at most a tile
  while (p->box < C::kTile && a.pool.page_size % (2 * p->box) == 0) p->box *= 2;
  p->nbox = C::kTile / p->box;
  p->tile_pages = C::kTile / a.pool.page_size;
  p->tile_rows = C::kTile % a.pool.page_size;
  p->scale_log2 = a.sm_scale * kLog2e;
  const int64_t qe[3] = {C::kD, a.Hq, a.n_tokens}, qs[3] = {1, C::kD, a.q_stride};
  const int qb[3] = {64, p->G, p->tpt};
  const int64_t ke[4] = {C::kD, a.pool.page_size, a.pool.Hkv, a.pool.n_pages};
  const int64_t ks[4] = {1, a.pool.ks[2], a.pool.ks[1], a.pool.ks[0]};
  const int kb[4] = {64, p->box, 1, 1};
  // V's 64-dim blocks are a dimension of their own: one box brings all of a row
  const int64_t ve[5] = {64, a.pool.page_size, C::kDB, a.pool.Hkv, a.pool.n_pages};
  const int64_t vs[5] = {1, a.pool.vs[2], 64, a.pool.vs[1], a.pool.vs[0]};
  const int vb[5] = {64, p->box, C::kDB, 1, 1};
  return (!C::kQueryMap || encode(&p->q, a.Q, 3, qe, qs, qb)) && encode(&p->k, a.pool.K, 4, ke, ks, kb) &&
         encode(&p->v, a.pool.V, 5, ve, vs, vb);
}

}  // namespace jssa
