// Attention over a paged cache for few query rows: a KV head's group and new tokens of a sequence
// together fill at most 16 rows, 32 for d = 64 (decode, and a few speculated tokens).
//
// Such a call is bound by the bytes of K and V.  On the 128-row tiles of the large kernel it would
// spend 8 to 128 times the matrix work that it needs (whose power lowers the clock: one token over
// 4 x 115K rows of 8 heads took 333 us under load there), and one warp's rows would hold up each tile.
// Here 16 keys of a tile belong to one warp (two warps that halve the output's columns for d = 256):
// it scores them with 16 x 8 x 16 MMAs, keeps its own maximum, sum and output rows in registers, and
// waits for nobody until the piece ends.  Then the warps' rows are added up in shared memory.
//
// Measured on a B200: one token over 4 x 100K-131K rows of 8 heads, d = 128, 299 us, the rate of a plain
// copy; with the 128-row tiles 303, and 333 under sustained load.  One token of a 2K sequence 15 us
// (16.7), of 64 sequences of 700-3,000 tokens 93 us (105), of 16 with d = 64 49 us (62).  Two query rows
// over 8 windows of 1,024 keys, d = 256: 28 us, of which 5 until the first keys arrive, 11 for 67 MB of
// keys and values, and 10 to add up the warps and merge the pieces.
//
// The work is cut, loaded (TMA boxes that never cross a page, K and V of a tile in one stage) and
// merged as in the large kernel.  V rows that no query sees may hold anything: their fragments are
// zeroed in registers.  P goes into the product with V in two bf16 parts, p and p - bf16(p), 16 bits in
// all: with few rows a rounding of the weights to bf16 does not average out (on one token of a 2K
// sequence the output was off by 2.8e-3, a bf16 output alone by 1.6e-3), and the MMAs have room.
#include "common.cuh"
#include "launch.h"
#include "paged_line.cuh"
#include "tcgen05.cuh"

namespace jssa {
namespace {

// Four 8 x 8 matrices from an address in the shared window, as they are and transposed.
__device__ __forceinline__ void ldmatrix_x4_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// MT: row tiles of 16.
template <int D, int MT>
struct Few {
  static constexpr int kD = D;
  static constexpr int kItemUnits = 4;
  static constexpr bool kQueryMap = false;
  static constexpr int kRows = 16 * MT;
  static constexpr int kTile = D == 256 ? 64 : 128;
  static constexpr int kWG = 1;
  static constexpr int kDB = D / 64;
  static constexpr int kKeyWarps = kTile / 16;           // warps side by side over a tile's keys
  static constexpr int kDimWarps = 8 / kKeyWarps;        // and over the output's columns
  static constexpr int kCols = D / kDimWarps;            // output columns of a warp
  static constexpr int kHalfStage = kTile * D * 2;       // K or V of a tile
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kSumBytes = 4 * kRows * kCols * 4;   // half the warps' output rows
  static constexpr int kSmem = 2 * kStages * kHalfStage + kSumBytes;
  static constexpr int kSoftmax = 256;
  static constexpr int kThreads = kSoftmax + 32;
};

template <int D, bool F32, int MT>
__global__ void __launch_bounds__((Few<D, MT>::kThreads), 1) paged_few_kernel(const __grid_constant__ PaParams p) {
  using C = Few<D, MT>;
  constexpr int kTile = C::kTile, kDB = C::kDB, kNS = C::kStages, kCols = C::kCols, kKeyWarps = C::kKeyWarps;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kNS], empty[kNS], piece_full[kPaPieces], piece_empty[kPaPieces], all_bar;
  __shared__ Piece pieces[kPaPieces], late_piece;
  __shared__ uint32_t bad_s[kPaBadRing];
  __shared__ float m_s[8][C::kRows], l_s[8][C::kRows];
  __shared__ int dead_s, last_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedAttnArgs& a = p.a;
  if (tid == 0) {
    prefetch_tensormap(&p.k);
    prefetch_tensormap(&p.v);
  }
  int64_t* seq_units = reinterpret_cast<int64_t*>(smem_raw);
  line_lengths<C>(p, seq_units);
  if (tid == 0) {
    dead_s = 0;
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);
    }
    for (int i = 0; i < kPaPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], 8);
    }
    mbar_init(&all_bar, 8);
    fence_mbarrier_init();
  }
  fence_async_smem();
  __syncthreads();
  const uint32_t kv_s = smem_u32(smem_raw);
  float* sum_s = reinterpret_cast<float*>(smem_raw + 2 * kNS * C::kHalfStage);
  const Waiter wait{&dead_s, a.status};
  auto all_ok = [&](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };

  if (warp == 8) {
    // ------------------------------------------------------------------ pieces and loads
    const int box = lane / kDB, db = lane % kDB;
    const bool on = box < p.nbox;
    uint32_t st = 0, st_par = 1, used = 0, tiles = 0;
    bool ok = true, late = false;
    const Start at0 = line_start<C>(p, seq_units);
    __syncwarp();
    fence_async_smem();
    Walk<C> walk(p, at0);
    for (int piece = 0; ok; ++piece) {
      const int at = piece % kPaPieces;
      if (piece >= kPaPieces) ok = all_ok(wait(&piece_empty[at], ((piece / kPaPieces) & 1) ^ 1));
      if (!ok) break;
      {
        Piece c = walk.next();
        if (piece == 0 && c.t1 > 0 && c.t0 > 0) {
          late = true;
          if (lane == 0) late_piece = c;
          __syncwarp();
          c = walk.next();
        }
        if (c.t1 == 0 && late) {
          late = false;
          c = late_piece;
        }
        if (lane == 0) {
          pieces[at] = c;
          mbar_arrive(&piece_full[at]);
        }
        __syncwarp();
      }
      const Piece& s = pieces[at];
      if (s.t1 == 0) break;
      BoxWalk<C> bw(p, s, box);
      int pg_next = bw.page(p, s, on);
      for (int i = s.t0; i < s.t1; ++i) {
        const int pg = pg_next, row = bw.row;
        bw.step(p, s.it);
        pg_next = i + 1 < s.t1 ? bw.page(p, s, on) : -2;
        ok = all_ok(wait(&empty[st], st_par));
        if (!ok) break;
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, pg == -1);
        const uint32_t loads = __popc(__ballot_sync(0xFFFFFFFFu, pg >= 0));
        if (lane == 0) {
          bad_s[tiles % kPaBadRing] = bad;
          if (bad) flag_error(a.status, DEVFLAG_BAD_INDEX);
          mbar_arrive_expect_tx(&full[st], 2 * loads * p.box * 128);
        }
        __syncwarp();
        const uint32_t k_at = kv_s + 2 * st * C::kHalfStage, v_at = k_at + C::kHalfStage;
        if (pg >= 0)
          tma_load_4d(k_at + db * (kTile * 128) + box * p.box * 128, &p.k, db * 64, row, s.h, pg, &full[st]);
        if (pg >= 0 && db == 0)
          tma_load_5d(v_at + box * p.box * (kDB * 128), &p.v, 0, row, 0, s.h, pg, &full[st]);
        used |= 1u << st;
        if (++st == kNS) st = 0, st_par ^= 1;
        ++tiles;
      }
    }
    if (dead_s && lane == 0) drain_copies(full, kNS, used, a.status);
  } else {
    // ------------------------------------------------------------------ attention
    const int kw = warp % kKeyWarps, dw = warp / kKeyWarps;  // this warp's keys and columns
    const int r0 = lane >> 2, c2 = (lane & 3) * 2;           // its rows r0, r0 + 8, ..., its columns c2, c2 + 1 of 8
    uint32_t st = 0, st_par = 0, tiles = 0, all_par = 0;
    bool ok = true;
    const int armed = warp == 7 ? wait_test_armed(a) : 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&all_bar);
      const bool x = all_ok(wait(&all_bar, all_par));
      all_par ^= 1;
      return x;
    };
    for (int piece = 0; ok; ++piece) {
      ok = all_ok(wait(&piece_full[piece % kPaPieces], (piece / kPaPieces) & 1));
      const Piece& s = pieces[piece % kPaPieces];
      if (!ok || s.t1 == 0) break;
      const int rows = s.it.ntok * p.G;
      uint32_t q[MT][D / 16][4];
      int pos[2 * MT];
#pragma unroll
      for (int y = 0; y < 2 * MT; ++y) {
        const int r = r0 + 8 * y, tok = min(r / p.G, s.it.ntok - 1);
        pos[y] = s.it.pf + tok;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.Q) +
                                                                (s.q0 + tok) * a.q_stride +
                                                                static_cast<int64_t>(s.h * p.G + r % p.G) * D + c2);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q[y >> 1][kk][y & 1] = r < rows ? __ldg(src + kk * 8) : 0u;
          q[y >> 1][kk][2 + (y & 1)] = r < rows ? __ldg(src + kk * 8 + 4) : 0u;
        }
      }
      const int pl = s.it.pf + s.it.ntok - 1;
      const int b_max = (a.window > 0 ? max(0, pl + 1 - a.window) : 0) - s.it.shift, c_min = s.it.pf + 1 - s.it.shift;
      float m[2 * MT], l[2 * MT];
      float o[MT][kCols / 8][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        m[2 * t] = m[2 * t + 1] = -INFINITY;
        l[2 * t] = l[2 * t + 1] = 0.f;
#pragma unroll
        for (int n = 0; n < kCols / 8; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
      }
      for (int i = s.t0; i < s.t1; ++i) {
        ok = all_ok(wait(&full[st], st_par));
        if (!ok) break;
        const uint32_t k_at = kv_s + 2 * st * C::kHalfStage, v_at = k_at + C::kHalfStage;
        const int k0 = 16 * kw, v0 = i * kTile + k0;
        // scores of keys k0 .. k0 + 15
        float x[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][0][e] = x[t][1][e] = 0.f;
        {
          const int key = k0 + (lane >> 4) * 8 + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            ldmatrix_x4_at(b, k_at + (kk >> 2) * (kTile * 128) + key * 128 + ((((kk & 3) * 2 + ch) ^ (key & 7)) << 4));
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              mma_bf16_16816(x[t][0], q[t][kk], b[0], b[1]);
              mma_bf16_16816(x[t][1], q[t][kk], b[2], b[3]);
            }
          }
        }
        const uint32_t bad = bad_s[tiles % kPaBadRing];
        const bool lost = (bad >> ((k0 / p.box) * kDB)) & 1;
        const bool edge = lost || v0 < b_max || v0 + 16 > c_min;
        uint32_t keep[2] = {~0u, ~0u};  // halves of a V fragment register: keys c2, c2 + 1 (and 8 further)
        if (edge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int v = v0 + 8 * n + c2 + e, t = v < s.it.s_al ? v : v + s.it.shift;  // place and token
#pragma unroll
              for (int y = 0; y < 2 * MT; ++y) {
                const bool seen = !lost && t <= pos[y] && (a.window == 0 || t > pos[y] - a.window || t < a.n_sinks);
                if (!seen) x[y >> 1][n][2 * (y & 1) + e] = -INFINITY;
              }
              if (lost || v >= s.it.nv || (v >= s.it.z0 && v < s.it.z1)) keep[n] &= e ? 0x0000FFFFu : 0xFFFF0000u;
            }
        }
        // each row's maximum over the warp's keys; the output is rescaled when it grows by more than 2^8
        float mx[2 * MT];
        bool move = false;
#pragma unroll
        for (int y = 0; y < 2 * MT; ++y) {
          const float(&z)[2][4] = x[y >> 1];
          const int e = 2 * (y & 1);
          mx[y] = fmaxf(fmaxf(z[0][e], z[0][e + 1]), fmaxf(z[1][e], z[1][e + 1]));
          mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 1));
          mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], 2));
          move |= m[y] == -INFINITY ? mx[y] > -INFINITY : (mx[y] - m[y]) * p.scale_log2 > 8.f;
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
          for (int y = 0; y < 2 * MT; ++y) {
            const float mn = fmaxf(m[y], mx[y]);
            const float w = m[y] == -INFINITY ? 0.f : exp2_approx((m[y] - mn) * p.scale_log2);
            m[y] = mn;
            l[y] *= w;
#pragma unroll
            for (int n = 0; n < kCols / 8; ++n) {
              o[y >> 1][n][2 * (y & 1)] *= w;
              o[y >> 1][n][2 * (y & 1) + 1] *= w;
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 2 * MT; ++y) {
          const float mm = m[y] == -INFINITY ? 0.f : m[y] * p.scale_log2;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& z = x[y >> 1][n][2 * (y & 1) + e];
              z = exp2_approx(fmaf(z, p.scale_log2, -mm));
              l[y] += z;
            }
        }
        uint32_t hi[MT][4];
        uint32_t lo[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int f = 0; f < 4; ++f) {  // A fragment: row r0 + 8 (f & 1), keys c2, c2 + 1 of half f >> 1
            const float p0 = x[t][f >> 1][2 * (f & 1)], p1 = x[t][f >> 1][2 * (f & 1) + 1];
            hi[t][f] = pack_bf16x2(p0, p1);
            lo[t][f] =
                pack_bf16x2(p0 - bf16_bits_to_float(hi[t][f] & 0xFFFFu), p1 - __uint_as_float(hi[t][f] & 0xFFFF0000u));
          }
        {
          const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
          const uint32_t vb_at = v_at + (k0 / p.box) * p.box * (kDB * 128) + (k0 % p.box) * 128 + key * 128;
#pragma unroll
          for (int n = 0; n < kCols / 16; ++n) {
            const int ch = dw * (kCols / 8) + 2 * n + (lane >> 4);  // 8-dim chunk
            uint32_t b[4];
            ldmatrix_x4_trans_at(b, vb_at + (ch >> 3) * p.box * 128 + (((ch & 7) ^ (key & 7)) << 4));
            if (edge) b[0] &= keep[0], b[1] &= keep[1], b[2] &= keep[0], b[3] &= keep[1];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              mma_bf16_16816(o[t][2 * n], hi[t], b[0], b[1]);
              mma_bf16_16816(o[t][2 * n + 1], hi[t], b[2], b[3]);
              mma_bf16_16816(o[t][2 * n], lo[t], b[0], b[1]);
              mma_bf16_16816(o[t][2 * n + 1], lo[t], b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == kNS) st = 0, st_par ^= 1;
        ++tiles;
      }
      if (!ok) break;
      // ---- the warps' rows on one maximum, then their sums
#pragma unroll
      for (int y = 0; y < 2 * MT; ++y) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 1);
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], 2);
        if (m[y] == -INFINITY) l[y] = 0.f;
        if ((lane & 3) == 0) m_s[warp][r0 + 8 * y] = m[y], l_s[warp][r0 + 8 * y] = l[y];
      }
      ok = all_ok(armed != 1) && meet();
      if (!ok) break;
      auto row_max = [&](int r) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kKeyWarps; ++w) M = fmaxf(M, m_s[w][r]);
        return M;
      };
#pragma unroll
      for (int y = 0; y < 2 * MT; ++y) {
        const float M = row_max(r0 + 8 * y);
        const float w = m[y] == -INFINITY ? 0.f : exp2_approx((m[y] - M) * p.scale_log2);
#pragma unroll
        for (int n = 0; n < kCols / 8; ++n) {
          o[y >> 1][n][2 * (y & 1)] *= w;
          o[y >> 1][n][2 * (y & 1) + 1] *= w;
        }
      }
      // four warps' worth of room: the upper half of the key warps hands its rows down, then the rest of them
      constexpr int kHalf = kKeyWarps / 2;
      auto room = [&](int k, int r, int c) { return sum_s + ((k * C::kDimWarps + dw) * C::kRows + r) * kCols + c; };
      auto put = [&](int k) {
#pragma unroll
        for (int n = 0; n < kCols / 8; ++n)
#pragma unroll
          for (int y = 0; y < 2 * MT; ++y)
            *reinterpret_cast<float2*>(room(k, r0 + 8 * y, 8 * n + c2)) =
                make_float2(o[y >> 1][n][2 * (y & 1)], o[y >> 1][n][2 * (y & 1) + 1]);
      };
      if (kw >= kHalf) put(kw - kHalf);
      ok = meet();
      if (!ok) break;
      if (kw < kHalf) {
#pragma unroll
        for (int n = 0; n < kCols / 8; ++n)
#pragma unroll
          for (int y = 0; y < 2 * MT; ++y) {
            const float2 t = *reinterpret_cast<const float2*>(room(kw, r0 + 8 * y, 8 * n + c2));
            o[y >> 1][n][2 * (y & 1)] += t.x;
            o[y >> 1][n][2 * (y & 1) + 1] += t.y;
          }
        put(kw);
      }
      ok = meet();
      if (!ok) break;
      const bool whole = s.c_first == s.c_last;
      const int slot_out = 2 * static_cast<int>(blockIdx.x) + (static_cast<int>(blockIdx.x) == s.c_first ? 1 : 0);
      for (int idx = tid; idx < rows * (D / 4); idx += C::kSoftmax) {
        const int r = idx / (D / 4), c = idx % (D / 4) * 4, d0 = c / kCols;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
          const float* from = sum_s + ((k * C::kDimWarps + d0) * C::kRows + r) * kCols + c % kCols;
          const float4 y = *reinterpret_cast<const float4*>(from);
          t.x += y.x, t.y += y.y, t.z += y.z, t.w += y.w;
        }
        const float M = row_max(r);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kKeyWarps; ++w)
          L += m_s[w][r] == -INFINITY ? 0.f : exp2_approx((m_s[w][r] - M) * p.scale_log2) * l_s[w][r];
        if (whole) {
          const float g = L > 0.f ? 1.f / L : 0.f;
          t.x *= g, t.y *= g, t.z *= g, t.w *= g;
          const int64_t to = (s.q0 + r / p.G) * a.Hq + s.h * p.G + r % p.G;
          if constexpr (F32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.O) + to * D + c) = t;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + to * D + c) =
                make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
          if (c == 0 && a.lse) a.lse[to] = L > 0.f ? M * a.sm_scale + logf(L) : -INFINITY;
        } else {
          const int64_t at = static_cast<int64_t>(slot_out) * a.rows_cap + r;
          *reinterpret_cast<float4*>(a.part_o + at * D + c) = t;
          if (c == 0) a.part_ml[at] = make_float2(M, L);
        }
      }
      ok = meet();  // the partial is written, and sum_s, m_s and l_s have been read
      if (!ok) break;
      if (!whole) {
        if (tid == 0) {
          const int n = s.c_last - s.c_first + 1;
          __threadfence();
          const bool last = atomicAdd(a.counters + s.c_first, 1) == n - 1;
          if (last) a.counters[s.c_first] = 0;
          __threadfence();
          last_s = last;
        }
        ok = meet();
        if (!ok) break;
        if (last_s) merge_pieces<C, F32>(p, s);
        ok = meet();  // last_s has been read
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[piece % kPaPieces]);
    }
    if (armed == 1) wait_test_disarm(a.status);
  }
  __syncthreads();
}

template <int D, bool F32, int MT>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  using C = Few<D, MT>;
  PaParams p{};
  if (!paged_params<C>(a, C::kRows / (a.Hq / a.pool.Hkv), &p)) return cudaErrorInvalidValue;
  auto kernel = paged_few_kernel<D, F32, MT>;
  static int done[64] = {0};
  const cudaError_t e = set_smem_limit_once(kernel, C::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_ex(kernel, dim3(num_sms), dim3(C::kThreads), C::kSmem, s, 0, p);
}

template <int D, int MT>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  return a.out_bf16 ? launch<D, false, MT>(a, num_sms, s) : launch<D, true, MT>(a, num_sms, s);
}

}  // namespace

// Up to 16 rows, both sides measured: 16 rows over 8 caches of 5K, d = 128, 41.3 us here and 52.7 in the large kernel;
// d = 256 76.6 and 75.2, but 4 rows 68.3 and 71.9.  Two row tiles pay for d = 64 only: 8 tokens of 4-head groups over 16
// caches of 12K and 8 KV heads 105 us here and 120 in the large kernel; for d = 128, where a tile must shrink to 64
// keys, over 8 caches of 5K 69 and 49 (short runs).
bool paged_few_rows(int d, int64_t rows) { return rows <= (d == 64 ? 32 : 16); }

cudaError_t launch_paged_few(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  const bool one = static_cast<int64_t>(a.max_q_len) * (a.Hq / a.pool.Hkv) <= 16;
  switch (a.pool.d) {
    case 64: return one ? launch<64, 1>(a, num_sms, s) : launch<64, 2>(a, num_sms, s);
    case 128: return launch<128, 1>(a, num_sms, s);
    case 256: return launch<256, 1>(a, num_sms, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace jssa
