// Attention of each sequence's newest tokens over a paged cache: causal, with an optional
// sliding window and sinks, on the fifth-generation tensor cores.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(sm_scale q . k_t - m),  t over the visible tokens
//
// in one pass over K and V with a running maximum m and sum per row.  The query rows of one KV
// head's group stand side by side: row r of a query tile is token r / G, head r % G of the group,
// so that one tile of 128 rows serves a single token of 128 heads and 128 tokens of one head
// alike, and a K/V row is read once for the whole group.  (Calls of few rows per sequence and KV
// head go to paged_few.cu.)
//
// Items: (sequence, KV head, block of query tiles).  An item's keys are a list of 128 (64 for
// d = 256) at a time, its tiles: the sink pages' first rows, then the rows from the first
// query's window to the last query.  All tiles of all items form one line that is cut into equal
// pieces, one per CTA (one CTA per SM): long caches with few rows are split, ragged batches are
// balanced, and the host needs no lengths.  An item that is cut leaves unnormalised partial
// outputs with their maxima and sums in the workspace.  They are merged in the order of the cuts, so
// results do not depend on timing: items of many rows by a second launch, whose blocks come as CTAs
// leave (the last CTA alone took 2 us per piece: 500 tokens of one head over 40K keys 79 us, so 42),
// the others by the CTA that finishes them last.
//
// Per tile:  S = Q K^T (M = 128 rows, N = keys), P = exp2(S - m) by one thread per row, written
// over S in tensor memory, O += P V with P as the tensor-memory operand.  Two softmax
// warpgroups (one for d = 256) take turns with the tensor core: items of more than one query tile
// give each warpgroup a tile of rows; items of one give them every other tile of keys, and the
// two halves are added at the end.  O stays in tensor memory; the maximum that P refers to
// moves only when a row's grows by more than 2^8, so O is rarely rescaled.
//
// P goes into the product with V in two bf16 parts, bf16(p) and p - bf16(p), so that it is good to 2^-16:
// with an fp32 output, and for every sequence whose new tokens fit one query tile (at most 128 rows per KV head), whatever
// else is in the call.  Longer ones with a bf16 output have it rounded to bf16, which adds about as much error as
// rounding the output does, and one exponential in 16 from a cubic good to 7.5e-5 (in the sums and in lse too).
// Maxima, sums and O are fp32.
//
// Warps: softmax; then one that issues the MMAs, one that walks the pieces and loads Q and K, one
// that loads V (TMA boxes that never cross a page; two warps, because with 16-row pages one took
// 3,900 cycles to issue a tile's boxes against 3,600 of the tile's work), and one that zeroes
// the V rows of a loaded tile that no query of the item sees: P is 0 there, but such rows may
// hold infinities or NaN.
//
// What bounds it, measured on a B200 (d = 128, 4 query heads per KV head, bf16 output): 4 x 512 tokens at 32K 1,079 us
// and an 8K prompt from nothing 585 us, call after call at the power-capped clock: 1.01 and 0.94 PFLOP/s of bf16, 0.72
// and 0.67 of the matrix rate measured under that cap.  The 8K prompt with d = 64 takes 480 us (0.57 PFLOP/s:
// the same softmax for half the matrix work), with d = 256 and 16 heads 628 (0.88), with an fp32 output 872 (its second
// part of P is half as much matrix work again).
// A tile of two query tiles takes about 3,600 cycles for 2,048 of matrix work: a row's softmax (load of S, maximum, 128
// exponentials, store of P: 2,300 cycles while the other warpgroup shares the pipes) and its products follow one
// another; neither the tensor pipe (43 %) nor the issue slots (31 %) are full.  Tried and slower (short runs,
// before the power cap): tiles of 64 keys with two S slots per stream (the N = 64 score MMAs take as long as N = 128
// ones: 1,427 us against 950), four softmax warpgroups on half tiles (1,430), S read twice in chunks (1,277).
// The products begin with the first half of P (about 1 %); a few of the exponentials go to the FMA pipe (none 983,
// an eighth or a sixteenth 950, a quarter 1,012 us).
//
// Every wait is bounded; on a timeout the kernel raises DEVFLAG_TIMEOUT, all roles leave their
// loops, copies and MMAs in flight are drained, and tensor memory is freed.
#include <type_traits>

#include <cuda.h>

#include "common.cuh"
#include "launch.h"
#include "paged_line.cuh"
#include "tcgen05.cuh"

namespace jssa {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kPaOCol = 256;   // first TMEM column of O; S (and P over it) below
constexpr float kPaRescale = 8.f;   // log2 margin before the running maximum moves
constexpr int kPaCubicEvery = 16;    // of so many pairs of exponentials, one goes to the FMA pipe

template <int D>
struct Pa {
  static constexpr int kD = D;
  static constexpr int kItemUnits = 8;                   // 2: chunks and prompts took 4 and 6 % longer
  static constexpr bool kQueryMap = true;                // queries come by TMA
  static constexpr int kTile = D == 256 ? 64 : 128;      // keys per tile
  static constexpr int kWG = D == 256 ? 1 : 2;           // softmax warpgroups
  static constexpr int kDB = D / 64;                     // 64-dim blocks of a row
  static constexpr int kStageBytes = kTile * D * 2;
  static constexpr int kStages = D == 64 ? 8 : 5;
  static constexpr int kQBlock = 128 * 128;              // 128 rows x 64 dims
  static constexpr int kQBytes = kQBlock * kDB;
  // with the static arrays (3 KB, a multiple of the dynamic array's alignment) all of an SM's shared memory for d = 128
  static constexpr int kSmem = kWG * kQBytes + kStages * kStageBytes;
  static constexpr int kSoftmax = kWG * 128;             // softmax threads
  static constexpr int kThreads = kSoftmax + 128;
  static constexpr uint32_t kSCols = kTile;              // columns of one S slot (two slots)
};

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of two values on the FMA pipe, for x < 127: x = n + f with n the nearest integer, read off the low
// bits of x + 1.5 2^23, and 2^f on [-1/2, 1/2] by the cubic of least maximal relative error (7.5e-5, found by
// exchange; p is rounded to bf16, 3.9e-3).  What x = -126 and everything below it gives, kExp2Least, is taken off at the
// end: a masked key's weight has to be 0, because the value that it would bring along may be as large as bf16 goes.
constexpr float kCubic0 = 0.999928057f;
constexpr uint32_t kExp2Least = 0x007FFB49u;  // the bits of kCubic0, 126 off its exponent
__device__ __forceinline__ uint64_t exp2_cubic2(uint64_t x) {
  float a, b, na, nb;
  unpack2(x, a, b);
  x = pack2(fmaxf(a, -126.f), fmaxf(b, -126.f));
  const uint64_t magic = pack2(12582912.f, 12582912.f);
  const uint64_t t = add2(x, magic);
  const uint64_t n = add2(t, pack2(-12582912.f, -12582912.f));
  const uint64_t f = fma2(n, pack2(-1.f, -1.f), x);
  uint64_t y = fma2(f, pack2(0.0551716685f, 0.0551716685f), pack2(0.242611125f, 0.242611125f));
  y = fma2(y, f, pack2(0.693260968f, 0.693260968f));
  y = fma2(y, f, pack2(kCubic0, kCubic0));
  unpack2(y, a, b);
  unpack2(t, na, nb);
  const float least = __uint_as_float(kExp2Least | 0x80000000u);
  return add2(pack2(__uint_as_float(__float_as_uint(a) + (__float_as_uint(na) << 23)),
                    __uint_as_float(__float_as_uint(b) + (__float_as_uint(nb) << 23))),
              pack2(least, least));
}

// F32: fp32 outputs; TWO: P in two bf16 parts in every item, else in those that hold all of a sequence's new tokens.
template <int D, bool F32, bool TWO>
__global__ void __launch_bounds__(Pa<D>::kThreads, 1) paged_attn_kernel(const __grid_constant__ PaParams p) {
  using C = Pa<D>;
  constexpr int kTile = C::kTile, kWG = C::kWG, kDB = C::kDB, kNS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t q_full, q_empty, kv_full[kNS], kv_empty[kNS], edge_full[kNS], s_full[2], p_half[2],
      p_full[2], o_full[2], piece_full[kPaPieces], piece_empty[kPaPieces], wg_bar, drain;
  __shared__ Piece pieces[kPaPieces], late_piece;
  __shared__ uint32_t tmem_base_s, bad_s[kPaBadRing];
  __shared__ float ml_s[2][2][128];  // solo items: each warpgroup's maxima and sums
  __shared__ int dead_s, last_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedAttnArgs& a = p.a;

  asm volatile("griddepcontrol.launch_dependents;");  // the merge's blocks may come as CTAs leave
  if (tid == 0) {
    prefetch_tensormap(&p.q);
    prefetch_tensormap(&p.k);
    prefetch_tensormap(&p.v);
  }

  // ---- each sequence's length on the line (per KV head), into the ring, which is still empty
  int64_t* seq_units = reinterpret_cast<int64_t*>(smem_raw + kWG * C::kQBytes);
  line_lengths<C>(p, seq_units);
  if (tid == 0) {
    dead_s = 0;
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
      mbar_init(&edge_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kPaPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], C::kSoftmax / 32 + 3);
    }
    mbar_init(&wg_bar, C::kSoftmax);
    mbar_init(&drain, 1);
    fence_mbarrier_init();
  }
  constexpr int kMmaWarp = kWG * 4, kLoadWarp = kMmaWarp + 1, kZeroWarp = kMmaWarp + 2,
                kValueWarp = kMmaWarp + 3;
  if (warp == kMmaWarp) tmem_alloc(&tmem_base_s, kTmemCols);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const uint32_t base = smem_u32(smem_raw);
  const uint32_t q_s = base, kv_s = base + kWG * C::kQBytes;
  const Waiter wait{&dead_s, a.status};
  // The load warp walks the pieces and publishes them; every other warp takes them in order.
  auto take = [&](int k, bool* ok) -> const Piece& {
    *ok = __all_sync(0xFFFFFFFFu, wait(&piece_full[k % kPaPieces], (k / kPaPieces) & 1)) != 0;
    if (*ok && pieces[k % kPaPieces].t1 == 0) *ok = false;
    return pieces[k % kPaPieces];
  };
  auto all_ok = [&](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };
  auto release = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[k % kPaPieces]);
  };

  // Two softmax warpgroups at 200 registers and the other four warps at 104 make up the launch's 384 x 168
  // (208 and 88: chunks 2 % slower; the split stands at the head of each branch, where the compiler can use it).
  if (warp < kMmaWarp) {
    // ------------------------------------------------------------------ softmax and output
    if constexpr (kWG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int wg = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane, tr = r / p.G;
    const int rows_tile = p.tpt * p.G;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t s_par = 0, o_par = 0;    // phases of s_full and o_full, a bit per slot
    uint32_t tiles0 = 0, wg_par = 0;  // tiles before the piece
    bool ok = true;
    auto sync_wgs = [&]() {
      mbar_arrive(&wg_bar);
      const bool x = all_ok(wait(&wg_bar, wg_par));
      wg_par ^= 1;
      return x;
    };
    for (int piece = 0; ok; ++piece) {
      const Piece& s = take(piece, &ok);
      if (!ok) break;
      const bool solo = s.it.solo;
      [[maybe_unused]] const bool few = s.it.few;
      const int qoff = !solo && wg == 1 ? p.tpt : 0;
      const bool valid = r < rows_tile && qoff + tr < s.it.ntok;
      const bool active = __any_sync(0xFFFFFFFFu, valid);
      const int pos = s.it.pf + min(qoff + tr, s.it.ntok - 1), pl = s.it.pf + s.it.ntok - 1;
      // this row sees places [0, va) and [vb, vc) of the list; all rows see [b_max, c_min)
      const int W = a.window;
      const int va = W > 0 ? min(a.n_sinks, pos + 1) : 0;
      const int vb = (W > 0 ? max(0, pos + 1 - W) : 0) - s.it.shift, vc = pos + 1 - s.it.shift;
      const int b_max = (W > 0 ? max(0, pl + 1 - W) : 0) - s.it.shift, c_min = s.it.pf + 1 - s.it.shift;
      const bool split_keys = kWG == 2 && solo;
      const int o_slot = kWG == 2 ? wg : 0;
      float m = -INFINITY, l = 0.f;
      bool first = true;
      int prev = 0;  // slot of the tile before (with one warpgroup two products may be under way, hence a barrier each)
      for (int i = s.t0 + (split_keys ? wg : 0); i < s.t1; i += split_keys ? 2 : 1) {
        const int slot = kWG == 2 ? wg : ((i - s.t0) & 1);
        ok = all_ok(wait(&s_full[slot], (s_par >> slot) & 1));
        s_par ^= 1u << slot;
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t s_col = trow + slot * C::kSCols;
          const int v0 = i * kTile;
          const uint32_t bad = bad_s[(tiles0 + i - s.t0) % kPaBadRing];
          const bool masked = bad || v0 < b_max || v0 + kTile > c_min;
          float x[kTile];
          if constexpr (kTile == 128) tmem_ld128(s_col, x);
          else tmem_ld64(s_col, x);
          // 32 scores from column 32 c on, those that this row does not see at -infinity
          auto hide = [&](int c, float* y) {
            const int at = v0 + 32 * c;
            uint32_t w = bits_below(va - at) | (bits_below(vc - at) & ~bits_below(vb - at));
            if (bad)
              for (int k = 0; k < p.nbox; ++k)
                if ((bad >> (k * kDB)) & 1)
                  w &= ~(bits_below((k + 1) * p.box - 32 * c) & ~bits_below(k * p.box - 32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = (w >> e) & 1 ? y[e] : -INFINITY;
          };
          if (masked) {
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c) hide(c, x + 32 * c);
          }
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int e = 4; e < kTile; e += 8) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
              m4[f] = fmaxf(fmaxf(m4[f], x[e + f]), e + 4 + f < kTile ? x[e + 4 + f] : -INFINITY);
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const bool move = m == -INFINITY ? mx > -INFINITY : (mx - m) * p.scale_log2 > kPaRescale;
          if (__any_sync(0xFFFFFFFFu, move)) {
            float alpha = 1.f;
            if (move) {
              alpha = m == -INFINITY ? 0.f : exp2_approx((m - mx) * p.scale_log2);
              m = mx;
              l *= alpha;
            }
            if (!first) {  // the products before this tile have to be done; with two streams its scores came after them
              if constexpr (kWG == 1) {
                ok = all_ok(wait(&o_full[prev], ((o_par >> prev) & 1) ^ 1));
                if (!ok) break;
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                float v[32];
                tmem_ld32(trow + kPaOCol + o_slot * D + 32 * c, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= alpha;
                tmem_st32(trow + kPaOCol + o_slot * D + 32 * c, v);
              }
            }
          }
          const float mm = m == -INFINITY ? 0.f : m * p.scale_log2;
          const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), mm2 = pack2(-mm, -mm);
          uint64_t l2[2] = {0, 0};
          // P of 32 scores over the columns they come from: in the first 16, its remainder in the other 16
          auto weigh = [&](int c, const float* y, auto two_parts) {
            constexpr bool kTwo = decltype(two_parts)::value, kCubic = !kTwo && kWG == 2;
            uint32_t hi[16];
            [[maybe_unused]] uint32_t lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t z = fma2(pack2(y[2 * e], y[2 * e + 1]), scale2, mm2);
              float p0, p1;
              uint64_t pp;
              if (kCubic && e % kPaCubicEvery == kPaCubicEvery - 1) {
                pp = exp2_cubic2(z);
                unpack2(pp, p0, p1);
              } else {
                unpack2(z, p0, p1);
                p0 = exp2_approx(p0);
                p1 = exp2_approx(p1);
                pp = pack2(p0, p1);
              }
              l2[e & 1] = add2(l2[e & 1], pp);
              hi[e] = pack_bf16x2(p0, p1);
              if constexpr (kTwo)
                lo[e] =
                    pack_bf16x2(p0 - bf16_bits_to_float(hi[e] & 0xFFFFu), p1 - __uint_as_float(hi[e] & 0xFFFF0000u));
            }
            if (c == kTile / 64) {  // the first half of P is stored: its product can begin
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_half[slot]);
            }
            tmem_st16_nowait(s_col + 32 * c, hi);
            if constexpr (kTwo) tmem_st16_nowait(s_col + 32 * c + 16, lo);
          };
          if (!TWO && few) {  // rare beside prompts: the scores are read again, so that the other way keeps its registers
#pragma unroll 1
            for (int c = 0; c < kTile / 32; ++c) {
              float y[32];
              tmem_ld32(s_col + 32 * c, y);
              if (masked) hide(c, y);
              weigh(c, y, std::true_type{});
            }
          } else {
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c) weigh(c, x + 32 * c, std::bool_constant<TWO>{});
          }
          float la, lb;
          unpack2(add2(l2[0], l2[1]), la, lb);
          l += la + lb;
          tmem_st_wait();
        } else if (lane == 0) {
          mbar_arrive(&p_half[slot]);
        }
        first = false;
        if (kWG == 1) o_par ^= 1u << slot;
        prev = slot;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[slot]);
      }
      tiles0 += s.t1 - s.t0;
      if (!ok) break;
      if (!first) {
        if (kWG == 2) o_par ^= 1u << prev;  // once a piece
        ok = all_ok(wait(&o_full[prev], ((o_par >> prev) & 1) ^ 1));
        if (!ok) break;
      }
      if (m == -INFINITY) l = 0.f;
      // the row's factor on each accumulator that holds a share of it
      float f0 = 1.f, f1 = 0.f;
      if (split_keys) {
        ml_s[wg][0][r] = m;
        ml_s[wg][1][r] = l;
        ok = sync_wgs();
        if (!ok) break;
        const float m0 = ml_s[0][0][r], m1 = ml_s[1][0][r], l0 = ml_s[0][1][r], l1 = ml_s[1][1][r];
        m = fmaxf(m0, m1);
        f0 = l0 > 0.f ? exp2_approx((m0 - m) * p.scale_log2) : 0.f;
        f1 = l1 > 0.f ? exp2_approx((m1 - m) * p.scale_log2) : 0.f;
        l = f0 * l0 + f1 * l1;
      }
      tc_fence_after();
      const bool whole = s.c_first == s.c_last, tall = tall_item<C>(s.it, p.G);
      const int row = (solo ? 0 : wg * rows_tile) + r;  // within the item
      const int64_t orow = (s.q0 + row / p.G) * a.Hq + s.h * p.G + row % p.G;
      const int slot_out = 2 * static_cast<int>(blockIdx.x) + (static_cast<int>(blockIdx.x) == s.c_first ? 1 : 0);
      const int64_t prow = static_cast<int64_t>(slot_out) * a.rows_cap + row;
      if (active) {
        const float g = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        const int c0 = split_keys ? wg * (D / 64) : 0, c1 = split_keys ? c0 + D / 64 : D / 32;
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float v[32];
          if (split_keys) {
            float y[32];
            tmem_ld32(trow + kPaOCol + 32 * c, v);
            tmem_ld32(trow + kPaOCol + D + 32 * c, y);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (f0 != 0.f ? f0 * v[e] : 0.f) + (f1 != 0.f ? f1 * y[e] : 0.f);
          } else {
            tmem_ld32(trow + kPaOCol + o_slot * D + 32 * c, v);
          }
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= g;
            if (whole) store_out32<F32>(a.O, orow * D + 32 * c, v);
            else if (!tall) store_out32<true>(a.part_o, prow * D + 32 * c, v);
            else {  // word by word, the rows side by side
              float4* to = part_word(a, D, slot_out, 8 * c) + row;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                to[static_cast<int64_t>(e) * a.rows_cap] =
                    make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
          __syncwarp();
        }
        if (valid && !(split_keys && wg == 1)) {
          if (!whole) a.part_ml[prow] = make_float2(m, l);
          else if (a.lse) a.lse[orow] = l > 0.f ? m * a.sm_scale + logf(l) : -INFINITY;
        }
      }
      tc_fence_before();
      if (whole || tall) {
        if (split_keys) ok = sync_wgs();  // neither accumulator is overwritten before both have read it
        release(piece);
        continue;
      }
      // ---- the last CTA of a cut item merges its pieces (the barrier orders the warps' partials before
      // thread 0's fence, which orders them before its count)
      ok = sync_wgs();
      if (!ok) break;
      if (tid == 0) {
        const int n = s.c_last - s.c_first + 1;
        __threadfence();
        const bool last = atomicAdd(a.counters + s.c_first, 1) == n - 1;
        if (last) a.counters[s.c_first] = 0;
        __threadfence();
        last_s = last;
      }
      ok = sync_wgs();
      if (!ok) break;
      if (last_s) merge_pieces<C, F32>(p, s);
      release(piece);
    }
  } else {
    if constexpr (kWG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------------ pieces, Q and K
      const int box = lane / kDB, db = lane % kDB;
      const bool on = box < p.nbox;
      uint32_t st = 0, st_par = 1, used = 0, tiles = 0;  // the next stage, its phase before, stages in use; tiles begun
      bool ok = true;
      const Start at0 = line_start<C>(p, seq_units);
      __syncwarp();  // seq_units has been read; loads write there next
      fence_async_smem();
      Walk<C> walk(p, at0);
      // The rest of an item that an earlier CTA began comes last: the CTAs of a head then go through its
      // keys side by side, and find them in L2.
      bool late = false;
      if (lane == 0) a.cuts[blockIdx.x].pieces = 0;
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
            if (c.t1 > 0 && c.t0 == 0 && c.t1 < c.it.ntiles && tall_item<C>(c.it, p.G))
              a.cuts[blockIdx.x] = {c.q0, c.it.ntok * p.G, c.h, c.c_last - c.c_first + 1};
            pieces[at] = c;
            mbar_arrive(&piece_full[at]);
          }
          __syncwarp();
        }
        const Piece& s = pieces[at];
        if (s.t1 == 0) break;
        BoxWalk<C> bw(p, s, box);
        int pg_next = bw.page(p, s, on);
        if (piece > 0) ok = all_ok(wait(&q_empty, (piece - 1) & 1));
        if (!ok) break;
        const int nqt = s.it.solo ? 1 : 2;
        if (lane == 0) mbar_arrive_expect_tx(&q_full, nqt * kDB * p.tpt * p.G * 128);
        __syncwarp();
        if (lane < nqt * kDB)
          tma_load_3d(q_s + (lane / kDB) * C::kQBytes + db * C::kQBlock, &p.q, db * 64, s.h * p.G,
                      static_cast<int>(s.q0) + (lane / kDB) * p.tpt, &q_full);
        for (int i = s.t0; i < s.t1; ++i) {
          const int pg = pg_next, row = bw.row;
          bw.step(p, s.it);
          pg_next = i + 1 < s.t1 ? bw.page(p, s, on) : -2;  // the next tile's, while this one waits
          ok = all_ok(wait(&kv_empty[st], st_par));
          if (!ok) break;
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, pg == -1);
          const uint32_t loads = __popc(__ballot_sync(0xFFFFFFFFu, pg >= 0));
          if (lane == 0) {
            bad_s[tiles % kPaBadRing] = bad;
            if (bad) flag_error(a.status, DEVFLAG_BAD_INDEX);
            mbar_arrive_expect_tx(&kv_full[st], loads * p.box * 128);
          }
          __syncwarp();
          if (pg >= 0)
            tma_load_4d(kv_s + st * C::kStageBytes + db * (kTile * 128) + box * p.box * 128, &p.k, db * 64, row, s.h,
                        pg, &kv_full[st]);
          used |= 1u << st;
          st += 2;
          if (st >= kNS) st -= kNS, st_par ^= 1;
          ++tiles;
        }
      }
      if (dead_s && lane == 0) drain_copies(kv_full, kNS, used, a.status);  // Q: the MMA thread
    } else if (warp == kValueWarp) {
      // ------------------------------------------------------------------ V
      const int box = lane;
      const bool on = box < p.nbox;
      uint32_t st = 1, st_par = 1, used = 0;
      bool ok = true;
      const int armed = wait_test_armed(a);
      for (int piece = 0; ok; ++piece) {
        const Piece& s = take(piece, &ok);
        if (!ok) break;
        BoxWalk<C> bw(p, s, box);
        int pg_next = bw.page(p, s, on);
        for (int i = s.t0; i < s.t1; ++i) {
          const int pg = pg_next, row = bw.row;
          bw.step(p, s.it);
          pg_next = i + 1 < s.t1 ? bw.page(p, s, on) : -2;
          ok = all_ok(wait(&kv_empty[st], st_par));
          if (!ok) break;
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, pg == -1);
          const uint32_t loads = __popc(__ballot_sync(0xFFFFFFFFu, pg >= 0));
          uint64_t* bar = bad || edge_tile<C>(s.it, i) ? &edge_full[st] : &kv_full[st];
          if (lane == 0) mbar_arrive_expect_tx(bar, loads * p.box * (kDB * 128));
          __syncwarp();
          if (pg >= 0 && !(armed == 1 && used == 0))
            tma_load_5d(kv_s + st * C::kStageBytes + box * p.box * (kDB * 128), &p.v, 0, row, 0, s.h, pg, bar);
          used |= 1u << st;
          st += 2;
          if (st >= kNS) st -= kNS, st_par ^= 1;
        }
        if (ok) release(piece);
      }
      if (armed == 1) wait_test_disarm(a.status);
      if (dead_s && lane == 0) {  // V comes on either barrier of its stage
        drain_copies(kv_full, kNS, used, a.status);
        drain_copies(edge_full, kNS, used, a.status);
      }
    } else if (warp == kZeroWarp) {
      // ------------------------------------------------------------------ unseen V rows
      const bool on = lane < p.nbox;
      uint32_t st = 1, par = 0;  // the next V's stage; phase of each edge barrier
      bool ok = true;
      for (int piece = 0; ok; ++piece) {
        const Piece& s = take(piece, &ok);
        if (!ok) break;
        BoxWalk<C> bw(p, s, lane);
        int pg_next = bw.page(p, s, on);
        for (int i = s.t0; i < s.t1; ++i) {
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, pg_next == -1), here = st;
          bw.step(p, s.it);
          pg_next = i + 1 < s.t1 ? bw.page(p, s, on) : -2;
          st += 2;
          if (st >= kNS) st -= kNS;
          if (!bad && !edge_tile<C>(s.it, i)) continue;
          ok = all_ok(wait(&edge_full[here], (par >> here) & 1));
          if (!ok) break;
          par ^= 1u << here;
          for (int r = lane; r < kTile; r += 32) {
            const int v = i * kTile + r, box = r / p.box;
            if (((bad >> box) & 1) || v >= s.it.nv || (v >= s.it.z0 && v < s.it.z1)) {
              const uint32_t at = kv_s + here * C::kStageBytes + box * p.box * (kDB * 128) + (r - box * p.box) * 128;
#pragma unroll
              for (int x = 0; x < kDB * 8; ++x)
                st_shared_v4(at + (x >> 3) * p.box * 128 + (x & 7) * 16, 0, 0, 0, 0);
            }
          }
        fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[here]);
        }
        if (ok) release(piece);
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ MMAs
      if (lane == 0) {
        // One thread issues everything, so what it does between two MMAs is kept to a few instructions:
        // descriptors are a low word per stage plus constants, ring places are stepped, not computed.
        const uint32_t idesc_s = instr_desc(128, kTile, false, false);
        const uint32_t idesc_o = instr_desc(128, D, true, false);
        const uint32_t q_lo = (q_s >> 4) | (1u << 16);
        const uint32_t k_lo = (kv_s >> 4) | (1u << 16);
        // V lies box by box: 64-dim blocks a box apart, and a box's 16-key steps of all blocks before the next box's
        const uint32_t v_lo = (kv_s >> 4) | (static_cast<uint32_t>(p.box * 8) << 16);
        const int box_shift = 31 - __clz(p.box >> 4), box_skip = (kDB - 1) * p.box * 8;
        uint32_t p_par = 0;          // phases of p_full, a bit per slot
        // the ring holds K_0, V_0, K_1, V_1, ...: the next K's and the next V's stage and phase
        uint32_t ks = 0, k_par = 0, vs = 1, v_par = 0;
        bool ok = true;
        auto next_k = [&]() {
          ks += 2;
          if (ks >= kNS) ks -= kNS, k_par ^= 1;
        };
        auto next_v = [&]() {
          vs += 2;
          if (vs >= kNS) vs -= kNS, v_par ^= 1;
        };
        auto scores = [&](int slot, int qt, uint32_t stage) {
          const uint32_t qa = q_lo + qt * (C::kQBytes >> 4), ka = k_lo + stage * (C::kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_lo(tmem + slot * C::kSCols, qa + (kk >> 2) * (C::kQBlock >> 4) + (kk & 3) * 2,
                         ka + (kk >> 2) * (kTile * 128 >> 4) + (kk & 3) * 2, idesc_s, kk != 0);
        };
        // the steps k0 <= kt < k1 of the product of one part of P with V
        auto product = [&](int slot, int o, uint32_t stage, bool first, int k0, int k1, int part) {
          const uint32_t va = v_lo + stage * (C::kStageBytes >> 4);
#pragma unroll
          for (int kt = k0; kt < k1; ++kt)
            umma_bf16_ts_lo(tmem + kPaOCol + o * D,
                            tmem + slot * C::kSCols + (kt >> 1) * 32 + part * 16 + (kt & 1) * 8,
                            va + kt * (2048 >> 4) + (kt >> box_shift) * box_skip, idesc_o, part || kt ? 1u : !first);
        };
        auto values = [&](int slot, int o, uint32_t stage, bool first, int k0, int k1) {
          product(slot, o, stage, first, k0, k1, 0);
          if constexpr (TWO) product(slot, o, stage, first, k0, k1, 1);
        };
        for (int piece = 0; ok; ++piece) {
          const int at = piece % kPaPieces;
          ok = wait(&piece_full[at], (piece / kPaPieces) & 1);
          if (!ok || pieces[at].t1 == 0) break;
          const int n = pieces[at].t1 - pieces[at].t0;
          const bool pair = !pieces[at].it.solo;
          [[maybe_unused]] const bool few = pieces[at].it.few;
          mbar_arrive(&piece_empty[at]);
          ok = wait(&q_full, piece & 1) && wait(&kv_full[ks], k_par);
          if (!ok) break;
          tc_fence_after();
          scores(0, 0, ks);
          umma_commit(&s_full[0]);
          if (pair) {
            scores(1, 1, ks);
            umma_commit(&s_full[1]);
          }
          umma_commit(&kv_empty[ks]);
          if (n == 1) umma_commit(&q_empty);
          next_k();
          if (pair) {
            // a stream's next scores follow its product, so s_full tells its warps too that the product is done
            for (int i = 0; i < n; ++i) {
              const bool more = i + 1 < n;
              ok = wait(&kv_full[vs], v_par) && wait(&p_half[0], p_par & 1);
              if (!ok) break;
              tc_fence_after();
              values(0, 0, vs, i == 0, 0, kTile / 32);
              ok = wait(&p_full[0], p_par & 1);
              if (!ok) break;
              tc_fence_after();
              values(0, 0, vs, false, kTile / 32, kTile / 16);
              if (more) {
                ok = wait(&kv_full[ks], k_par);
                if (!ok) break;
                scores(0, 0, ks);
                umma_commit(&s_full[0]);
              } else {
                umma_commit(&o_full[0]);
              }
              ok = wait(&p_half[1], p_par >> 1);
              if (!ok) break;
              tc_fence_after();
              values(1, 1, vs, i == 0, 0, kTile / 32);
              ok = wait(&p_full[1], p_par >> 1);
              if (!ok) break;
              tc_fence_after();
              values(1, 1, vs, false, kTile / 32, kTile / 16);
              umma_commit(&kv_empty[vs]);
              next_v();
              if (more) {
                scores(1, 1, ks);
                umma_commit(&s_full[1]);
                umma_commit(&kv_empty[ks]);
                if (i + 2 == n) umma_commit(&q_empty);
                next_k();
              } else {
                umma_commit(&o_full[1]);
              }
              p_par ^= 3;
            }
          } else {
            // tiles take turns with the slots
            if (n > 1) {
              ok = wait(&kv_full[ks], k_par);
              if (!ok) break;
              scores(1, 0, ks);
              umma_commit(&s_full[1]);
              umma_commit(&kv_empty[ks]);
              if (n == 2) umma_commit(&q_empty);
              next_k();
            }
            for (int i = 0; i < n; ++i) {
              const int slot = i & 1, o = kWG == 2 ? slot : 0;
              const bool more = i + 2 < n;
              ok = wait(&kv_full[vs], v_par) && wait(&p_full[slot], (p_par >> slot) & 1);
              if (!ok) break;
              p_par ^= 1u << slot;
              tc_fence_after();
              values(slot, o, vs, i == 0 || (kWG == 2 && i == 1), 0, kTile / 16);
              if constexpr (!TWO)
                if (few) product(slot, o, vs, false, 0, kTile / 16, 1);
              umma_commit(&kv_empty[vs]);
              if (kWG == 1 || !more) umma_commit(&o_full[slot]);
              next_v();
              if (more) {
                ok = wait(&kv_full[ks], k_par);
                if (!ok) break;
                scores(slot, 0, ks);
                umma_commit(&kv_empty[ks]);
                if (i + 3 == n) umma_commit(&q_empty);
                umma_commit(&s_full[slot]);
                next_k();
              }
            }
          }
        }
        umma_commit(&drain);  // every MMA and commit before it, in the error case too
        mbar_wait_bounded(&drain, 0, a.status);
        if (dead_s) drain_copies(&q_full, 1, 1, a.status);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merges the cut items of many rows.  A block takes 32 rows and 32 columns of one; a thread takes one 16-byte word
// of a row, four pieces' loads under way at once, in the order of the pieces.
template <int D, bool F32>
__global__ void __launch_bounds__(256, 5) paged_merge_kernel(PagedAttnArgs a, int G, float scale_log2) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention's launch is complete
  const PagedCut cut = a.cuts[blockIdx.x];
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), word = blockIdx.z * 8 + (threadIdx.x >> 5);
  if (cut.pieces == 0 || row >= cut.rows) return;
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kParts = 4;
  for (int k0 = 0; k0 < cut.pieces; k0 += kParts) {
    float2 ml[kParts];
    float4 v[kParts];
#pragma unroll
    for (int y = 0; y < kParts; ++y) {
      ml[y] = make_float2(-INFINITY, 0.f);
      v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + y >= cut.pieces) continue;
      // an item's first piece is the last of its CTA, the others the first of theirs
      const int slot = 2 * (static_cast<int>(blockIdx.x) + k0 + y) + (k0 + y == 0 ? 1 : 0);
      ml[y] = __ldcg(a.part_ml + static_cast<int64_t>(slot) * a.rows_cap + row);
      v[y] = __ldcg(part_word(a, D, slot, word) + row);
    }
    float mn = M;
#pragma unroll
    for (int y = 0; y < kParts; ++y) mn = fmaxf(mn, ml[y].x);
    const float z = mn == -INFINITY ? 0.f : mn * scale_log2;
    const float w = exp2_approx(fmaf(M, scale_log2, -z));
    M = mn;
    L *= w;
    o.x *= w, o.y *= w, o.z *= w, o.w *= w;
#pragma unroll
    for (int y = 0; y < kParts; ++y) {
      const float u = exp2_approx(fmaf(ml[y].x, scale_log2, -z));
      L = fmaf(u, ml[y].y, L);
      o.x = fmaf(u, v[y].x, o.x), o.y = fmaf(u, v[y].y, o.y), o.z = fmaf(u, v[y].z, o.z), o.w = fmaf(u, v[y].w, o.w);
    }
  }
  const float g = L > 0.f ? 1.f / L : 0.f;
  const int64_t to = (cut.q0 + row / G) * a.Hq + cut.h * G + row % G;
  if constexpr (F32)
    reinterpret_cast<float4*>(static_cast<float*>(a.O) + to * D)[word] =
        make_float4(o.x * g, o.y * g, o.z * g, o.w * g);
  else
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + to * D)[word] =
        make_uint2(pack_bf16x2(o.x * g, o.y * g), pack_bf16x2(o.z * g, o.w * g));
  if (word == 0 && a.lse) a.lse[to] = L > 0.f ? M * a.sm_scale + logf(L) : -INFINITY;
}

// ------------------------------------------------------------------ host
template <int D, bool F32, bool TWO>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  using C = Pa<D>;
  PaParams p;
  if (!paged_params<C>(a, paged_attn_tile_tokens(a.Hq / a.pool.Hkv), &p)) return cudaErrorInvalidValue;
  auto kernel = paged_attn_kernel<D, F32, TWO>;
  static int done[64] = {0};
  const cudaError_t e = set_smem_limit_once(kernel, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const cudaError_t e2 = launch_ex(kernel, dim3(num_sms), dim3(C::kThreads), C::kSmem, s, 0, p);
  // rows that an item may have (tall_item)
  const int64_t rows = static_cast<int64_t>(a.max_q_len) * p.G;
  if (e2 != cudaSuccess || rows <= (C::kWG == 1 ? 32 : p.tpt * p.G)) return e2;
  const dim3 blocks(num_sms, (a.rows_cap + 31) / 32, D / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, F32>, a, p.G, p.scale_log2);
}

// Where no sequence can have more than 128 rows per KV head, a kernel of its own has nothing but the two-part form: 8
// tokens of 8-head groups over 16 caches of 12K, d = 64: 47.5 us, 52.4 in the one that has both; of 4-head groups over 8
// caches of 5K, d = 128: 53.2 and 55.1.  P, and so the result's precision, is the same in either.
template <int D>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  const bool two = static_cast<int64_t>(a.max_q_len) * (a.Hq / a.pool.Hkv) <= 128;
  if (!a.out_bf16) return launch<D, true, true>(a, num_sms, s);
  return two ? launch<D, false, true>(a, num_sms, s) : launch<D, false, false>(a, num_sms, s);
}

}  // namespace

int paged_attn_tile_tokens(int G) { return 128 / G; }

int paged_attn_rows(int d, int G, int64_t max_q_len) {
  const int64_t item = static_cast<int64_t>(paged_attn_tile_tokens(G)) * (d == 256 ? 1 : 2);
  return static_cast<int>(min64(item, max_q_len)) * G;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int num_sms, cudaStream_t s) {
  switch (a.pool.d) {
    case 64: return launch<64>(a, num_sms, s);
    case 128: return launch<128>(a, num_sms, s);
    case 256: return launch<256>(a, num_sms, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace jssa
