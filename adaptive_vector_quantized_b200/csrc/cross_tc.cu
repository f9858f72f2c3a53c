// Exact attention over another sequence on the tensor cores (bf16).
//
//   S = scale Q K^T,  P = exp(S - m),  O = P V / sum(P),
// in one pass over the keys with a running maximum and sum (fp32).
//
// A block works on pairs of 128-row tiles of one head; both tiles share every
// K and V tile that TMA brings through a ring in shared memory.  One warp loads,
// one clears V's rows of keys that are left out, two issue the MMAs of a tile
// each, two groups of four warps do the softmax, a row to a
// thread.  S and O stay in TMEM; P overwrites its S there (bf16, two to a
// column) and is the first operand of P V straight from TMEM.
//
// A softmax step takes 64 keys, half a key tile, and S has a buffer for each
// half: S of the next step is formed while this one is exponentiated.  With
// steps of 128 keys S would have to wait for P V of the same tile (TMEM has no
// room for a second buffer at d = 128); 16384 x 16384, 8 heads of 128: 1.36 ms
// like that, 1.03 ms in halves, although a product with 64 columns takes 48
// clocks of shared memory reads instead of 32.  With the last round's items split
// over the keys 0.91 ms (1.21 PFLOP/s; captured, in bursts: run for seconds the power
// cap makes it 1.05).
//
// The accumulator is rescaled only when a row's maximum has grown by more than
// 2^8 since the scale in use (P then stays below 2^8, and its rounding to bf16
// is relative): rare after the first tiles, so the groups do it themselves.
//
// Bound by the exponentials at d = 64 (16 a clock and SM), by them and the
// tensor pipe alike at d = 128; so a quarter of them go to the FMA pipe
// (fm::exp2_poly2, 7.5e-5 relative, a fiftieth of P's rounding).  Scores that are
// not finite go by the row's maximum, not by that exponential.
#include "cross_tc.cuh"

namespace avq {

namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps;  // and the next: one for each tile of a pair
constexpr int kLoadWarp = kMmaWarp + 2, kCleanWarp = kLoadWarp + 1;
constexpr int kThreads = 384;  // three warpgroups
// Registers per thread: 168 at launch (64512 in all), then 216 for the softmax
// groups, whose threads hold a row's 64 scores and as many of their results, and 72
// for the third (2 * 216 + 72 = 3 * 168).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;

template <int D>
struct Smem {
  static constexpr int kBlocks = D / 64;                      // 64-column blocks of a tile
  static constexpr int kTileBytes = kRowTile * D * 2;
  static constexpr int kQBufs = D == 64 ? 2 : 1;              // the next item's Q while this one's is in use
  // Ring of units: V of a key tile and K of the one after it (of the next item
  // after an item's last), which are used together.
  static constexpr int kUnits = D == 64 ? 3 : 2;
  static constexpr int kUnitBytes = 2 * kTileBytes;           // V | K
  static constexpr int kQ = 0;                                // [kQBufs][2] tiles
  static constexpr int kRing = kQ + kQBufs * 2 * kTileBytes;
  static constexpr int kOut = kRing + kUnits * kUnitBytes;    // [8 warps][32 rows][64 columns]
  static constexpr int kBar = kOut + kSoftmaxWarps * 4096;
  // full[units], empty[units], ready[units], q_full[bufs][2], q_empty[bufs], s_full[2][2], p_ready[2][2], o_full[2],
  // tail[2], drain[2]
  static constexpr int kBars = 3 * kUnits + 3 * kQBufs + 14;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kTotal = kMisc + 16;
};

struct Maps {
  CUtensorMap q, k, v, o;
};

constexpr int kStep = 64;  // keys of a softmax step: half a key tile

// One item: a pair of row tiles of a head and a range of key tiles.
struct Item {
  int b, h, kb, kh, row0, tiles, count, t0, t1, parts;
};

__device__ __forceinline__ Item item_of(const CrossArgs& a, int i, int pairs) {
  Item x;
  const Part part = part_of(a, i);
  x.parts = part.parts;
  const int bh = part.item / pairs, pair = part.item - bh * pairs;
  x.b = bh / a.Hq;
  x.h = bh - x.b * a.Hq;
  x.kb = x.b / a.per_b;
  x.kh = x.h / a.per_h;
  x.row0 = pair * 2 * kRowTile;
  x.tiles = x.row0 + kRowTile < a.Nq ? 2 : 1;
  x.count = key_count(a, x.kb);
  const int kt = (x.count + kKeyTile - 1) / kKeyTile;
  x.t0 = part_begin(kt, part.split, part.parts);
  x.t1 = part_begin(kt, part.split + 1, part.parts);
  return x;
}

// exp2 of 32 scores (fp32 in r) as c2 * s - base, packed to bf16 in out[16];
// the sum of the unrounded values is added to `sum`.
template <bool kMasked>
__device__ __forceinline__ void exp_chunk(const uint32_t* r, float2 c2, float2 nbase, uint32_t* out, float2* sum) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float2 s = fm::f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    float2 x = fm::fma2(s, c2, nbase);
    // a step with keys left out (their scores -inf) keeps the exact zero of exp2(-inf)
    const bool poly = !kMasked && (i & 3) == 3;
    const float2 e = poly ? fm::exp2_poly2(x) : fm::f2(tc::ex2(x.x), tc::ex2(x.y));
    sum[i & 1] = fm::add2(sum[i & 1], e);
    out[i] = pack_bf16x2(e.x, e.y);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_tc_kernel(const __grid_constant__ Maps maps, const CrossArgs a,
                                                              unsigned int* err, int items, int pairs) {
  using S = Smem<D>;
  constexpr int KB = S::kBlocks;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBar);
  uint64_t* empty = full + S::kUnits;
  uint64_t* ready = empty + S::kUnits;
  uint64_t* q_full = ready + S::kUnits;
  uint64_t* q_empty = q_full + 2 * S::kQBufs;
  uint64_t* s_full = q_empty + S::kQBufs;
  uint64_t* p_ready = s_full + 4;  // both [tile][half of the key tile]
  uint64_t* o_full = p_ready + 4;
  uint64_t* tail = o_full + 2;  // P V of the step before an item's last
  uint64_t* drain = tail + 2;
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + S::kMisc);
  int* sAbort = reinterpret_cast<int*>(sm + S::kMisc + 4);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kBars; ++i) {
      uint64_t* b = full + i;
      const bool both = (b >= empty && b < ready) || (b >= q_empty && b < s_full);  // the two MMA warps
      tc::mbar_init(b, b >= p_ready && b < o_full ? 4 : both ? 2 : 1);
    }
    tc::fence_mbar_init();
    *sAbort = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(sTmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  grid_dependency_wait();  // the inputs, and whoever still reads the outputs
  const Guard guard{err, sAbort};
  const uint32_t tmem = *sTmem;
  // columns: S of each tile, the halves of a key tile apart | O0 | O1
  auto tS = [&](int t, int half) { return tmem + t * (2 * kStep) + half * kStep; };
  auto tO = [&](int t) { return tmem + 4 * kStep + t * D; };

  if (warp >= kSoftmaxWarps) {
    tc::regs_give<kOtherRegs>();
    if (warp == kLoadWarp) {
      if (lane == 0) {
        uint32_t g = 0, q = 0;  // units, items' Q loaded so far
        bool ok = true;
        auto load = [&](uint8_t* dst, const CUtensorMap* map, const Strides& st, int row, int h, int b, uint64_t* bar) {
#pragma unroll
          for (int c = 0; c < KB; ++c)
            tc::tma_load_4d(dst + c * kKeyTile * 128, map, c * 64, row, st.h != 0 ? h : 0, st.b != 0 ? b : 0, bar);
        };
        // a unit: V of tile jv of item v (none if v is null), then K of tile jk of item k;
        // the Q of an item goes ahead of its first K
        auto load_unit = [&](const Item* v, int jv, const Item* k, int jk) {
          const int slot = g % S::kUnits;
          if (!guard.wait(empty + slot, (g / S::kUnits & 1) ^ 1)) return false;
          uint8_t* dst = sm + S::kRing + slot * S::kUnitBytes;
          const int tiles = (v != nullptr) + (k != nullptr);
          tc::mbar_arrive_expect_tx(full + slot, tiles * S::kTileBytes);
          ++g;
          if (v != nullptr) load(dst, &maps.v, a.vs, jv * kKeyTile, v->kh, v->kb, full + slot);
          if (k == nullptr) return true;
          const bool fresh = jk == k->t0;
          bool got = true;
          if (fresh) {
            const int buf = q % S::kQBufs;
            got = guard.wait(q_empty + buf, (q / S::kQBufs & 1) ^ 1);
            if (got) {
              uint8_t* qd = sm + S::kQ + buf * 2 * S::kTileBytes;
              for (int t = 0; t < 2; ++t) {
                uint64_t* bar = q_full + 2 * buf + t;
                if (t < k->tiles) {
                  tc::mbar_arrive_expect_tx(bar, S::kTileBytes);
                  load(qd + t * S::kTileBytes, &maps.q, a.qs, k->row0 + t * kRowTile, k->h, k->b, bar);
                } else {
                  tc::mbar_arrive(bar);  // keeps the phases alike
                }
              }
              ++q;
            }
          }
          // also after a wait that ran out: the unit's bytes are awaited at the end
          load(dst + S::kTileBytes, &maps.k, a.ks, jk * kKeyTile, k->kh, k->kb, full + slot);
          return got;
        };
        Item last{};
        bool have = false;
        for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
          const Item x = item_of(a, i, pairs);
          if (x.t0 >= x.t1) continue;
          ok = load_unit(have ? &last : nullptr, last.t1 - 1, &x, x.t0);
          for (int j = x.t0; j + 1 < x.t1 && ok; ++j) ok = load_unit(&x, j, &x, j + 1);
          last = x;
          have = true;
        }
        if (have && ok) load_unit(&last, last.t1 - 1, nullptr, 0);
        // nothing of this block's copies may be in flight when it ends
        for (uint32_t k = g > S::kUnits ? g - S::kUnits : 0; k < g; ++k)
          tc::mbar_wait(full + k % S::kUnits, k / S::kUnits & 1, 1000000ull);
        for (uint32_t k = q > S::kQBufs ? q - S::kQBufs : 0; k < q; ++k)
          for (int t = 0; t < 2; ++t)
            tc::mbar_wait(q_full + 2 * (k % S::kQBufs) + t, k / S::kQBufs & 1, 1000000ull);
      }
    } else if (warp == kCleanWarp) {
      // V's rows of keys that are left out become zeros before the MMA warps read them
      uint32_t g = 0;
      auto pass = [&](const Item* x, int j) {  // the unit with V of tile j of item x (none if null)
        const uint32_t slot = g % S::kUnits;
        if (!wait_warp(guard, full + slot, g / S::kUnits & 1)) return false;
        ++g;
        if (x != nullptr && !tile_full(a, j * kKeyTile, x->count))
          clear_rows<D>(sm + S::kRing + slot * S::kUnitBytes, key_bits(a, x->kb, j * kKeyTile, x->count, lane),
                        min((x->count - j * kKeyTile + 15) & ~15, a.Nk - j * kKeyTile), lane);
        if (lane == 0) tc::mbar_arrive(ready + slot);
        return true;
      };
      Item last{};
      bool have = false, ok = true;
      for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
        const Item x = item_of(a, i, pairs);
        if (x.t0 >= x.t1) continue;
        ok = pass(have ? &last : nullptr, last.t1 - 1);
        for (int j = x.t0; j + 1 < x.t1 && ok; ++j) ok = pass(&x, j);
        last = x;
        have = true;
      }
      if (have && ok) pass(&last, last.t1 - 1);
    } else {
      // One warp issues the MMAs of one tile of the pairs.  A turn of the loop
      // takes a unit of the ring: by halves, P V of the key tile `cur` and behind
      // it S of the tile `next`, into the same half of S.  So S is there a step
      // ahead of the softmax.  The pipe holds only a few MMAs: whatever else the
      // thread does between them must be little, and falls to the other tile's.
      const int t = warp - kMmaWarp;
      const uint64_t ring = tc::sdesc_sw128(tc::smem_u32(sm + S::kRing), kKeyTile * 128, 1024);
      const uint64_t ring_k = tc::sdesc_sw128(tc::smem_u32(sm + S::kRing + S::kTileBytes), 16, 1024);
      const uint64_t qtile = tc::sdesc_sw128(tc::smem_u32(sm + S::kQ + t * S::kTileBytes), 16, 1024);
      constexpr uint32_t kUnit16 = S::kUnitBytes >> 4, kTile16 = S::kTileBytes >> 4, kHalf16 = kStep * 128 >> 4;
      constexpr uint32_t idesc_o = tc::idesc_bf16(kRowTile, D, 0, 1);
      const uint32_t o = tO(t);
      uint64_t *my_s = s_full + 2 * t, *my_p = p_ready + 2 * t;
      int i = blockIdx.x, j = 0, t0 = 0, t1 = 0, count = 0, left = 0;  // `next`: its item and keys
      bool on = false, more;                                          // the pair has this tile
      auto settle = [&] {                                             // the first tile at or after item i
        for (; i < items; i += gridDim.x) {
          const Item x = item_of(a, i, pairs);
          t0 = j = uniform(x.t0);
          t1 = uniform(x.t1);
          count = uniform(x.count);
          on = t < x.tiles;
          left = min(kKeyTile, count - j * kKeyTile);
          if (t0 < t1) return true;
        }
        return false;
      };
      more = settle();
      int cur_left = 0;  // of `cur`: 0 before the first
      bool cur_on = false, cur_last = false;
      uint32_t add = 0, slot = 0, phase = 0, buf = 0, q_phase = 0, p_phase = 0;  // p_phase: bit h for half h
      bool ok = true;
      while (cur_left > 0 || more) {
        ok = wait_all(guard, ready + slot, phase);
        if (!ok) break;
        const bool fresh = j == t0, next_on = more && on, next_last = j + 1 == t1;
        if (next_on && fresh) ok = wait_all(guard, q_full + 2 * buf + t, q_phase);
        if (!ok) break;
        const uint64_t vd = ring + slot * kUnit16, kd = ring_k + slot * kUnit16, qd = qtile + buf * 2 * kTile16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t s = tS(t, half);
          if (cur_on && cur_left > half * kStep) {
            ok = wait_all(guard, my_p + half, p_phase >> half & 1);
            if (!ok) break;
            p_phase ^= 1u << half;
            tc::tc_fence_after();
            if (tc::elect_one()) {
              if (cur_left >= (half + 1) * kStep) {
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k)
                  tc::mma_bf16_ts(o, s + k * 8, vd + half * kHalf16 + k * (2048 >> 4), idesc_o,
                                  half > 0 || k > 0 ? 1 : add);
              } else {
                for (int k = 0; k * 16 < cur_left - half * kStep; ++k)
                  tc::mma_bf16_ts(o, s + k * 8, vd + half * kHalf16 + k * (2048 >> 4), idesc_o,
                                  half > 0 || k > 0 ? 1 : add);
              }
              if (cur_last && cur_left <= (half + 1) * kStep) {
                tc::mma_commit(o_full + t);
              } else if (half == 0 ? cur_last : next_on && !fresh && next_last && left <= kStep) {
                tc::mma_commit(tail + t);
              }
            }
          }
          if (next_on && left > half * kStep) {
            const uint32_t idesc =
                left >= (half + 1) * kStep
                    ? tc::idesc_bf16(kRowTile, kStep, 0, 0)
                    : tc::idesc_bf16(kRowTile, 0, 0, 0) + (uint32_t)((left - half * kStep + 15) >> 4 << 1 << 17);
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const int off = ((k >> 2) * (kRowTile * 128) + (k & 3) * 32) >> 4;
                tc::mma_bf16(s, qd + off, kd + half * kHalf16 + off, idesc, k > 0);
              }
              tc::mma_commit(my_s + half);
            }
          }
        }
        if (!ok) break;
        if (tc::elect_one()) tc::mma_commit(empty + slot);
        if (++slot == S::kUnits) {
          slot = 0;
          phase ^= 1;
        }
        cur_left = more ? left : 0;
        cur_on = next_on;
        cur_last = next_last;
        add = !fresh;
        if (more) {
          ++j;
          left = min(kKeyTile, count - j * kKeyTile);
          if (j == t1) {
            if (tc::elect_one()) tc::mma_commit(q_empty + buf);
            if (++buf == S::kQBufs) {
              buf = 0;
              q_phase ^= 1;
            }
            i += gridDim.x;
            more = settle();
          }
        }
      }
      // every MMA done before TMEM is given back
      if (tc::elect_one()) tc::mma_commit(drain + t);
      __syncwarp();
      tc::mbar_wait(drain + t, 0, 1000000ull);
    }
  } else {
    tc::regs_take<kSoftmaxRegs>();
    const int t = warp >> 2;  // the group's tile of the pair
    const int quarter = warp & 3;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int row = quarter * 32 + lane;
    uint8_t* out = sm + S::kOut + warp * 4096;
    const float c2f = a.scale * kLog2e;
    const float2 c2 = fm::f2(c2f, c2f);
    uint32_t s_phase = 0, tail_phase = 0, o_phase = 0;  // s_phase: bit h for half h
    bool ok = true;
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
      const Item x = item_of(a, i, pairs);
      if (t >= x.tiles) continue;
      const int r0 = x.row0 + t * kRowTile;
      const size_t grow = ((size_t)x.b * a.Hq + x.h) * a.Nq + r0 + row;
      const bool live = r0 + row < a.Nq;
      float m = -INFINITY;  // maximum behind the scale in use
      float2 sum[2] = {fm::f2(0.f, 0.f), fm::f2(0.f, 0.f)};
      const int first = x.t0 * kKeyTile, end = min(x.t1 * kKeyTile, x.count);
      for (int k0 = first, half = 0; k0 < end; k0 += kStep, half ^= 1) {
        const bool whole = a.key_mask == nullptr && k0 + kStep <= x.count;
        uint32_t bits[2];
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            bits[c] = __ballot_sync(0xffffffffu, key_seen(a, x.kb, k0 + 32 * c + lane, x.count));
        }
        const uint32_t sS = tS(t, half) + lane_off;
        ok = wait_warp(guard, s_full + 2 * t + half, s_phase >> half & 1);
        if (!ok) break;
        s_phase ^= 1u << half;
        tc::tc_fence_after();
        const bool upper = whole || k0 + 32 < end;  // the last step may have keys in its first 32 columns alone
        uint32_t r[kStep];
        tc::tmem_ld32(sS, r);
        if (upper) tc::tmem_ld32(sS + 32, r + 32);
        tc::tmem_wait_ld();
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (bits[c] != 0xffffffffu) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(bits[c] >> k & 1u)) r[c * 32 + k] = 0xff800000u;  // whatever stands there
            }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < kStep; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top[e] = fm::max3_nan(top[e], __uint_as_float(r[k + 2 * e]), __uint_as_float(r[k + 2 * e + 1]));
        const float step_top = fm::max3_nan(fm::max3_nan(top[0], top[1], top[2]), top[3], top[3]);
        if (k0 == first) {
          m = step_top;
        } else {
          // NaN counts as grown: it must reach the output
          const bool grown = step_top != -INFINITY && !((step_top - m) * c2f <= 8.f);
          if (__any_sync(0xffffffffu, grown)) {
            // P V of the step before must have been added.  It is ahead of the next
            // step's S in the pipe, and of `tail` when this step is the item's last.
            if (k0 + kStep < end) ok = wait_warp(guard, s_full + 2 * t + (half ^ 1), s_phase >> (half ^ 1) & 1);
            else ok = wait_warp(guard, tail + t, tail_phase);
            if (!ok) break;
            tc::tc_fence_after();
            const float keep = grown ? exp2f((m - step_top) * c2f) : 1.f;
            const float2 keep2 = fm::f2(keep, keep);
            if (grown) m = step_top;
            sum[0] = fm::mul2(sum[0], keep2);
            sum[1] = fm::mul2(sum[1], keep2);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tc::tmem_ld16(tO(t) + lane_off + c * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
              tc::tmem_st16(tO(t) + lane_off + c * 16, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m * c2f;
        const float2 nbase = fm::f2(-base, -base);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
          if (whole) {
            exp_chunk<false>(r + c * 32, c2, nbase, p, sum);
          } else {
            if (c == 1 && !upper) break;
            exp_chunk<true>(r + c * 32, c2, nbase, p, sum);
          }
          tc::tmem_st16(sS + c * 16, p);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_ready + 2 * t + half);
      }
      if (!ok) break;
      if (end - first > kStep) tail_phase ^= 1;
      float z = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      // The FMA pipe's exponential is 2^-126 at least, and hides a NaN.  A NaN score
      // is in the sum all the same (the whole row's exponents are NaN then); what is
      // left are a score of +inf, whose row is NaN, and rows of -inf alone.
      if (m == INFINITY) z = NAN;
      if (m == -INFINITY) z = 0.f;
      const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : z);
      const float lse = z == 0.f ? -INFINITY : a.scale * m + logf(z);
      const bool any = x.t0 < x.t1;
      if (any) {
        ok = wait_warp(guard, o_full + t, o_phase);
        if (!ok) break;
        o_phase ^= 1;
        tc::tc_fence_after();
      }
      const size_t prow = (size_t)(i - a.whole) * (2 * kRowTile) + t * kRowTile + row;  // of a partial result
      if (live) {
        if (x.parts > 1) a.part_lse[prow] = lse;
        else if (a.lse != nullptr) a.lse[grow] = lse;
      }
      if (x.parts > 1) {
        // partial results stay in fp32: a row to a thread, straight to memory
        float* dst = a.part + prow * D;
        if (any) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tc::tmem_ld16(tO(t) + lane_off + c * 16, o);
            tc::tmem_wait_ld();
            if (live) {
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<float4*>(dst + c * 16 + k) =
                    make_float4(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv,
                                __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
            }
          }
        }
        tc::tc_fence_before();
        continue;
      }
#pragma unroll
      for (int cb = 0; cb < KB; ++cb) {
        if (lane == 0) tc::bulk_wait_group_read0();  // the staging rows are free again
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          if (any) {
            tc::tmem_ld32(tO(t) + lane_off + cb * 64 + c * 32, o);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 v;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(o[k * 8 + 2 * e]) * inv, __uint_as_float(o[k * 8 + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(out + lane * 128 + (((c * 4 + k) ^ (lane & 7)) << 4)) = v;
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (r0 + quarter * 32 < a.Nq)
            tc::tma_store_4d(&maps.o, out, cb * 64, r0 + quarter * 32, a.os.h != 0 ? x.h : 0, a.os.b != 0 ? x.b : 0);
          tc::bulk_commit_group();
        }
      }
      tc::tc_fence_before();  // O is read before the arrival that lets the next item write it
    }
    if (lane == 0) tc::bulk_wait_group0();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t run(const CrossArgs& a, unsigned int* err, cudaStream_t st, LaunchLog& log) {
  Maps m;
  cudaError_t e = make_tmap_view_bf16(&m.q, a.Q, a.qs, a.B, a.Hq, a.Nq, D, kRowTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.k, a.K, a.ks, a.Bk, a.Hk, a.Nk, D, kKeyTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.v, a.V, a.vs, a.Bk, a.Hk, a.Nk, D, kKeyTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.o, a.O, a.os, a.B, a.Hq, a.Nq, D, 32);
  if (e != cudaSuccess) return e;
  constexpr int smem = Smem<D>::kTotal + 1024;
  e = allow_smem<cross_tc_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  const int pairs = (a.Nq + 2 * kRowTile - 1) / (2 * kRowTile);
  const int items = a.B * a.Hq * pairs;
  const int launch = a.whole + (items - a.whole) * a.splits;
  const int grid = launch < num_sms() ? launch : num_sms();
  e = launch_after(cross_tc_kernel<D>, dim3(grid), dim3(kThreads), smem, st, m, a, err, launch, pairs);
  if (e == cudaSuccess && a.whole < items) e = launch_cross_join_items(a, items, pairs, 2 * kRowTile, true, st, log);
  return e;
}

}  // namespace

cudaError_t launch_cross_tc(const CrossArgs& a, unsigned int* err, cudaStream_t st, LaunchLog& log) {
  log.add("cross_tc");
  return a.d == 64 ? run<64>(a, err, st, log) : run<128>(a, err, st, log);
}

}  // namespace avq
