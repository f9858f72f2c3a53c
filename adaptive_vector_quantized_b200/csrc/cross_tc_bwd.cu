// Gradients of the exact attention on the tensor cores (bf16), without atomics:
// dK and dV by blocks that own a tile of keys and walk the rows, dQ by blocks
// that own a tile of rows and walk the keys.  S and dP are formed in both (7
// products of tiles instead of 5), so that every sum has one owner and a fixed
// order and no gradient passes through memory in fp32.
//
//   P = exp(S - lse),  dP = dO V^T,  dS = P (dP - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K;  dK = dQ = 0 with one key alone.
//
// A block has two groups of four warps for the elementwise work (a TMEM lane to
// a thread, half of the tile's columns to a group), a warp that loads by TMA, one
// that fetches lse and delta (dK/dV) or clears K's rows of keys that are left
// out (dQ), and two that issue the MMAs of a chain each, since what a warp does
// between MMAs would leave the tensor pipe idle.  P and dS overwrite
// S and dP in TMEM as bf16 and are first operands from there.
//   dK/dV:  S(j) -> P(j) -> dV(j), S(j+1)     dP(j) -> dS(j) -> dK(j), dP(j+1)
//   dQ:     S(j), S(j+1) in turn              dP(j) -> dS(j) -> dQ(j), dP(j+1)
// For dK and dV the chains run apart for the two groups' halves of a tile, so
// that one group works while the MMAs of the other's half do (8192 rows x 4096
// keys, 8 heads of 128 on 4: 298 us against 312 when both were built); for dQ, whose
// S is a step ahead anyhow, whole tiles are better (233 us against 246): a product
// with 64 columns takes 48 clocks of shared memory reads, one with 128 takes 64.
// What bound both most was the MMA warps' own issue: run converged, with their
// descriptors in uniform registers, they brought the whole call from 463 to 394 us
// (captured, in bursts; 407 us now, with every wait agreed on by its warp: 845 TFLOP/s
// of the 5 products that the formulas need; 467 under the power cap, run for seconds).
//
// With at most one key tile (text states) and d = 64 the dK/dV blocks see every
// key of a row, and TMEM has room: they form dQ too, from a copy of dS in shared
// memory (the rows of dS^T are keys, so it is read column by column), and Q and
// dO are read once: 24 heads of 4096 rows over 77 keys 65 us apart, 39 us so,
// 32 us with the converged MMA warps.
#include "cross_tc.cuh"

namespace avq {

namespace {

constexpr int kWorkWarps = 8;
constexpr int kMmaWarp = 8;  // and the next: the chain of S, the chain of dP
constexpr int kLoadWarp = 10, kHelpWarp = 11;
constexpr int kThreads = 384;
// registers: 168 a thread at launch, then 2 * 216 + 72 = 3 * 168
constexpr int kWorkRegs = 216, kOtherRegs = 72;

template <int D>
struct Smem {
  static constexpr int kBlocks = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;
  // Rings of the walked tiles: the first of each pair (Q, or K) is held from the
  // product of its S to that of the gradient, the second (dO, or V) for less.
  static constexpr int kSlotsA = 3, kSlotsB = 2;
  static constexpr int kOwn = 0;  // the block's own two tiles; results staged there
  static constexpr int kRingA = 2 * kTileBytes;
  static constexpr int kRingB = kRingA + kSlotsA * kTileBytes;
  static constexpr int kRows = kRingB + kSlotsB * kTileBytes;  // [2 stages][lse, delta][128]
  // where dK/dV blocks form dQ too: dS [2 halves of the rows][128 keys][64], dQ staged [8 warps][32 rows][64]
  static constexpr bool kRoom = D == 64;
  static constexpr int kDS = kRows + 2 * 1024;
  static constexpr int kOutQ = kDS + (kRoom ? 2 * 16384 : 0);
  static constexpr int kBar = kOutQ + (kRoom ? kWorkWarps * 4096 : 0);
  // a_full[3], a_empty[3], a_ready[3], b_full[2], b_empty[2], own_full, own_empty, s_full[2], dp_full[2], p_ready[2],
  // ds_ready[2], done, rows_full[2], rows_empty[2], drain[2], dq_full[2], dq_taken[2], own_ready
  static constexpr int kBars = 3 * kSlotsA + 2 * kSlotsB + 22;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kTotal = kMisc + 16;
};

struct Bars {
  uint64_t *a_full, *a_empty, *a_ready, *b_full, *b_empty, *own_full, *own_empty, *s_full, *dp_full, *p_ready,
      *ds_ready, *done, *rows_full, *rows_empty, *drain, *dq_full, *dq_taken, *own_ready;
};
template <int D>
__device__ __forceinline__ Bars bars_of(uint8_t* sm) {
  using S = Smem<D>;
  Bars b;
  b.a_full = reinterpret_cast<uint64_t*>(sm + S::kBar);
  b.a_empty = b.a_full + S::kSlotsA;
  b.a_ready = b.a_empty + S::kSlotsA;
  b.b_full = b.a_ready + S::kSlotsA;
  b.b_empty = b.b_full + S::kSlotsB;
  b.own_full = b.b_empty + S::kSlotsB;
  b.own_empty = b.own_full + 1;
  b.s_full = b.own_empty + 1;
  b.dp_full = b.s_full + 2;
  b.p_ready = b.dp_full + 2;
  b.ds_ready = b.p_ready + 2;
  b.done = b.ds_ready + 2;
  b.rows_full = b.done + 1;
  b.rows_empty = b.rows_full + 2;
  b.drain = b.rows_empty + 2;
  b.dq_full = b.drain + 2;
  b.dq_taken = b.dq_full + 2;
  b.own_ready = b.dq_taken + 2;
  return b;
}
// A ring's slot and phase, stepped along.
template <int kSlots>
struct Turn {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// b_users: threads that release a slot of the second ring; p_warps: warps that
// arrive at a p_ready; done_users: threads whose last MMAs complete an item.
template <int D>
__device__ __forceinline__ void init_bars(const Bars& b, int b_users, int p_warps, int done_users) {
  for (int i = 0; i < Smem<D>::kBars; ++i) {
    uint64_t* x = b.a_full + i;
    uint32_t n = 1;
    if (x == b.own_empty || (x >= b.rows_empty && x < b.drain)) n = kWorkWarps;
    if (x >= b.b_empty && x < b.own_full) n = b_users;
    if (x >= b.p_ready && x < b.ds_ready) n = p_warps;
    if ((x >= b.ds_ready && x < b.done) || (x >= b.dq_taken && x < b.own_ready)) n = kWorkWarps / 2;
    if (x == b.done) n = done_users;
    tc::mbar_init(x, n);
  }
  tc::fence_mbar_init();
}

// Waits, with a limit, for the last load into each slot of a ring (`loads` in
// all; t: the turn after the last): nothing may be in flight when a block ends.
template <int kSlots>
__device__ __forceinline__ void drain_ring(uint64_t* full, Turn<kSlots> t, uint32_t loads) {
  for (uint32_t k = 0; k < kSlots; ++k, t.step())  // t.slot: the slot whose last load is oldest
    if (loads + k >= kSlots) tc::mbar_wait(full + t.slot, t.phase ^ 1, 1000000ull);
}

struct Maps {
  CUtensorMap q, g, k, v, out0, out1, out2;  // out: dV, dK and dQ, or dQ alone
};

// A [128 rows][D] tile by TMA
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, const Strides& st, int row, int h,
                                          int b, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    tc::tma_load_4d(dst + c * 128 * 128, map, c * 64, row, st.h != 0 ? h : 0, st.b != 0 ? b : 0, bar);
}

// D[128 x N] = A[128][D] B[N][D]^T, both tiles of rows in shared memory
template <int D, int N>
__device__ __forceinline__ void mma_rows_rows(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, N, 0, 0);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const int off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
    tc::mma_bf16(d, a + off, b + off, idesc, k > 0);
  }
}
// D[128 x D] (+)= A[128][64] B[64][D]: A in TMEM, B rows of a tile in shared memory
template <int D>
__device__ __forceinline__ void mma_tmem_cols(uint32_t d, uint32_t a, uint64_t b, uint32_t more) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, D, 0, 1);
#pragma unroll
  for (int k = 0; k < 4; ++k) tc::mma_bf16_ts(d, a + k * 8, b + k * (2048 >> 4), idesc, k > 0 ? 1 : more);
}
constexpr int kHalf16 = 64 * 128 >> 4;  // from a tile's row 0 to its row 64, in units of a descriptor

// -log2e lse of a row; one with scores of -inf alone has lse = -inf and P = 0.
__device__ __forceinline__ float row_shift(float lse) { return lse == -INFINITY ? -INFINITY : -lse * kLog2e; }

// p = exp2(c2 s + nl) for 32 scores, a quarter of them on the FMA pipe
template <bool kVec>
__device__ __forceinline__ void exp_chunk(const uint32_t* r, float2 c2, const float* nl, float2 nl1, float2* p) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 l = kVec ? fm::f2(nl[2 * i], nl[2 * i + 1]) : nl1;
    const float2 x = fm::fma2(fm::f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), c2, l);
    p[i] = (i & 3) == 3 ? fm::exp2_poly2_any(x) : fm::f2(tc::ex2(x.x), tc::ex2(x.y));
  }
}

// 64 columns of an accumulator row (times f; 0 for a key that is left out, `on`
// false, whatever the rows held), as bf16 into the warp's staging rows, then to
// memory by TMA.
__device__ __forceinline__ void store_block(uint32_t taddr, float f, bool on, uint8_t* out, const CUtensorMap* map,
                                            int col, int row, int rows, int h, int b, int lane) {
  if (lane == 0) tc::bulk_wait_group_read0();
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t o[32];
    tc::tmem_ld32(taddr + c * 32, o);
    tc::tmem_wait_ld();
    if (!on) {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0u;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4 v;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__uint_as_float(o[k * 8 + 2 * e]) * f, __uint_as_float(o[k * 8 + 2 * e + 1]) * f);
      *reinterpret_cast<uint4*>(out + lane * 128 + (((c * 4 + k) ^ (lane & 7)) << 4)) = v;
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (row < rows) tc::tma_store_4d(map, out, col, row, h, b);
    tc::bulk_commit_group();
  }
}
// The same row in fp32, straight to memory (partial results).
template <int D>
__device__ __forceinline__ void store_partial(uint32_t taddr, float f, bool on, float* dst, bool live) {
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t o[16];
    tc::tmem_ld16(taddr + c * 16, o);
    tc::tmem_wait_ld();
    if (!on) {
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = 0u;
    }
    if (live) {
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *reinterpret_cast<float4*>(dst + c * 16 + k) =
            make_float4(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f, __uint_as_float(o[k + 2]) * f,
                        __uint_as_float(o[k + 3]) * f);
    }
  }
}

// ---- dK and dV -------------------------------------------------------------------

struct KeyItem {
  int kb, kh, k0, count, split;
  int i0, i1;  // row tiles of the query heads and entries that share the key head
};
// any_rows: also of a tile with no key (its rows' dQ are written here).
__device__ __forceinline__ KeyItem key_item(const CrossArgs& a, int i, int ktiles, int rtiles, bool any_rows = false) {
  KeyItem x;
  x.k0 = i % ktiles * 128;
  const int rest = i / ktiles;
  x.split = rest % a.splits;
  const int bh = rest / a.splits;
  x.kb = bh / a.Hk;
  x.kh = bh % a.Hk;
  x.count = key_count(a, x.kb);
  const int all = any_rows || x.k0 < x.count ? a.per_b * a.per_h * rtiles : 0;
  x.i0 = part_begin(all, x.split, a.splits);
  x.i1 = part_begin(all, x.split + 1, a.splits);
  return x;
}
struct RowTile {
  int b, h, row0;
};
__device__ __forceinline__ RowTile row_tile(const CrossArgs& a, const KeyItem& x, int i, int rtiles) {
  const int rg = i / rtiles;
  return RowTile{x.kb * a.per_b + rg / a.per_h, x.kh * a.per_h + rg % a.per_h, (i - rg * rtiles) * 128};
}

// The work of a block that is number `block` of `blocks`.
template <int D, bool kWithQ>
__device__ __forceinline__ void form_dkv(uint8_t* sm, const Maps& maps, const CrossArgs& a, unsigned int* err,
                                         int items, int ktiles, int rtiles, int block, int blocks) {
  using S = Smem<D>;
  // kWithQ: the whole grid, by its special registers (two registers that would spill)
  auto first = [&] { return kWithQ ? (int)blockIdx.x : block; };
  auto stride = [&] { return kWithQ ? (int)gridDim.x : blocks; };
  const Bars bar = bars_of<D>(sm);
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + S::kMisc);
  int* sAbort = reinterpret_cast<int*>(sm + S::kMisc + 4);
  float* sRows = reinterpret_cast<float*>(sm + S::kRows);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    init_bars<D>(bar, 2, kWorkWarps / 2, 2);
    *sAbort = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(sTmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  grid_dependency_wait();  // delta, and everything before it
  if (kWithQ) allow_dependents();
  const Guard guard{err, sAbort};
  const uint32_t tmem = *sTmem;
  // S | dP | dV | dK, and behind them dQ of even and of odd steps
  const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 256 + D, tQ = tmem + 256 + 2 * D;

  if (warp >= kWorkWarps) {
    tc::regs_give<kOtherRegs>();
    if (warp == kLoadWarp) {
      if (lane == 0) {
        Turn<S::kSlotsA> ta;
        Turn<S::kSlotsB> tb;
        uint32_t na = 0, nb = 0, own = 0;
        bool ok = true;
        for (int i = first(); i < items && ok; i += stride()) {
          const KeyItem x = key_item(a, i, ktiles, rtiles);
          if (x.i0 >= x.i1) continue;
          ok = guard.wait(bar.own_empty, (own & 1) ^ 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(bar.own_full, 2 * S::kTileBytes);
          load_tile<D>(sm + S::kOwn, &maps.k, a.ks, x.k0, x.kh, x.kb, bar.own_full);
          load_tile<D>(sm + S::kOwn + S::kTileBytes, &maps.v, a.vs, x.k0, x.kh, x.kb, bar.own_full);
          ++own;
          for (int j = x.i0; j < x.i1; ++j) {
            const RowTile r = row_tile(a, x, j, rtiles);
            ok = guard.wait(bar.a_empty + ta.slot, ta.phase ^ 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(bar.a_full + ta.slot, S::kTileBytes);
            load_tile<D>(sm + S::kRingA + ta.slot * S::kTileBytes, &maps.q, a.qs, r.row0, r.h, r.b,
                         bar.a_full + ta.slot);
            ta.step();
            ++na;
            ok = guard.wait(bar.b_empty + tb.slot, tb.phase ^ 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(bar.b_full + tb.slot, S::kTileBytes);
            load_tile<D>(sm + S::kRingB + tb.slot * S::kTileBytes, &maps.g, a.gs, r.row0, r.h, r.b,
                         bar.b_full + tb.slot);
            tb.step();
            ++nb;
          }
        }
        drain_ring(bar.a_full, ta, na);
        drain_ring(bar.b_full, tb, nb);
        if (own > 0) tc::mbar_wait(bar.own_full, (own - 1) & 1, 1000000ull);
      }
    } else if (warp == kHelpWarp) {
      uint32_t n = 0, own = 0;
      bool ok = true;
      for (int i = first(); i < items && ok; i += stride()) {
        const KeyItem x = key_item(a, i, ktiles, rtiles);
        if (kWithQ && x.i0 < x.i1) {
          // K's rows of keys that are left out become zeros: K is a factor of dS K
          ok = wait_all(guard, bar.own_full, own & 1);
          if (!ok) break;
          ++own;
          if (!tile_full(a, x.k0, x.count))
            clear_rows<D>(sm + S::kOwn, key_bits(a, x.kb, x.k0, x.count, lane), min(128, a.Nk - x.k0), lane);
          if (lane == 0) tc::mbar_arrive(bar.own_ready);
        }
        for (int j = x.i0; j < x.i1; ++j, ++n) {
          const RowTile r = row_tile(a, x, j, rtiles);
          const size_t head = ((size_t)r.b * a.Hq + r.h) * a.Nq;
          float l[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = r.row0 + 32 * e + lane;
            const bool in = row < a.Nq;  // past the end: P = exp2(-inf)
            l[e] = in ? row_shift(__ldg(a.lse + head + row)) : -INFINITY;
            d[e] = in ? -__ldg(a.delta + head + row) : 0.f;
          }
          ok = wait_all(guard, bar.rows_empty + (n & 1), (n >> 1 & 1) ^ 1);
          if (!ok) break;
          float* dst = sRows + (n & 1) * 256;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dst[32 * e + lane] = l[e];
            dst[128 + 32 * e + lane] = d[e];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar.rows_full + (n & 1));
        }
      }
    } else {
      const bool second = warp > kMmaWarp;  // the chain of dP
      const uint64_t own = tc::sdesc_sw128(tc::smem_u32(sm + S::kOwn), 16, 1024);
      const uint64_t ring_a = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingA), 16, 1024);
      const uint64_t ring_b = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingB), 16, 1024);
      const uint64_t ring_a_mn = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingA), 128 * 128, 1024);
      const uint64_t ring_b_mn = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingB), 128 * 128, 1024);
      constexpr int kTile16 = S::kTileBytes >> 4;
      Turn<S::kSlotsA> ta;  // Q and dO of the row tile whose gradients are next,
      Turn<S::kSlotsB> tb;
      Turn<S::kSlotsA> ta1;  // and of the one whose S and dP are
      Turn<S::kSlotsB> tb1;
      uint32_t own_n = 0, steps = 0;
      bool ok = true;
      // S^T = K Q^T or dP^T = V dO^T of half a row tile's rows
      auto form = [&](int half) {
        const uint32_t d = (second ? tP : tS) + half * 64;
        if (!second) {
          if (half == 0 && !wait_all(guard, bar.a_full + ta1.slot, ta1.phase)) return false;
          if (tc::elect_one()) {
            mma_rows_rows<D, 64>(d, own, ring_a + ta1.slot * kTile16 + half * kHalf16);
            tc::mma_commit(bar.s_full + half);
          }
          if (half == 1) ta1.step();
        } else {
          if (half == 0 && !wait_all(guard, bar.b_full + tb1.slot, tb1.phase)) return false;
          if (tc::elect_one()) {
            mma_rows_rows<D, 64>(d, own + kTile16, ring_b + tb1.slot * kTile16 + half * kHalf16);
            tc::mma_commit(bar.dp_full + half);
            if (half == 1) tc::mma_commit(bar.b_empty + tb1.slot);  // dO: the chain of S releases it too
          }
          if (half == 1) tb1.step();
        }
        return true;
      };
      for (int i = first(); i < items && ok; i += stride()) {
        const KeyItem x = key_item(a, i, ktiles, rtiles);
        const int tiles = uniform(x.i1 - x.i0);
        if (tiles <= 0) continue;
        ok = wait_all(guard, kWithQ ? bar.own_ready : bar.own_full, own_n & 1) && form(0) && form(1);
        if (!ok) break;
        ++own_n;
        uint32_t more = 0;
        for (int left = tiles; left > 0 && ok; --left, ++steps) {
          uint64_t* const full = second ? bar.a_full + ta.slot : bar.b_full + tb.slot;
          ok = wait_all(guard, full, second ? ta.phase : tb.phase);
          if (!ok) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = wait_all(guard, (second ? bar.ds_ready : bar.p_ready) + half, steps & 1);
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
              if (!second) {  // dV += P^T dO
                mma_tmem_cols<D>(tV, tS + half * 64, ring_b_mn + tb.slot * kTile16 + half * kHalf16, more);
              } else {  // dK += dS^T Q
                mma_tmem_cols<D>(tK, tP + half * 64, ring_a_mn + ta.slot * kTile16 + half * kHalf16, more);
              }
            }
            more = 1;
            if (left > 1) ok = form(half);
            if (!ok) break;
          }
          if (!ok) break;
          if (!second) {
            if (tc::elect_one()) tc::mma_commit(bar.b_empty + tb.slot);
            tb.step();
          } else {
            if (tc::elect_one()) tc::mma_commit(bar.a_empty + ta.slot);
            ta.step();
            if constexpr (kWithQ) {  // dQ = dS K: the columns of dS^T as rows
              const uint32_t buf = steps & 1;
              ok = wait_all(guard, bar.dq_taken + buf, (steps >> 1 & 1) ^ 1);
              if (!ok) break;
              tc::tc_fence_after();
              const uint64_t ds = tc::sdesc_sw128(tc::smem_u32(sm + S::kDS), 128 * 128, 1024);
              const uint64_t own_mn = tc::sdesc_sw128(tc::smem_u32(sm + S::kOwn), 128 * 128, 1024);
              constexpr uint32_t idesc = tc::idesc_bf16(128, D, 1, 1);
              if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  tc::mma_bf16(tQ + buf * D, ds + k * (2048 >> 4), own_mn + k * (2048 >> 4), idesc, k > 0);
                tc::mma_commit(bar.dq_full + buf);
              }
            }
          }
          if (left == 1) {
            if (tc::elect_one()) tc::mma_commit(bar.done);
          }
        }
      }
      uint64_t* drain = bar.drain + second;
      if (tc::elect_one()) tc::mma_commit(drain);
      __syncwarp();
      tc::mbar_wait(drain, 0, 1000000ull);
    }
  } else {
    tc::regs_take<kWorkRegs>();
    const int half = warp >> 2, quarter = warp & 3;  // rows 64 half .. + 63 of the row tile; key lanes of the tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t* out = sm + S::kOwn + warp * 4096;
    const float c2f = a.scale * kLog2e;
    const float2 c2 = fm::f2(c2f, c2f);
    uint32_t steps = 0, dones = 0;
    bool ok = true;
    RowTile before{};  // the row tile of the step before, whose dQ is under way
    float factor = 0.f;  // on dS K and dS^T Q
    // dQ of step n: its group (they take turns) writes the rows
    auto write_q = [&](uint32_t n) {
      const uint32_t buf = n & 1;
      if (!wait_all(guard, bar.dq_full + buf, n >> 1 & 1)) return false;
      tc::tc_fence_after();
      if (half == (int)buf) {
        store_block(tQ + buf * D + lane_off, factor, true, sm + S::kOutQ + warp * 4096, &maps.out2, 0,
                    before.row0 + quarter * 32, a.Nq, a.Hq > 1 ? before.h : 0, a.B > 1 ? before.b : 0, lane);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar.dq_taken + buf);
      }
      return true;
    };
    for (int i = first(); i < items && ok; i += stride()) {
      const KeyItem x = key_item(a, i, ktiles, rtiles);
      if (kWithQ && x.count == 0) {  // no key: dQ = 0
        const KeyItem y = key_item(a, i, ktiles, rtiles, true);
        for (int j = y.i0; j < y.i1; ++j) {
          const RowTile r = row_tile(a, y, j, rtiles);
          for (int e = threadIdx.x; e < 128 * D / 8; e += kWorkWarps * 32) {
            const int row = r.row0 + e / (D / 8);
            if (row < a.Nq)
              *reinterpret_cast<uint4*>(static_cast<bf16*>(a.dQ) +
                                        (((size_t)r.b * a.Hq + r.h) * a.Nq + row) * D + e % (D / 8) * 8) =
                  make_uint4(0, 0, 0, 0);
          }
        }
      }
      factor = lone_key(a, x.kb, x.count) ? 0.f : a.scale;
      const int key = x.k0 + quarter * 32 + lane;
      const bool live = key_seen(a, x.kb, key, x.count);
      for (int j = x.i0; j < x.i1; ++j, ++steps) {
        const float* rows = sRows + (steps & 1) * 256 + half * 64;
        ok = wait_all(guard, bar.rows_full + (steps & 1), steps >> 1 & 1) &&
             wait_all(guard, bar.s_full + half, steps & 1);
        if (!ok) break;
        tc::tc_fence_after();
        float2 p[32];
        uint32_t r[64];
        tc::tmem_ld32(tS + lane_off + half * 64, r);
        tc::tmem_ld32(tS + lane_off + half * 64 + 32, r + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
          float nl[32];
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(nl + e) = *reinterpret_cast<const float4*>(rows + c * 32 + e);
          exp_chunk<true>(r + c * 32, c2, nl, c2, p + c * 16);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (!live) p[c * 16 + e] = fm::f2(0.f, 0.f);  // whatever stands in the key's row
            w[e] = pack_bf16x2(p[c * 16 + e].x, p[c * 16 + e].y);
          }
          tc::tmem_st16(tS + lane_off + half * 64 + c * 16, w);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar.p_ready + half);
        ok = wait_all(guard, bar.dp_full + half, steps & 1);
        if (!ok) break;
        tc::tc_fence_after();
        tc::tmem_ld32(tP + lane_off + half * 64, r);
        tc::tmem_ld32(tP + lane_off + half * 64 + 32, r + 32);
        tc::tmem_wait_ld();
        if (kWithQ && j > x.i0) {  // dQ of the step before has been formed from the last dS
          ok = write_q(steps - 1);
          if (!ok) break;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
          float nd[32];
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(nd + e) = *reinterpret_cast<const float4*>(rows + 128 + c * 32 + e);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = c * 32 + 2 * e;
            float2 d = fm::add2(fm::f2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                fm::f2(nd[2 * e], nd[2 * e + 1]));
            d = fm::mul2(d, p[c * 16 + e]);
            w[e] = live ? pack_bf16x2(d.x, d.y) : 0u;
          }
          tc::tmem_st16(tP + lane_off + half * 64 + c * 16, w);
          if constexpr (kWithQ) {
            const int row = quarter * 32 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(sm + S::kDS + half * 16384 + row * 128 + (((c * 4 + e) ^ (row & 7)) << 4)) =
                  make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        }
        if constexpr (kWithQ) {
          tc::fence_proxy_async_smem();
          before = row_tile(a, x, j, rtiles);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar.ds_ready + half);
          tc::mbar_arrive(bar.rows_empty + (steps & 1));
        }
      }
      if (!ok) break;
      if (kWithQ && x.i0 < x.i1) {
        ok = write_q(steps - 1);
        if (!ok) break;
      }
      // group 0 writes dV, group 1 dK
      const bool any = x.i0 < x.i1;
      const uint32_t acc = (half == 0 ? tV : tK) + lane_off;
      const float f = half == 0 ? 1.f : factor;
      const size_t elems = (size_t)a.Bk * a.Hk * a.Nk * D;
      const size_t at = (((size_t)x.kb * a.Hk + x.kh) * a.Nk + key) * D;
      if (any) {
        ok = wait_all(guard, bar.done, dones & 1);
        if (!ok) break;
        ++dones;
        tc::tc_fence_after();
      }
      if (a.splits > 1) {
        float* dst = a.part + ((size_t)x.split * 2 + (half == 0 ? 1 : 0)) * elems + at;
        if (any) {
          store_partial<D>(acc, f, live, dst, key < a.Nk);
        } else if (key < a.Nk) {
          for (int c = 0; c < D; c += 4) *reinterpret_cast<float4*>(dst + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else if (any) {
#pragma unroll
        for (int cb = 0; cb < S::kBlocks; ++cb)
          store_block(acc + cb * 64, f, live, out, half == 0 ? &maps.out0 : &maps.out1, cb * 64,
                      x.k0 + quarter * 32, a.Nk, a.Hk > 1 ? x.kh : 0, a.Bk > 1 ? x.kb : 0, lane);
      } else if (key < a.Nk) {
        bf16* dst = static_cast<bf16*>(half == 0 ? a.dV : a.dK) + at;
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
      }
      tc::tc_fence_before();
      if (any) {
        if (lane == 0) {
          tc::bulk_wait_group_read0();  // K and V may be loaded over the staging rows
          tc::mbar_arrive(bar.own_empty);
        }
        __syncwarp();
      }
    }
    if (lane == 0) tc::bulk_wait_group0();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---- dQ ------------------------------------------------------------------------------

struct RowItem {
  int b, h, kb, kh, row0, count, t0, t1, parts;
};
__device__ __forceinline__ RowItem row_item(const CrossArgs& a, int i, int rtiles) {
  RowItem x;
  const Part part = part_of(a, i);
  x.parts = part.parts;
  x.row0 = part.item % rtiles * 128;
  const int bh = part.item / rtiles;
  x.b = bh / a.Hq;
  x.h = bh % a.Hq;
  x.kb = x.b / a.per_b;
  x.kh = x.h / a.per_h;
  x.count = key_count(a, x.kb);
  const int kt = (x.count + 127) / 128;
  x.t0 = part_begin(kt, part.split, part.parts);
  x.t1 = part_begin(kt, part.split + 1, part.parts);
  return x;
}

template <int D>
__device__ __forceinline__ void form_dq(uint8_t* sm, const Maps& maps, const CrossArgs& a, unsigned int* err,
                                        int items, int rtiles, int block, int blocks) {
  using S = Smem<D>;
  const Bars bar = bars_of<D>(sm);
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + S::kMisc);
  int* sAbort = reinterpret_cast<int*>(sm + S::kMisc + 4);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    init_bars<D>(bar, 1, kWorkWarps, 1);
    *sAbort = 0;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(sTmem, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  grid_dependency_wait();  // delta, and everything before it
  const Guard guard{err, sAbort};
  const uint32_t tmem = *sTmem;
  const uint32_t tP = tmem + 256, tQ = tmem + 384;  // S of even steps | S of odd steps | dP | dQ

  if (warp >= kWorkWarps) {
    tc::regs_give<kOtherRegs>();
    if (warp == kLoadWarp) {
      if (lane == 0) {
        Turn<S::kSlotsA> ta;
        Turn<S::kSlotsB> tb;
        uint32_t na = 0, nb = 0, own = 0;
        bool ok = true;
        for (int i = block; i < items && ok; i += blocks) {
          const RowItem x = row_item(a, i, rtiles);
          if (x.t0 >= x.t1) continue;
          ok = guard.wait(bar.own_empty, (own & 1) ^ 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(bar.own_full, 2 * S::kTileBytes);
          load_tile<D>(sm + S::kOwn, &maps.q, a.qs, x.row0, x.h, x.b, bar.own_full);
          load_tile<D>(sm + S::kOwn + S::kTileBytes, &maps.g, a.gs, x.row0, x.h, x.b, bar.own_full);
          ++own;
          for (int j = x.t0; j < x.t1; ++j) {
            ok = guard.wait(bar.a_empty + ta.slot, ta.phase ^ 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(bar.a_full + ta.slot, S::kTileBytes);
            load_tile<D>(sm + S::kRingA + ta.slot * S::kTileBytes, &maps.k, a.ks, j * 128, x.kh, x.kb,
                         bar.a_full + ta.slot);
            ta.step();
            ++na;
            ok = guard.wait(bar.b_empty + tb.slot, tb.phase ^ 1);
            if (!ok) break;
            tc::mbar_arrive_expect_tx(bar.b_full + tb.slot, S::kTileBytes);
            load_tile<D>(sm + S::kRingB + tb.slot * S::kTileBytes, &maps.v, a.vs, j * 128, x.kh, x.kb,
                         bar.b_full + tb.slot);
            tb.step();
            ++nb;
          }
        }
        drain_ring(bar.a_full, ta, na);
        drain_ring(bar.b_full, tb, nb);
        if (own > 0) tc::mbar_wait(bar.own_full, (own - 1) & 1, 1000000ull);
      }
    } else if (warp == kHelpWarp) {
      // K's rows of keys that are left out become zeros: K is a factor of dS K too
      Turn<S::kSlotsA> ta;
      bool ok = true;
      for (int i = block; i < items && ok; i += blocks) {
        const RowItem x = row_item(a, i, rtiles);
        for (int j = x.t0; j < x.t1; ++j, ta.step()) {
          ok = wait_all(guard, bar.a_full + ta.slot, ta.phase);
          if (!ok) break;
          if (!tile_full(a, j * 128, x.count))  // rows past the tensor's end came as zeros
            clear_rows<D>(sm + S::kRingA + ta.slot * S::kTileBytes, key_bits(a, x.kb, j * 128, x.count, lane),
                          min(128, a.Nk - j * 128), lane);
          if (lane == 0) tc::mbar_arrive(bar.a_ready + ta.slot);
        }
      }
    } else {
      const bool second = warp > kMmaWarp;  // the chain of dP
      const uint64_t own = tc::sdesc_sw128(tc::smem_u32(sm + S::kOwn), 16, 1024);
      const uint64_t ring_a = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingA), 16, 1024);
      const uint64_t ring_b = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingB), 16, 1024);
      const uint64_t ring_a_mn = tc::sdesc_sw128(tc::smem_u32(sm + S::kRingA), 128 * 128, 1024);
      constexpr int kTile16 = S::kTileBytes >> 4;
      Turn<S::kSlotsA> ta;
      Turn<S::kSlotsB> tb;
      uint32_t own_n = 0, steps = 0;
      bool ok = true;
      auto gradient = [&] {  // dP = dO V^T
        if (!wait_all(guard, bar.b_full + tb.slot, tb.phase)) return false;
        if (tc::elect_one()) {
          mma_rows_rows<D, 128>(tP, own + kTile16, ring_b + tb.slot * kTile16);
          tc::mma_commit(bar.dp_full);
          tc::mma_commit(bar.b_empty + tb.slot);
        }
        tb.step();
        return true;
      };
      for (int i = block; i < items && ok; i += blocks) {
        const RowItem x = row_item(a, i, rtiles);
        const int tiles = uniform(x.t1 - x.t0);
        if (tiles <= 0) continue;
        ok = wait_all(guard, bar.own_full, own_n & 1);
        if (!ok) break;
        ++own_n;
        if (second) {
          ok = gradient();
          uint32_t more = 0;
          for (int left = tiles; left > 0 && ok; --left, ++steps) {
            ok = wait_all(guard, bar.a_ready + ta.slot, ta.phase) && wait_all(guard, bar.ds_ready, steps & 1) &&
                 wait_all(guard, bar.ds_ready + 1, steps & 1);
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {  // dQ += dS K
              mma_tmem_cols<D>(tQ, tP, ring_a_mn + ta.slot * kTile16, more);
              mma_tmem_cols<D>(tQ, tP + 64, ring_a_mn + ta.slot * kTile16 + kHalf16, 1);
              tc::mma_commit(bar.a_empty + ta.slot);
              if (left == 1) tc::mma_commit(bar.done);
            }
            more = 1;
            ta.step();
            if (left > 1) ok = gradient();
          }
        } else {
          // S of each step in the half of TMEM that the step before the last has left
          for (int left = tiles; left > 0; --left, ++steps) {
            ok = wait_all(guard, bar.a_ready + ta.slot, ta.phase) &&
                 wait_all(guard, bar.p_ready + (steps & 1), (steps >> 1 & 1) ^ 1);
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
              mma_rows_rows<D, 128>(tmem + (steps & 1) * 128, own, ring_a + ta.slot * kTile16);
              tc::mma_commit(bar.s_full + (steps & 1));
            }
            ta.step();
          }
        }
      }
      uint64_t* drain = bar.drain + second;
      if (tc::elect_one()) tc::mma_commit(drain);
      __syncwarp();
      tc::mbar_wait(drain, 0, 1000000ull);
    }
  } else {
    tc::regs_take<kWorkRegs>();
    const int half = warp >> 2, quarter = warp & 3;  // keys 64 half .. + 63 of the key tile; row lanes of the tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t* out = sm + S::kOwn + warp * 4096;
    const float c2f = a.scale * kLog2e;
    const float2 c2 = fm::f2(c2f, c2f);
    uint32_t steps = 0, dones = 0;
    bool ok = true;
    for (int i = block; i < items && ok; i += blocks) {
      const RowItem x = row_item(a, i, rtiles);
      const int row = x.row0 + quarter * 32 + lane;
      const size_t at = ((size_t)x.b * a.Hq + x.h) * a.Nq + row;
      const bool in = row < a.Nq;
      const float l = in ? row_shift(__ldg(a.lse + at)) : -INFINITY;
      const float dl = in ? -__ldg(a.delta + at) : 0.f;
      const float2 nl = fm::f2(l, l), nd = fm::f2(dl, dl);
      for (int j = x.t0; j < x.t1; ++j, ++steps) {
        const bool whole = tile_full(a, j * 128, x.count);
        uint32_t bits[2] = {0xffffffffu, 0xffffffffu};
        if (!whole) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
            bits[w] = __ballot_sync(0xffffffffu, key_seen(a, x.kb, j * 128 + half * 64 + 32 * w + lane, x.count));
        }
        ok = wait_all(guard, bar.s_full + (steps & 1), steps >> 1 & 1);
        if (!ok) break;
        tc::tc_fence_after();
        float2 p[32];
        uint32_t r[64];
        tc::tmem_ld32(tmem + (steps & 1) * 128 + lane_off + half * 64, r);
        tc::tmem_ld32(tmem + (steps & 1) * 128 + lane_off + half * 64 + 32, r + 32);
        tc::tmem_wait_ld();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar.p_ready + (steps & 1));  // S is in registers
#pragma unroll
        for (int c = 0; c < 2; ++c) exp_chunk<false>(r + c * 32, c2, nullptr, nl, p + c * 16);
        ok = wait_all(guard, bar.dp_full, steps & 1);
        if (!ok) break;
        tc::tc_fence_after();
        tc::tmem_ld32(tP + lane_off + half * 64, r);
        tc::tmem_ld32(tP + lane_off + half * 64 + 32, r + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = c * 32 + 2 * e;
            float2 d = fm::add2(fm::f2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), nd);
            d = fm::mul2(d, p[c * 16 + e]);
            if (!whole) {  // P or dP of a key that is left out may be anything
              if (!(bits[c] >> (2 * e) & 1u)) d.x = 0.f;
              if (!(bits[c] >> (2 * e + 1) & 1u)) d.y = 0.f;
            }
            w[e] = pack_bf16x2(d.x, d.y);
          }
          tc::tmem_st16(tP + lane_off + half * 64 + c * 16, w);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar.ds_ready + half);
      }
      if (!ok) break;
      const bool any = x.t0 < x.t1;
      if (any) {
        ok = wait_all(guard, bar.done, dones & 1);
        if (!ok) break;
        ++dones;
        tc::tc_fence_after();
      }
      // 64 columns of dQ to a group
      const float factor = lone_key(a, x.kb, x.count) ? 0.f : a.scale;
      if (half < S::kBlocks) {
        if (x.parts > 1) {
          float* dst = a.part + ((size_t)(i - a.whole) * 128 + quarter * 32 + lane) * D + half * 64;
          if (any) {
            store_partial<64>(tQ + lane_off + half * 64, factor, true, dst, in);
          } else if (in) {
            for (int c = 0; c < 64; c += 4) *reinterpret_cast<float4*>(dst + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        } else if (any) {
          store_block(tQ + lane_off + half * 64, factor, true, out, &maps.out2, half * 64, x.row0 + quarter * 32, a.Nq,
                      a.Hq > 1 ? x.h : 0, a.B > 1 ? x.b : 0, lane);
        } else if (in) {
          bf16* dst = static_cast<bf16*>(a.dQ) + at * D + half * 64;
          for (int c = 0; c < 64; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
        }
      }
      tc::tc_fence_before();
      if (any) {
        if (lane == 0) {
          tc::bulk_wait_group_read0();  // Q and dO may be loaded over the staging rows
          tc::mbar_arrive(bar.own_empty);
        }
        __syncwarp();
      }
    }
    if (lane == 0) tc::bulk_wait_group0();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// ---- the launches ------------------------------------------------------------------------

// Whether the shared memory is aligned; no room is left to align it in the kernel.
__device__ __forceinline__ bool smem_aligned(const uint8_t* sm, unsigned int* err) {
  if (!(tc::smem_u32(sm) & 1023u)) return true;
  if (threadIdx.x == 0) atomicOr(err, kErrInternal);
  grid_dependency_wait();
  return false;
}

// The first key_blocks blocks form dK and dV, the others dQ with the arguments q, on the
// SMs that those leave.  One launch for both: a kernel of its own for dQ that
// started beside the other would read delta before its own wait for the work before
// it, and nothing else makes another kernel's writes visible.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_tc_backward_kernel(const __grid_constant__ Maps maps,
                                                                       const __grid_constant__ CrossArgs a,
                                                                       const __grid_constant__ CrossArgs q,
                                                                       unsigned int* err, int key_items,
                                                                       int row_items, int ktiles, int rtiles,
                                                                       int key_blocks) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (!smem_aligned(sm, err)) return;
  const int block = blockIdx.x;
  if (block < key_blocks)
    form_dkv<D, false>(sm, maps, a, err, key_items, ktiles, rtiles, block, key_blocks);
  else
    form_dq<D>(sm, maps, q, err, row_items, rtiles, block - key_blocks, (int)gridDim.x - key_blocks);
}

// One key tile: all three gradients.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_tc_dqkv_kernel(const __grid_constant__ Maps maps,
                                                                   const __grid_constant__ CrossArgs a,
                                                                   unsigned int* err, int items, int ktiles,
                                                                   int rtiles) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (!smem_aligned(sm, err)) return;
  form_dkv<D, true>(sm, maps, a, err, items, ktiles, rtiles, blockIdx.x, gridDim.x);
}

Strides dense(int B, int H, int N, int d) {
  return Strides{B > 1 ? (int64_t)H * N * d : 0, H > 1 ? (int64_t)N * d : 0, N > 1 ? (int64_t)d : 0};
}

template <int D>
cudaError_t maps_of(const CrossArgs& a, Maps* m) {
  cudaError_t e = make_tmap_view_bf16(&m->q, a.Q, a.qs, a.B, a.Hq, a.Nq, D, 128);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m->g, a.G, a.gs, a.B, a.Hq, a.Nq, D, 128);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m->k, a.K, a.ks, a.Bk, a.Hk, a.Nk, D, 128);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m->v, a.V, a.vs, a.Bk, a.Hk, a.Nk, D, 128);
  return e;
}

// a, q: the arguments for dK and dV, and for dQ.
template <int D>
cudaError_t run(const CrossArgs& a, const CrossArgs& q, unsigned int* err, cudaStream_t st, LaunchLog& log) {
  Maps m;
  const Strides ks = dense(a.Bk, a.Hk, a.Nk, D), qs = dense(a.B, a.Hq, a.Nq, D);
  cudaError_t e = maps_of<D>(a, &m);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.out0, a.dV, ks, a.Bk, a.Hk, a.Nk, D, 32);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.out1, a.dK, ks, a.Bk, a.Hk, a.Nk, D, 32);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.out2, a.dQ, qs, a.B, a.Hq, a.Nq, D, 32);
  if (e != cudaSuccess) return e;
  constexpr int smem = Smem<D>::kTotal;
  const int ktiles = (a.Nk + 127) / 128, rtiles = (a.Nq + 127) / 128;
  const int key_items = a.Bk * a.Hk * ktiles * a.splits;
  const int key_blocks = key_items < num_sms() ? key_items : num_sms();
  if constexpr (D == 64) {
    if (cross_tc_dkv_forms_dq(a.Nk, D)) {
      log.add("cross_tc_dqkv");
      e = allow_smem<cross_tc_dqkv_kernel<D>>(smem);
      if (e != cudaSuccess) return e;
      return launch_after(cross_tc_dqkv_kernel<D>, dim3(key_blocks), dim3(kThreads), smem, st, m, a, err, key_items,
                          ktiles, rtiles);
    }
  }
  log.add("cross_tc_backward");
  e = allow_smem<cross_tc_backward_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  const int items = a.B * a.Hq * rtiles;
  const int row_items = q.whole + (items - q.whole) * q.splits;
  const int row_blocks = row_items < num_sms() ? row_items : num_sms();
  e = launch_after(cross_tc_backward_kernel<D>, dim3(key_blocks + row_blocks), dim3(kThreads), smem, st, m, a, q, err,
                   key_items, row_items, ktiles, rtiles, key_blocks);
  if (e == cudaSuccess && q.whole < items) e = launch_cross_join_items(q, items, rtiles, 128, false, st, log);
  return e;
}

}  // namespace

bool cross_tc_dkv_forms_dq(int Nk, int d) { return d == 64 && Nk <= 128; }

cudaError_t launch_cross_tc_backward(const CrossArgs& a, const CrossArgs& q, unsigned int* err, cudaStream_t st,
                                     LaunchLog& log) {
  return a.d == 64 ? run<64>(a, q, err, st, log) : run<128>(a, q, err, st, log);
}

}  // namespace avq
