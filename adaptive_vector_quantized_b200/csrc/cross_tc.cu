// Exact attention over another sequence on the tensor cores (bf16).
//
//   S = scale Q K^T,  P = exp(S - m),  O = P V / sum(P),
// in one pass over the keys with a running maximum and sum (fp32).
//
// A block works on pairs of 128-row tiles of one head; both tiles share every
// K and V tile that TMA brings through a ring in shared memory.  One warp loads,
// one issues the MMAs, two groups of four warps do the softmax, a row to a
// thread.  S and O stay in TMEM; P overwrites its S there (bf16, two to a
// column) and is the first operand of P V straight from TMEM.  While one group
// exponentiates its tile the tensor cores work for the other: after P V of a
// tile the next S of the same tile is issued, ordered by the pipe itself.
//
// The accumulator is rescaled only when a row's maximum has grown by more than
// 2^8 since the scale in use (P then stays below 2^8, and its rounding to bf16
// is relative): rare after the first tiles, so the groups do it themselves.
//
// Bound by the exponentials at d = 64 (16 a clock and SM against 2 MMAs of 256
// clocks for 16384 of them), by tensor and exponentials alike at d = 128; so a
// quarter of them go to the FMA pipe (fm::exp2_poly2, 7.5e-5 relative, a
// fiftieth of P's rounding).
#include "cross_tc.cuh"

namespace avq {

namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 384;  // three warpgroups, two warps of the last idle
// Registers per thread: 168 at launch (64512 in all), then 216 for the softmax
// groups' row of 128 scores and 72 for the third (2 * 216 + 72 = 3 * 168).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;

template <int D>
struct Smem {
  static constexpr int kBlocks = D / 64;                      // 64-column blocks of a tile
  static constexpr int kTileBytes = kRowTile * D * 2;
  static constexpr int kQBufs = D == 64 ? 2 : 1;              // the next item's Q while this one's is in use
  static constexpr int kSlots = D == 64 ? 6 : 4;              // ring of K and V tiles, in the order of use
  static constexpr int kQ = 0;                                // [kQBufs][2] tiles
  static constexpr int kRing = kQ + kQBufs * 2 * kTileBytes;
  static constexpr int kOut = kRing + kSlots * kTileBytes;    // [8 warps][32 rows][64 columns]
  static constexpr int kBar = kOut + kSoftmaxWarps * 4096;
  // full[slots], empty[slots], q_full[bufs][2], q_empty[bufs], s_full[2], p_ready[2], o_full[2], drain
  static constexpr int kBars = 2 * kSlots + 3 * kQBufs + 7;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kTotal = kMisc + 16;
};

struct Maps {
  CUtensorMap q, k, v, o;
};

// One item: a pair of row tiles of a head and a range of key tiles.
struct Item {
  int b, h, kb, kh, row0, tiles, count, t0, t1, split;
};

__device__ __forceinline__ Item item_of(const CrossArgs& a, int i, int pairs) {
  Item x;
  const int pair = i % pairs, rest = i / pairs;
  x.split = rest % a.splits;
  const int bh = rest / a.splits;
  x.b = bh / a.Hq;
  x.h = bh % a.Hq;
  x.kb = x.b / (a.B / a.Bk);
  x.kh = x.h / (a.Hq / a.Hk);
  x.row0 = pair * 2 * kRowTile;
  x.tiles = x.row0 + kRowTile < a.Nq ? 2 : 1;
  x.count = key_count(a, x.kb);
  const int kt = (x.count + kKeyTile - 1) / kKeyTile;
  x.t0 = (int)((long long)kt * x.split / a.splits);
  x.t1 = (int)((long long)kt * (x.split + 1) / a.splits);
  return x;
}

// exp2 of 32 scores (fp32 in r) as c2 * s - base, packed to bf16 in out[16];
// the sum of the unrounded values is added to `sum`.
template <bool kMasked>
__device__ __forceinline__ void exp_chunk(const uint32_t* r, float2 c2, float2 nbase, uint32_t bits, uint32_t* out,
                                          float2* sum) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float2 s = fm::f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    float2 x = fm::fma2(s, c2, nbase);
    if constexpr (kMasked) {
      if (!(bits >> (2 * i) & 1u)) x.x = -INFINITY;
      if (!(bits >> (2 * i + 1) & 1u)) x.y = -INFINITY;
    }
    // a masked tile keeps the exact zero of exp2(-inf)
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
  uint64_t* empty = full + S::kSlots;
  uint64_t* q_full = empty + S::kSlots;
  uint64_t* q_empty = q_full + 2 * S::kQBufs;
  uint64_t* s_full = q_empty + S::kQBufs;
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + S::kMisc);
  int* sAbort = reinterpret_cast<int*>(sm + S::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kBars; ++i) {
      uint64_t* b = full + i;
      tc::mbar_init(b, b == p_ready || b == p_ready + 1 ? 4 : 1);
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
  const Guard guard{err, sAbort};
  const uint32_t tmem = *sTmem;
  // columns: S0 | S1 | O0 | O1
  auto tS = [&](int t) { return tmem + t * kKeyTile; };
  auto tO = [&](int t) { return tmem + 2 * kKeyTile + t * D; };

  if (warp >= kSoftmaxWarps) {
    tc::regs_give<kOtherRegs>();
    if (warp == kLoadWarp) {
      if (lane == 0) {
        uint32_t n = 0, q = 0;  // K and V tiles, items' Q loaded so far
        bool ok = true;
        for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
          const Item x = item_of(a, i, pairs);
          if (x.t0 >= x.t1) continue;
          const int buf = q % S::kQBufs;
          ok = guard.wait(q_empty + buf, (q / S::kQBufs & 1) ^ 1);
          if (!ok) break;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, const Strides& st, int row, int h, int b, uint64_t* bar) {
            tc::mbar_arrive_expect_tx(bar, S::kTileBytes);
#pragma unroll
            for (int c = 0; c < KB; ++c)
              tc::tma_load_4d(dst + c * kKeyTile * 128, map, c * 64, row, st.h != 0 ? h : 0, st.b != 0 ? b : 0, bar);
          };
          auto load_kv = [&](int j, bool v) {
            const int slot = n % S::kSlots;
            if (!guard.wait(empty + slot, (n / S::kSlots & 1) ^ 1)) return false;
            load(sm + S::kRing + slot * S::kTileBytes, v ? &maps.v : &maps.k, v ? a.vs : a.ks, j * kKeyTile, x.kh, x.kb,
                 full + slot);
            ++n;
            return true;
          };
          uint8_t* dst = sm + S::kQ + buf * 2 * S::kTileBytes;
          load(dst, &maps.q, a.qs, x.row0, x.h, x.b, q_full + 2 * buf);
          ok = load_kv(x.t0, false);
          if (x.tiles == 2)
            load(dst + S::kTileBytes, &maps.q, a.qs, x.row0 + kRowTile, x.h, x.b, q_full + 2 * buf + 1);
          else
            tc::mbar_arrive(q_full + 2 * buf + 1);  // keeps the phases alike
          ++q;
          for (int j = x.t0; j < x.t1 && ok; ++j) {
            ok = load_kv(j, true);
            if (ok && j + 1 < x.t1) ok = load_kv(j + 1, false);
          }
        }
        // nothing of this block's copies may be in flight when it ends
        for (uint32_t k = n > S::kSlots ? n - S::kSlots : 0; k < n; ++k)
          tc::mbar_wait(full + k % S::kSlots, k / S::kSlots & 1, 1000000ull);
        for (uint32_t k = q > S::kQBufs ? q - S::kQBufs : 0; k < q; ++k)
          for (int t = 0; t < 2; ++t)
            tc::mbar_wait(q_full + 2 * (k % S::kQBufs) + t, k / S::kQBufs & 1, 1000000ull);
      }
    } else if (warp == kMmaWarp) {
      // Steps: (item, key tile) in the order of the softmax groups.  Each turn of
      // the loop issues P V of one step and, tile by tile behind it, S of the next.
      struct Step {
        int i, j, t0, t1, count, kb, tiles;
      };
      auto settle = [&](Step& s) {  // the first step at or after item s.i
        for (; s.i < items; s.i += gridDim.x) {
          const Item x = item_of(a, s.i, pairs);
          s.j = s.t0 = x.t0;
          s.t1 = x.t1;
          s.count = x.count;
          s.kb = x.kb;
          s.tiles = x.tiles;
          if (s.t0 < s.t1) return;
        }
        s.tiles = 0;
      };
      uint32_t n = 0, q = 0, p_phase = 0;
      bool ok = true;
      Step cur{}, next{};  // cur: no tiles yet
      next.i = blockIdx.x;
      settle(next);
      const uint64_t ring = tc::sdesc_sw128(tc::smem_u32(sm + S::kRing), 16, 1024);
      const uint64_t qtile = tc::sdesc_sw128(tc::smem_u32(sm + S::kQ), 16, 1024);
      const uint64_t vring = tc::sdesc_sw128(tc::smem_u32(sm + S::kRing), kKeyTile * 128, 1024);
      int buf = 0;
      while (ok && cur.tiles + next.tiles > 0) {
        uint32_t vslot = 0;
        if (cur.tiles > 0) {
          vslot = n % S::kSlots;
          ok = guard.wait(full + vslot, n / S::kSlots & 1);
          if (!ok) break;
          ++n;
          const int k0 = cur.j * kKeyTile;
          if (!tile_full(a, k0, cur.count))
            clear_rows<D>(sm + S::kRing + vslot * S::kTileBytes, key_bits(a, cur.kb, k0, cur.count, lane),
                          min((cur.count - k0 + 15) & ~15, a.Nk - k0), lane);
        }
        const uint32_t kslot = n % S::kSlots;
        const bool fresh = next.j == next.t0;  // the next step starts an item
        if (next.tiles > 0 && fresh) buf = q % S::kQBufs;
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          if (t < cur.tiles) {
            ok = guard.wait(p_ready + t, p_phase >> t & 1);
            if (!ok) break;
            p_phase ^= 1u << t;
            tc::tc_fence_after();
            if (lane == 0) {
              const uint32_t idesc = tc::idesc_bf16(kRowTile, D, 0, 1);
              const int ksteps = min(kKeyTile, cur.count - cur.j * kKeyTile + 15) >> 4;
              uint64_t vd = vring + (vslot * S::kTileBytes >> 4);
              uint32_t pa = tS(t), more = cur.j > cur.t0;
#pragma unroll 1
              for (int k = 0; k < ksteps; ++k) {
                tc::mma_bf16_ts(tO(t), pa, vd, idesc, more);
                vd += 2048 >> 4;
                pa += 8;
                more = 1;
              }
              if (cur.j + 1 == cur.t1) tc::mma_commit(o_full + t);
            }
            __syncwarp();
          }
          if (t < next.tiles) {
            if (t == 0) ok = guard.wait(full + kslot, n / S::kSlots & 1);
            if (ok && fresh) ok = guard.wait(q_full + 2 * buf + t, q / S::kQBufs & 1);
            if (!ok) break;
            if (lane == 0) {
              const int left = next.count - next.j * kKeyTile;
              const uint32_t idesc = tc::idesc_bf16(kRowTile, left >= kKeyTile ? kKeyTile : (left + 15) & ~15, 0, 0);
              const uint64_t qd = qtile + ((buf * 2 + t) * S::kTileBytes >> 4);
              const uint64_t kd = ring + (kslot * S::kTileBytes >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const int off = ((k >> 2) * (kRowTile * 128) + (k & 3) * 32) >> 4;
                tc::mma_bf16(tS(t), qd + off, kd + off, idesc, k > 0);
              }
              tc::mma_commit(s_full + t);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (lane == 0 && cur.tiles > 0) tc::mma_commit(empty + vslot);
        if (next.tiles > 0) {
          if (lane == 0) tc::mma_commit(empty + kslot);
          ++n;
          if (fresh) ++q;
          if (lane == 0 && next.j + 1 == next.t1) tc::mma_commit(q_empty + buf);
        }
        __syncwarp();
        cur = next;
        if (next.tiles > 0 && ++next.j == next.t1) {
          next.i += gridDim.x;
          settle(next);
        }
      }
      // every MMA done before TMEM is given back
      if (lane == 0) tc::mma_commit(drain);
      __syncwarp();
      tc::mbar_wait(drain, 0, 1000000ull);
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
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
      const Item x = item_of(a, i, pairs);
      if (t >= x.tiles) continue;
      const int r0 = x.row0 + t * kRowTile;
      const size_t grow = ((size_t)x.b * a.Hq + x.h) * a.Nq + r0 + row;
      const bool live = r0 + row < a.Nq;
      float m = -INFINITY;  // maximum behind the scale in use
      float2 sum[2] = {fm::f2(0.f, 0.f), fm::f2(0.f, 0.f)};
      for (int j = x.t0; j < x.t1; ++j) {
        const int k0 = j * kKeyTile;
        const bool whole = tile_full(a, k0, x.count);
        KeyBits bits;
        int chunks = 4;
        if (!whole) {
          bits = key_bits(a, x.kb, k0, x.count, lane);
          chunks = min(4, (x.count - k0 + 31) >> 5);
        }
        ok = guard.wait(s_full + t, s_phase);
        if (!ok) break;
        s_phase ^= 1;
        tc::tc_fence_after();
        uint32_t r[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) tc::tmem_ld32(tS(t) + lane_off + c * 32, r + c * 32);
        tc::tmem_wait_ld();
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (whole) {
#pragma unroll
          for (int k = 0; k < 128; k += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              top[u] = fm::max3_nan(top[u], __uint_as_float(r[k + 2 * u]), __uint_as_float(r[k + 2 * u + 1]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < chunks) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (bits.w[c] >> k & 1u)
                  top[k & 3] = fm::max3_nan(top[k & 3], top[k & 3], __uint_as_float(r[c * 32 + k]));
            }
        }
        const float tile_top = fm::max3_nan(fm::max3_nan(top[0], top[1], top[2]), top[3], top[3]);
        if (j == x.t0) {
          m = tile_top;
        } else {
          // NaN counts as grown: it must reach the output
          const bool grown = tile_top != -INFINITY && !((tile_top - m) * c2f <= 8.f);
          if (__any_sync(0xffffffffu, grown)) {
            const float keep = grown ? exp2f((m - tile_top) * c2f) : 1.f;
            const float2 keep2 = fm::f2(keep, keep);
            if (grown) m = tile_top;
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
        if (whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
            exp_chunk<false>(r + c * 32, c2, nbase, 0, p, sum);
            tc::tmem_st16(tS(t) + lane_off + c * 16, p);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < chunks) {
              uint32_t p[16];
              exp_chunk<true>(r + c * 32, c2, nbase, bits.w[c], p, sum);
              tc::tmem_st16(tS(t) + lane_off + c * 16, p);
            }
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_ready + t);
      }
      if (!ok) break;
      const float z = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : z);
      const float lse = z == 0.f ? -INFINITY : a.scale * m + logf(z);
      const bool any = x.t0 < x.t1;
      if (any) {
        ok = guard.wait(o_full + t, o_phase);
        if (!ok) break;
        o_phase ^= 1;
        tc::tc_fence_after();
      }
      if (live) {
        if (a.splits > 1) a.part_lse[(size_t)x.split * a.B * a.Hq * a.Nq + grow] = lse;
        else if (a.lse != nullptr) a.lse[grow] = lse;
      }
      if (a.splits > 1) {
        // partial results stay in fp32: a row to a thread, straight to memory
        float* dst = a.part + ((size_t)x.split * a.B * a.Hq * a.Nq + grow) * D;
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
cudaError_t run(const CrossArgs& a, unsigned int* err, cudaStream_t st) {
  Maps m;
  cudaError_t e = make_tmap_view_bf16(&m.q, a.Q, a.qs, a.B, a.Hq, a.Nq, D, kRowTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.k, a.K, a.ks, a.Bk, a.Hk, a.Nk, D, kKeyTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.v, a.V, a.vs, a.Bk, a.Hk, a.Nk, D, kKeyTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&m.o, a.O, a.os, a.B, a.Hq, a.Nq, D, 32);
  if (e != cudaSuccess) return e;
  constexpr int smem = Smem<D>::kTotal + 1024;
  e = cudaFuncSetAttribute(cross_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int pairs = (a.Nq + 2 * kRowTile - 1) / (2 * kRowTile);
  const long long items = (long long)a.B * a.Hq * pairs * a.splits;
  const int grid = (int)(items < num_sms() ? items : num_sms());
  cross_tc_kernel<D><<<grid, kThreads, smem, st>>>(m, a, err, (int)items, pairs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_tc(const CrossArgs& a, unsigned int* err, cudaStream_t st, LaunchLog& log) {
  log.add("cross_tc");
  return a.d == 64 ? run<64>(a, err, st) : run<128>(a, err, st);
}

}  // namespace avq
