// Exact attention over another sequence for few rows per key head (bf16): a
// new token of each sequence, its query heads sharing a key head, the samples
// or beams that share an encoder sequence.
//
// All rows that read one (encoder sequence, key head) are taken together, 8 or
// 16 to a block, so K and V are read once for them; the keys are split over
// blocks (joined by a launch of its own) and over a block's four warps (joined
// in shared memory).  Bound by reading K and V.
//
// One thread keeps a ring of 64-key tiles of K and V in shared memory full by
// TMA, across items, so the loads in flight (64 to 96 KB a block, two an SM)
// do not depend on what the arithmetic waits for.  Loads straight into the
// registers of 16 warps, with the next tile's under way, reached 4.7 TB/s, the
// ring 6.2 (32 sequences of 8191 keys, 4 key heads of 128, 4 query heads each).
//
// Each of four warps takes 16 keys of a tile with mma.sync m16n8k16 (with 8 or
// 16 rows a 128-row tile of the tcgen05 path would be empty, and the arithmetic
// is a small part of the loads' time), its operands 16-byte pieces of the
// tile's rows:
//   S = Q K^T: thread (g, t) of the warp holds for key g the elements
//     32 s + 8 t .. + 7; the sum over d may run in any order, so these serve as
//     k elements of two steps, with Q loaded in the same order;
//   O^T += V^T P^T: S comes out as the layout of the second operand; the
//     thread loads elements 8 g .. 8 g + 7 of keys 2t, 2t+1, 2t+8, 2t+9 and
//     pairs the keys with byte permutes; elements 2 i and 2 i + 1 of the chunk
//     are the rows g and g + 8 of output tile i.  O^T takes half the registers
//     that O would with 8 rows, since a first operand has 16 rows.
#include "cross_tc.cuh"

namespace avq {

namespace {

constexpr int kWarps = 4;  // with 16 keys of a tile each; one more loads
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kTile = 64;  // keys of a tile

template <int D, int ROWS>
struct Smem {
  static constexpr int kBytes = kTile * D * 2;  // K or V of a tile: a slot of the ring
  // as many as leave room for two blocks beside the rows' results
  static constexpr int kSlots = D == 64 ? (ROWS == 8 ? 12 : 10) : (ROWS == 8 ? 5 : 4);
  static constexpr int kBar = kSlots * kBytes;  // full[slots], empty[slots], written, taken
  static constexpr int kBars = 2 * kSlots + 2;
  static constexpr int kMisc = kBar + kBars * 8;
  static constexpr int kTotal = kMisc + 16;
};

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Item {
  int kb, kh, chunk, split, count, t0, t1;
};
__device__ __forceinline__ Item item_of(const CrossArgs& a, int i, int chunks) {
  Item x;
  x.chunk = i % chunks;
  const int rest = i / chunks;
  x.split = rest % a.splits;
  const int kvh = rest / a.splits;
  x.kb = kvh / a.Hk;
  x.kh = kvh % a.Hk;
  x.count = key_count(a, x.kb);
  const int tiles = (x.count + kTile - 1) / kTile;
  x.t0 = part_begin(tiles, x.split, a.splits);
  x.t1 = part_begin(tiles, x.split + 1, a.splits);
  return x;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) cross_few_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                const __grid_constant__ CUtensorMap vmap,
                                                                const CrossArgs a, unsigned int* err, int items,
                                                                int chunks) {
  using S = Smem<D, ROWS>;
  constexpr int H = ROWS / 8;  // row halves: rows g and g + 8 of the 16-row tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBar);
  uint64_t* empty = full + S::kSlots;
  uint64_t* written = empty + S::kSlots;
  uint64_t* taken = written + 1;
  int* sAbort = reinterpret_cast<int*>(sm + S::kMisc);
  __shared__ __align__(16) float sO[kWarps][ROWS][D + 4];
  __shared__ float sM[kWarps][ROWS], sZ[kWarps][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kBars; ++i) tc::mbar_init(full + i, i < S::kSlots ? 1 : kWarps);
    tc::fence_mbar_init();
    *sAbort = 0;
  }
  __syncthreads();
  grid_dependency_wait();  // the inputs, and whoever still reads the outputs
  allow_dependents();
  const Guard guard{err, sAbort};

  if (warp == kWarps) {
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < items && ok; i += gridDim.x) {
        const Item x = item_of(a, i, chunks);
        const int kh = a.ks.h != 0 ? x.kh : 0, kb = a.ks.b != 0 ? x.kb : 0;
        const int vh = a.vs.h != 0 ? x.kh : 0, vb = a.vs.b != 0 ? x.kb : 0;
        for (int j = 2 * x.t0; j < 2 * x.t1; ++j, ++n) {  // K, then V of each tile
          const bool v = j & 1;
          const int slot = n % S::kSlots;
          ok = guard.wait(empty + slot, (n / S::kSlots & 1) ^ 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(full + slot, S::kBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tc::tma_load_4d(sm + slot * S::kBytes + c * kTile * 128, v ? &vmap : &kmap, c * 64, (j >> 1) * kTile,
                            v ? vh : kh, v ? vb : kb, full + slot);
        }
      }
      // nothing of this block's copies may be in flight when it ends
      for (uint32_t k = n > S::kSlots ? n - S::kSlots : 0; k < n; ++k)
        tc::mbar_wait(full + k % S::kSlots, k / S::kSlots & 1, 1000000ull);
    }
    return;
  }

  const int rows = a.per_b * a.per_h * a.Nq;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // 16-byte piece c of row r of a [64 keys][D] tile
  auto piece = [&](const uint8_t* tile, int r, int c) {
    return *reinterpret_cast<const uint4*>(tile + (c >> 3) * (kTile * 128) + r * 128 + (((c ^ r) & 7) << 4));
  };
  auto v_row = [&](int i) { return 16 * warp + 2 * t + (i & 1) + 8 * (i >> 1); };
  const float c2 = a.scale * kLog2e;
  uint32_t n = 0;
  int done = 0;  // items whose results went through shared memory
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const Item x = item_of(a, it, chunks);
    uint4 q[H][D / 32];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int r = x.chunk * ROWS + 8 * i + g;
      const RowAt at = row_at(a, x.kb, x.kh, r < rows ? r : 0);
      const bf16* Q = static_cast<const bf16*>(a.Q) + at.b * a.qs.b + at.h * a.qs.h + at.n * a.qs.n + 8 * t;
#pragma unroll
      for (int s = 0; s < D / 32; ++s) q[i][s] = r < rows ? __ldg(reinterpret_cast<const uint4*>(Q + 32 * s)) : zero;
    }
    // o[i][c][e]: row 8 i + 2 t + (e & 1), element 64 (c >> 2) + 8 g + 2 (c & 3) + (e >> 1)
    float o[H][D / 16][4], m[H], z[H];  // m, z: row 8 i + g
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) m[i] = -INFINITY, z[i] = 0.f;

    for (int j = x.t0; j < x.t1; ++j, n += 2) {
      const int kslot = n % S::kSlots, vslot = (n + 1) % S::kSlots;
      const uint8_t* kt = sm + kslot * S::kBytes;
      const uint8_t* vt = sm + vslot * S::kBytes;
      if (!wait_warp(guard, full + kslot, n / S::kSlots & 1)) return;
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          const uint4 q0 = q[0][d], q1 = H == 2 ? q[H - 1][d] : zero;
          const uint4 k = piece(kt, 16 * warp + 8 * nt + g, 4 * d + t);
          mma16816(s[nt], q0.x, q1.x, q0.y, q1.y, k.x, k.y);
          mma16816(s[nt], q0.z, q1.z, q0.w, q1.w, k.z, k.w);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty + kslot);
      if (!wait_warp(guard, full + vslot, (n + 1) / S::kSlots & 1)) return;
      uint4 v[4][D / 64];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < D / 64; ++d) v[i][d] = piece(vt, v_row(i), 8 * d + g);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty + vslot);  // the tile is in registers
      // scores s[nt][2 i + e]: row g + 8 i, key 16 warp + 8 nt + 2 t + e of the tile
      if (a.key_mask != nullptr || (j + 1) * kTile > x.count) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (key_seen(a, x.kb, j * kTile + v_row(i), x.count)) continue;
          s[i >> 1][i & 1] = s[i >> 1][2 + (i & 1)] = -INFINITY;
#pragma unroll
          for (int d = 0; d < D / 64; ++d) v[i][d] = zero;  // an infinity or NaN there meets no product
        }
      }
      float keep[H];
      bool grown = false;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        float top = fm::max3_nan(fm::max3_nan(s[0][2 * i], s[0][2 * i + 1], s[1][2 * i]), s[1][2 * i + 1], s[1][2 * i + 1]);
        top = fm::max3_nan(top, top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fm::max3_nan(top, top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the scale in use is kept until a maximum is more than 2^8 above it; NaN must reach the output
        const bool up = top != -INFINITY && !((top - m[i]) * c2 <= 8.f);
        keep[i] = up ? exp2f((m[i] - top) * c2) : 1.f;
        if (up) m[i] = top;
        grown = grown || up;
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          z[i] *= keep[i];
          const float f0 = __shfl_sync(0xffffffffu, keep[i], 8 * t), f1 = __shfl_sync(0xffffffffu, keep[i], 8 * t + 4);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[i][c][0] *= f0;
            o[i][c][1] *= f1;
            o[i][c][2] *= f0;
            o[i][c][3] *= f1;
          }
        }
      }
      uint32_t p[H][2];  // [row half][key half]
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float base = m[i] == -INFINITY ? 0.f : m[i] * c2;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float e0 = tc::ex2(fmaf(s[nt][2 * i], c2, -base)), e1 = tc::ex2(fmaf(s[nt][2 * i + 1], c2, -base));
          z[i] += e0 + e1;
          p[i][nt] = pack_bf16x2(e0, e1);
        }
      }
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        const uint32_t w[4][4] = {{v[0][d].x, v[0][d].y, v[0][d].z, v[0][d].w},
                                  {v[1][d].x, v[1][d].y, v[1][d].z, v[1][d].w},
                                  {v[2][d].x, v[2][d].y, v[2][d].z, v[2][d].w},
                                  {v[3][d].x, v[3][d].y, v[3][d].z, v[3][d].w}};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t a0 = __byte_perm(w[0][c], w[1][c], 0x5410u), a1 = __byte_perm(w[0][c], w[1][c], 0x7632u);
          const uint32_t a2 = __byte_perm(w[2][c], w[3][c], 0x5410u), a3 = __byte_perm(w[2][c], w[3][c], 0x7632u);
#pragma unroll
          for (int i = 0; i < H; ++i) mma16816(o[i][4 * d + c], a0, a1, a2, a3, p[i][0], p[i][1]);
        }
      }
    }
    // the warps' results: O over one scale of the block, then the sums
    if (done > 0 && !wait_warp(guard, taken, (done - 1) & 1)) return;  // the last item's have been read
#pragma unroll
    for (int i = 0; i < H; ++i) {
      z[i] += __shfl_xor_sync(0xffffffffu, z[i], 1);
      z[i] += __shfl_xor_sync(0xffffffffu, z[i], 2);
      if (t == 0) {
        sM[warp][8 * i + g] = m[i];
        sZ[warp][8 * i + g] = z[i];
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(&sO[warp][8 * i + 2 * t + e][64 * (c >> 2) + 8 * g + 2 * (c & 3)]) =
              make_float2(o[i][c][e], o[i][c][2 + e]);
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(written);
    if (!wait_warp(guard, written, done & 1)) return;
    for (int e = threadIdx.x; e < ROWS * (D / 4); e += kWarps * 32) {
      const int i = e / (D / 4), c = (e % (D / 4)) * 4;
      const int r = x.chunk * ROWS + i;
      if (r >= rows) break;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fm::max3_nan(top, top, sM[w][i]);
      float sum = 0.f, out[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = sM[w][i];
        if (mw == -INFINITY) continue;  // no key of this warp
        const float f = exp2f((mw - top) * c2);
        sum += f * sZ[w][i];
#pragma unroll
        for (int u = 0; u < 4; ++u) out[u] += f * sO[w][i][c + u];
      }
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
      for (int u = 0; u < 4; ++u) out[u] *= inv;
      const float lse = sum == 0.f ? -INFINITY : a.scale * top + logf(sum);
      const RowAt at = row_at(a, x.kb, x.kh, r);
      const size_t row = ((size_t)at.b * a.Hq + at.h) * a.Nq + at.n;
      const size_t all = (size_t)a.B * a.Hq * a.Nq;
      if (a.splits > 1) {
        put4(a.part + ((size_t)x.split * all + row) * D + c, out);
        if (c == 0) a.part_lse[(size_t)x.split * all + row] = lse;
      } else {
        put4(static_cast<bf16*>(a.O) + at.b * a.os.b + at.h * a.os.h + at.n * a.os.n + c, out);
        if (c == 0 && a.lse != nullptr) a.lse[row] = lse;
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(taken);
    ++done;
  }
}

template <int D, int ROWS>
cudaError_t run(const CrossArgs& a, unsigned int* err, cudaStream_t st) {
  const int rows = a.per_b * a.per_h * a.Nq;
  const int chunks = (rows + ROWS - 1) / ROWS;
  CUtensorMap k, v;
  cudaError_t e = make_tmap_view_bf16(&k, a.K, a.ks, a.Bk, a.Hk, a.Nk, D, kTile);
  if (e == cudaSuccess) e = make_tmap_view_bf16(&v, a.V, a.vs, a.Bk, a.Hk, a.Nk, D, kTile);
  if (e != cudaSuccess) return e;
  constexpr int smem = Smem<D, ROWS>::kTotal + 1024;
  e = allow_smem<cross_few_kernel<D, ROWS>>(smem);
  if (e != cudaSuccess) return e;
  const int items = a.Bk * a.Hk * chunks * a.splits;
  const int grid = items < 2 * num_sms() ? items : 2 * num_sms();
  return launch_after(cross_few_kernel<D, ROWS>, dim3(grid), dim3(kThreads), smem, st, k, v, a, err, items, chunks);
}

}  // namespace

cudaError_t launch_cross_few(const CrossArgs& a, unsigned int* err, cudaStream_t st, LaunchLog& log) {
  log.add("cross_few");
  const int rows = a.per_b * a.per_h * a.Nq;
  if (rows <= 8) return a.d == 64 ? run<64, 8>(a, err, st) : run<128, 8>(a, err, st);
  return a.d == 64 ? run<64, 16>(a, err, st) : run<128, 16>(a, err, st);
}

}  // namespace avq
