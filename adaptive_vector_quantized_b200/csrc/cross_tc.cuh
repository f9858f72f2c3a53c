// Shared by the tensor-core kernels of the exact attention: waits that give
// up, the keys of a tile that are looked at, and the zeroing of the others.
#pragma once

#include "cross.cuh"
#include "fastmath.cuh"

namespace avq {

constexpr int kRowTile = 128;  // rows of Q in one MMA tile
constexpr int kKeyTile = 128;  // keys of a tile

constexpr uint64_t kWaitNs = 2000000000ull;

// Waits end after 2 s, or soon after another warp has given up: the flag in
// shared memory makes every role of the block leave its loop.
struct Guard {
  unsigned int* err;
  volatile int* abort;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait_sleep(bar, parity, 20000u)) {
      if (*abort) return false;
      if (tc::globaltimer_ns() - t0 > kWaitNs) {
        atomicOr(err, kErrTimeout);
        *abort = 1;
        return false;
      }
    }
    return true;
  }
};

// The same for a warp as a whole: all its lanes agree, so that none stays behind in an
// operation that names all 32 when a wait runs out, and the compiler can keep what
// follows in uniform registers.  Guard::wait alone is for lanes that work alone.
__device__ __forceinline__ bool wait_all(const Guard& g, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, g.wait(bar, parity));
}
// wait_all with the lanes' agreement on every look at the barrier: for the warps that
// work on the forward pass's rows (16384 x 16384, 8 heads of 128: 906 us, 921 with
// wait_all; in the gradients wait_all: 8192 x 4096, 8 heads of 128 on 4: 406, 419 with
// this).
__device__ __forceinline__ bool wait_warp(const Guard& g, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  while (!__all_sync(0xffffffffu, tc::mbar_try_wait_sleep(bar, parity, 20000u))) {
    const bool late = tc::globaltimer_ns() - t0 > kWaitNs;
    if (late) {
      atomicOr(g.err, kErrTimeout);
      *g.abort = 1;
    }
    if (__any_sync(0xffffffffu, late || *g.abort)) return false;
  }
  return true;
}
// A value that every lane holds, known to the compiler as such.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Launch item i of a kernel that owns rows: the item of the problem, which of
// its parts, and of how many.
struct Part {
  int item, split, parts;
};
__device__ __forceinline__ Part part_of(const CrossArgs& a, int i) {
  if (i < a.whole) return Part{i, 0, 1};
  const int j = i - a.whole;
  return Part{a.whole + j / a.splits, j % a.splits, a.splits};
}

// Bit i of word w: key k0 + 32 w + i is looked at.  All lanes get all words.
struct KeyBits {
  uint32_t w[4];
};
__device__ __forceinline__ KeyBits key_bits(const CrossArgs& a, int kb, int k0, int count, int lane) {
  KeyBits m;
#pragma unroll
  for (int w = 0; w < 4; ++w) m.w[w] = __ballot_sync(0xffffffffu, key_seen(a, kb, k0 + 32 * w + lane, count));
  return m;
}
// No key of the tile is left out.
__device__ __forceinline__ bool tile_full(const CrossArgs& a, int k0, int count) {
  return a.key_mask == nullptr && k0 + kKeyTile <= count;
}

// Zeroes those of the first `rows` rows of a [128 keys][D] tile (blocks of 64
// columns, 128 bytes a row) whose keys are left out, by one warp: a product
// with 0 must not meet an infinity or NaN that stands there.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, const KeyBits& m, int rows, int lane) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int left = rows - 32 * w;
    uint32_t out = left <= 0 ? 0u : left >= 32 ? ~m.w[w] : ~m.w[w] & ((1u << left) - 1u);
    while (out) {
      const int r = 32 * w + __ffs(out) - 1;
      out &= out - 1;
      if (lane < D / 8)
        *reinterpret_cast<uint4*>(tile + (lane >> 3) * (kKeyTile * 128) + r * 128 + (lane & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace avq
