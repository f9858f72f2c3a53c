// Exact attention over another sequence's keys and values: what the kernels
// of the forward pass, the gradients and the joins share.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "tc_util.cuh"

namespace avq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Keys of encoder sequence kb that are looked at: lengths outside [0, Nk] are
// taken as the nearer end.
__device__ __forceinline__ int key_count(const CrossArgs& a, int kb) {
  if (a.kv_lens == nullptr) return a.Nk;
  const int n = __ldg(a.kv_lens + kb);
  return n < 0 ? 0 : (n > a.Nk ? a.Nk : n);
}
__device__ __forceinline__ bool key_seen(const CrossArgs& a, int kb, int j, int count) {
  return j < count && (a.key_mask == nullptr || __ldg(a.key_mask + (size_t)kb * a.Nk + j) != 0);
}

// Whether one key alone is looked at.  P is 1 then whatever the score: O is that key's
// V, dP and delta are the same number, and dS, dQ and dK are 0.  Formed in two orders
// they differ by their roundings, which must not be handed on as a gradient.
__device__ __forceinline__ bool lone_key(const CrossArgs& a, int kb, int count) {
  return a.lone != nullptr ? a.lone[kb] != 0 : count == 1;
}

// Row r of the rows that read encoder sequence kb and key head kh.
struct RowAt {
  int b, h, n;
};
__device__ __forceinline__ RowAt row_at(const CrossArgs& a, int kb, int kh, int r) {
  const int R = a.per_b, G = a.per_h;
  const int rg = r / a.Nq;
  return RowAt{kb * R + rg / G, kh * G + rg % G, r % a.Nq};
}

// Lets a kernel have `bytes` of dynamic shared memory: asked of the runtime once
// per kernel and device, since small calls are bound by the host.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Where part `split` of `parts` of n units begins (split == parts: where the last
// ends).  A 64-bit division takes hundreds of clocks: not for what is whole.
__device__ __forceinline__ int part_begin(int n, int split, int parts) {
  return split == 0 ? 0 : split == parts ? n : (int)((long long)n * split / parts);
}

template <typename T>
__device__ __forceinline__ void put4(T* p, const float* v);
template <>
__device__ __forceinline__ void put4<float>(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void put4<bf16>(bf16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

}  // namespace avq
