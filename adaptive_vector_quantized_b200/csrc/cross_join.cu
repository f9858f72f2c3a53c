// Small kernels around the exact attention: the join of partial results over
// a split axis, in a fixed order, and the rows' products dO O.
#include "cross.cuh"

namespace avq {

namespace {

constexpr int kThreads = 256;

// Partial outputs over disjoint key ranges, each a softmax of its own with its
// log-sum-exp: O = sum_s exp(lse_s - m) O_s / sum_s exp(lse_s - m), m the
// largest.  A range with no key has lse = -inf and its O is not read.
// One row per d / 4 lanes.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_join_kernel(const CrossArgs a) {
  grid_dependency_wait();
  constexpr int L = D / 4;
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const long long row = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (row >= rows) return;
  const int c = (threadIdx.x % L) * 4;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_lse[(size_t)s * rows + row]);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float l = a.part_lse[(size_t)s * rows + row];
    if (l == -INFINITY) continue;
    const float w = exp2f((l - m) * kLog2e);
    const float4 v = *reinterpret_cast<const float4*>(a.part + ((size_t)s * rows + row) * D + c);
    z += w;
    o[0] += w * v.x, o[1] += w * v.y, o[2] += w * v.z, o[3] += w * v.w;
  }
  const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : z);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  const int n = (int)(row % a.Nq), h = (int)(row / a.Nq % a.Hq), b = (int)(row / a.Nq / a.Hq);
  put4(static_cast<T*>(a.O) + b * a.os.b + h * a.os.h + n * a.os.n + c, o);
  if (c == 0 && a.lse != nullptr) a.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
}

// The same for items whose partial results lie together: [item][split][row], and
// for dQ, which is a plain sum.  One row per d / 4 lanes.
template <int D, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) cross_join_items_kernel(const CrossArgs a, int per_head, int rows,
                                                                    long long total) {
  grid_dependency_wait();
  constexpr int L = D / 4;
  const long long g = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (g >= total) return;
  const int c = (threadIdx.x % L) * 4;
  const int j = (int)(g / rows), r = (int)(g % rows);
  const int item = a.whole + j, bh = item / per_head;
  const int n = item % per_head * rows + r, h = bh % a.Hq, b = bh / a.Hq;
  if (n >= a.Nq) return;
  const size_t first = (size_t)j * a.splits * rows + r;
  float o[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f, m = -INFINITY;
  if constexpr (kSoftmax)
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_lse[first + (size_t)s * rows]);
  for (int s = 0; s < a.splits; ++s) {
    float w = 1.f;
    if constexpr (kSoftmax) {
      const float l = a.part_lse[first + (size_t)s * rows];
      if (l == -INFINITY) continue;
      w = exp2f((l - m) * kLog2e);
      z += w;
    }
    const float4 v = *reinterpret_cast<const float4*>(a.part + (first + (size_t)s * rows) * D + c);
    o[0] += w * v.x, o[1] += w * v.y, o[2] += w * v.z, o[3] += w * v.w;
  }
  const size_t row = ((size_t)b * a.Hq + h) * a.Nq + n;
  if constexpr (kSoftmax) {
    const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : z);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    put4(static_cast<bf16*>(a.O) + b * a.os.b + h * a.os.h + n * a.os.n + c, o);
    if (c == 0 && a.lse != nullptr) a.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
  } else {
    put4(static_cast<bf16*>(a.dQ) + row * D + c, o);
  }
}

// out[o][i] = sum_s part[s][o][i], in the order of s; n4: floats of an output / 4.
template <typename T>
__global__ void __launch_bounds__(kThreads) partial_sum_kernel(const float* part, int splits, T* out0, T* out1,
                                                               size_t n4) {
  grid_dependency_wait();
  const size_t all = out1 != nullptr ? 2 * n4 : n4;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (size_t)gridDim.x * kThreads) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(part + (s * all + i) * 4);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    put4(i < n4 ? out0 + i * 4 : out1 + (i - n4) * 4, v);
  }
}

// delta[row] = sum_d dO O, one row per d / 8 lanes: dO and O read once.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_delta_kernel(const CrossArgs a) {
  constexpr int L = D / 8;
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const long long row = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool in = row < rows;
  float s = 0.f;
  if (in) {
    const int c = (threadIdx.x % L) * 8;
    const int n = (int)(row % a.Nq), h = (int)(row / a.Nq % a.Hq), b = (int)(row / a.Nq / a.Hq);
    float x[8], y[8];
    load8(static_cast<const T*>(a.O) + b * a.os.b + h * a.os.h + n * a.os.n + c, x);
    load8(static_cast<const T*>(a.G) + b * a.gs.b + h * a.gs.h + n * a.gs.n + c, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i] * y[i];
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (in && threadIdx.x % L == 0) a.delta[row] = s;
}

template <typename T>
cudaError_t sum_as(const float* part, int splits, void* const* out, int outs, size_t n, cudaStream_t st) {
  const size_t n4 = n / 4;
  size_t blocks = (n4 * outs + kThreads - 1) / kThreads;
  const size_t most = (size_t)num_sms() * 8;
  if (blocks > most) blocks = most;
  return launch_after(partial_sum_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, part, splits,
                      static_cast<T*>(out[0]), outs > 1 ? static_cast<T*>(out[1]) : (T*)nullptr, n4);
}

}  // namespace

cudaError_t launch_cross_join(const CrossArgs& a, avq_dtype dt, cudaStream_t st, LaunchLog& log) {
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const int per = kThreads / (a.d / 4);
  const dim3 grid((unsigned)((rows + per - 1) / per));
  log.add("cross_join");
  if (dt == AVQ_F32)
    return a.d == 64 ? launch_after(cross_join_kernel<float, 64>, grid, dim3(kThreads), 0, st, a)
                     : launch_after(cross_join_kernel<float, 128>, grid, dim3(kThreads), 0, st, a);
  return a.d == 64 ? launch_after(cross_join_kernel<bf16, 64>, grid, dim3(kThreads), 0, st, a)
                   : launch_after(cross_join_kernel<bf16, 128>, grid, dim3(kThreads), 0, st, a);
}

cudaError_t launch_cross_join_items(const CrossArgs& a, int items, int per_head, int rows, bool softmax,
                                    cudaStream_t st, LaunchLog& log) {
  const long long total = (long long)(items - a.whole) * rows;
  const int per = kThreads / (a.d / 4);
  const dim3 grid((unsigned)((total + per - 1) / per));
  log.add("cross_join");
  auto run = [&](auto kernel) {
    return launch_after(kernel, grid, dim3(kThreads), 0, st, a, per_head, rows, total);
  };
  if (a.d == 64) return softmax ? run(cross_join_items_kernel<64, true>) : run(cross_join_items_kernel<64, false>);
  return softmax ? run(cross_join_items_kernel<128, true>) : run(cross_join_items_kernel<128, false>);
}

cudaError_t launch_partial_sum(avq_dtype dt, const float* part, int splits, void* const* out, int outs, size_t n,
                               cudaStream_t st, LaunchLog& log) {
  log.add("partial_sum");
  return dt == AVQ_F32 ? sum_as<float>(part, splits, out, outs, n, st) : sum_as<bf16>(part, splits, out, outs, n, st);
}

cudaError_t launch_cross_delta(const CrossArgs& a, avq_dtype dt, cudaStream_t st, LaunchLog& log) {
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const int per = kThreads / (a.d / 8);
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  log.add("cross_delta");
  if (dt == AVQ_F32) {
    if (a.d == 64) cross_delta_kernel<float, 64><<<grid, kThreads, 0, st>>>(a);
    else cross_delta_kernel<float, 128><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (a.d == 64) cross_delta_kernel<bf16, 64><<<grid, kThreads, 0, st>>>(a);
    else cross_delta_kernel<bf16, 128><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace avq
