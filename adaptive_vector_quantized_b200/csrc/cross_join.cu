// Small kernels around the exact attention: the join of partial results over
// a split axis, in a fixed order, and the rows' products dO O.
#include "cross.cuh"

namespace avq {

namespace {

constexpr int kThreads = 256;

// The join of a row's partial results, which stand at rows first, first + step, ...
// of `part` and entries of `part_lse`: columns c .. c + 3.  They are outputs over
// disjoint key ranges, each a softmax of its own with its log-sum-exp:
//   O = sum_s exp(lse_s - m) O_s / sum_s exp(lse_s - m),  m the largest;
// a range with no key has lse = -inf and its O was not written.  Without kSoftmax
// (dQ) they are summed.  kGroups groups of d / 4 lanes take every kGroups-th four
// of them and meet in shared memory: a row's 64 parts one after the other took 17
// us, and with few rows nothing else hides it.  Every order is fixed.
// Returns true in the lanes that hold the result.
template <int D, bool kSoftmax, int kGroups>
__device__ __forceinline__ bool join_row(const CrossArgs& a, size_t first, size_t step, int group, int c, float* o,
                                         float& m, float& z) {
  o[0] = o[1] = o[2] = o[3] = z = 0.f;
  m = -INFINITY;
  for (int s0 = group * 4; s0 < a.splits; s0 += kGroups * 4) {
    float l[4], top = m;
    float4 v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bool in = s0 + s < a.splits;
      l[s] = -INFINITY;
      if (in) l[s] = kSoftmax ? a.part_lse[first + (s0 + s) * step] : 0.f;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (l[s] != -INFINITY) v[s] = *reinterpret_cast<const float4*>(a.part + (first + (s0 + s) * step) * D + c);
      top = fmaxf(top, l[s]);
    }
    if constexpr (kSoftmax) {
      const float keep = m == -INFINITY ? 0.f : exp2f((m - top) * kLog2e);
      z *= keep;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= keep;
      m = top;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float w = !kSoftmax ? 1.f : l[s] == -INFINITY ? 0.f : exp2f((l[s] - m) * kLog2e);
      z += w;
      o[0] += w * v[s].x, o[1] += w * v[s].y, o[2] += w * v[s].z, o[3] += w * v[s].w;
    }
  }
  if constexpr (kGroups > 1) {
    __shared__ __align__(16) float so[kGroups][D];
    __shared__ float sm[kGroups], sz[kGroups];
    *reinterpret_cast<float4*>(&so[group][c]) = make_float4(o[0], o[1], o[2], o[3]);
    if (c == 0) sm[group] = m, sz[group] = z;
    __syncthreads();
    if (group > 0) return false;
    float top = m;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) top = fmaxf(top, sm[g]);
    o[0] = o[1] = o[2] = o[3] = z = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float w = !kSoftmax ? 1.f : sm[g] == -INFINITY ? 0.f : exp2f((sm[g] - top) * kLog2e);
      const float4 v = *reinterpret_cast<const float4*>(&so[g][c]);
      z += w * sz[g];
      o[0] += w * v.x, o[1] += w * v.y, o[2] += w * v.z, o[3] += w * v.w;
    }
    m = top;
  }
  if constexpr (kSoftmax) {
    const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : z);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
  }
  return true;
}

// Partial results of whole problems: [split][row].
template <typename T, int D, int kGroups>
__global__ void __launch_bounds__(kThreads) cross_join_kernel(const CrossArgs a) {
  grid_dependency_wait();
  constexpr int L = D / 4, kPer = kThreads / (L * kGroups);  // rows of a block
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const long long row = (long long)blockIdx.x * kPer + threadIdx.x / (L * kGroups);
  if (row >= rows) return;  // whole blocks when groups meet
  const int c = (threadIdx.x % L) * 4, group = threadIdx.x / L % kGroups;
  float o[4], m, z;
  if (!join_row<D, true, kGroups>(a, row, (size_t)rows, group, c, o, m, z)) return;
  const int n = (int)(row % a.Nq), h = (int)(row / a.Nq % a.Hq), b = (int)(row / a.Nq / a.Hq);
  put4(static_cast<T*>(a.O) + b * a.os.b + h * a.os.h + n * a.os.n + c, o);
  if (c == 0 && a.lse != nullptr) a.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
}

// Partial results of items: [item][split][row].
template <int D, bool kSoftmax, int kGroups>
__global__ void __launch_bounds__(kThreads) cross_join_items_kernel(const CrossArgs a, int per_head, int rows,
                                                                    long long total) {
  grid_dependency_wait();
  constexpr int L = D / 4, kPer = kThreads / (L * kGroups);
  const long long g = (long long)blockIdx.x * kPer + threadIdx.x / (L * kGroups);
  if (g >= total) return;
  const int c = (threadIdx.x % L) * 4, group = threadIdx.x / L % kGroups;
  const int j = (int)(g / rows), r = (int)(g % rows);
  const int item = a.whole + j, bh = item / per_head;
  const int n = item % per_head * rows + r, h = bh % a.Hq, b = bh / a.Hq;
  if (n >= a.Nq) return;
  float o[4], m, z;
  if (!join_row<D, kSoftmax, kGroups>(a, (size_t)j * a.splits * rows + r, rows, group, c, o, m, z)) return;
  const size_t row = ((size_t)b * a.Hq + h) * a.Nq + n;
  if constexpr (kSoftmax) {
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

// delta[row] = sum_d dO O, one row per d / 8 lanes: dO and O read once.  With a mask a
// block more for each encoder sequence, which counts the keys that are looked at as
// far as the second.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_delta_kernel(const CrossArgs a, unsigned row_blocks) {
  grid_dependency_wait();
  allow_dependents();
  if (blockIdx.x >= row_blocks) {
    const int kb = (int)(blockIdx.x - row_blocks), count = key_count(a, kb);
    int seen = 0;
    for (int j = 0; j < count && seen < 2; j += kThreads)
      seen += __syncthreads_count(key_seen(a, kb, j + (int)threadIdx.x, count));
    if (threadIdx.x == 0) a.lone[kb] = seen == 1;
    return;
  }
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

// Groups to a row: a block for many parts, one group for a few.
template <typename T, int D>
cudaError_t join(const CrossArgs& a, cudaStream_t st) {
  constexpr int kAll = kThreads / (D / 4);
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  if (a.splits > 4) return launch_after(cross_join_kernel<T, D, kAll>, dim3((unsigned)rows), dim3(kThreads), 0, st, a);
  return launch_after(cross_join_kernel<T, D, 1>, dim3((unsigned)((rows + kAll - 1) / kAll)), dim3(kThreads), 0, st, a);
}
template <int D, bool kSoftmax>
cudaError_t join_items(const CrossArgs& a, int items, int per_head, int rows, cudaStream_t st) {
  constexpr int kAll = kThreads / (D / 4);
  const long long total = (long long)(items - a.whole) * rows;
  if (a.splits > 4)
    return launch_after(cross_join_items_kernel<D, kSoftmax, kAll>, dim3((unsigned)total), dim3(kThreads), 0, st, a,
                        per_head, rows, total);
  return launch_after(cross_join_items_kernel<D, kSoftmax, 1>, dim3((unsigned)((total + kAll - 1) / kAll)),
                      dim3(kThreads), 0, st, a, per_head, rows, total);
}

}  // namespace

cudaError_t launch_cross_join(const CrossArgs& a, avq_dtype dt, cudaStream_t st, LaunchLog& log) {
  log.add("cross_join");
  if (dt == AVQ_F32) return a.d == 64 ? join<float, 64>(a, st) : join<float, 128>(a, st);
  return a.d == 64 ? join<bf16, 64>(a, st) : join<bf16, 128>(a, st);
}

cudaError_t launch_cross_join_items(const CrossArgs& a, int items, int per_head, int rows, bool softmax,
                                    cudaStream_t st, LaunchLog& log) {
  log.add("cross_join");
  if (softmax)
    return a.d == 64 ? join_items<64, true>(a, items, per_head, rows, st)
                     : join_items<128, true>(a, items, per_head, rows, st);
  return a.d == 64 ? join_items<64, false>(a, items, per_head, rows, st)
                   : join_items<128, false>(a, items, per_head, rows, st);
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
  const auto kernel = dt == AVQ_F32 ? (a.d == 64 ? cross_delta_kernel<float, 64> : cross_delta_kernel<float, 128>)
                                    : (a.d == 64 ? cross_delta_kernel<bf16, 64> : cross_delta_kernel<bf16, 128>);
  return launch_after(kernel, dim3(grid + (a.lone != nullptr ? a.Bk : 0)), dim3(kThreads), 0, st, a, grid);
}

}  // namespace avq
