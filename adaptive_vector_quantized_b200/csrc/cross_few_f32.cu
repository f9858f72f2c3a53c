// Exact attention over another sequence for few rows per key head, 32-bit inputs:
// what the bf16 kernel for few rows does, on the CUDA cores.
//
// All rows that read one (encoder sequence, key head) are taken four at a time, so
// K and V come from memory once for four rows (from L2 for the next four); the keys
// are split over blocks (joined by a launch of its own) and over a block's 16 groups
// of eight lanes (joined in shared memory).  Bound by reading K and V.
//
// A group has one key at a time; lane t of it the elements 4 t + 32 p .. + 3 of the
// key, the value and the rows.  The lanes' parts of four scores are added in a
// butterfly that halves the rows at each step (4 shuffles, not 12), after which
// lane t holds row t / 2: one exponential a lane.  Every lane copies just the pieces
// that it reads itself into a ring in shared memory, so the loads in flight wait for
// no barrier: 32 sequences of 4096 keys, 8 key heads of 128, 4 query heads each, 158
// us (6.8 TB/s); 64-row tiles take 3.6 ms, as they compute 16 times the rows.
#include "cross.cuh"
#include "fastmath.cuh"

namespace avq {

namespace {

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;  // keys of a step
constexpr int kRows = 4;

template <int D>
struct Ring {
  static constexpr int kPieces = D / 32;                       // 16-byte pieces of a lane
  static constexpr int kStage = 2 * kPieces * kThreads;        // of K and V, in pieces
  static constexpr int kStages = D == 64 ? 8 : 4;              // 64 KB: three blocks an SM
  static constexpr int kBytes = kStages * kStage * 16;
  static_assert(kGroups * kRows * D * 4 <= kBytes, "the groups' results take the ring's place");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 3) cross_few_f32_kernel(const CrossArgs a, int chunks) {
  using R = Ring<D>;
  constexpr int P = R::kPieces;
  extern __shared__ __align__(16) float4 ring[];
  __shared__ float sM[kGroups][kRows], sZ[kGroups][kRows];
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31, group = threadIdx.x / 8, t = threadIdx.x % 8;
  const int chunk = blockIdx.x % chunks, kvh = blockIdx.x / chunks, split = blockIdx.y;
  const int kb = kvh / a.Hk, kh = kvh % a.Hk;
  const int count = key_count(a, kb);
  const int steps = (count + kGroups - 1) / kGroups;
  const int t0 = part_begin(steps, split, a.splits), t1 = part_begin(steps, split + 1, a.splits);
  const float* K = static_cast<const float*>(a.K) + kb * a.ks.b + kh * a.ks.h + 4 * t;
  const float* V = static_cast<const float*>(a.V) + kb * a.vs.b + kh * a.vs.h + 4 * t;
  const int rows = a.per_b * a.per_h * a.Nq;
  unsigned int on = 0;  // bit s: the key in stage s of the ring is looked at
  auto fetch = [&](int step) {
    if (step < t1) {
      const int key = step * kGroups + group, stage = (step - t0) % R::kStages;
      if (key_seen(a, kb, key, count)) {
        on |= 1u << stage;
        float4* to = ring + stage * R::kStage + threadIdx.x;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          tc::cp_async16(to + p * kThreads, K + key * a.ks.n + 32 * p);
          tc::cp_async16(to + (P + p) * kThreads, V + key * a.vs.n + 32 * p);
        }
      } else {
        on &= ~(1u << stage);
      }
    }
    tc::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < R::kStages - 1; ++s) fetch(t0 + s);
  float4 q[kRows][P];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = chunk * kRows + i;
    const RowAt x = row_at(a, kb, kh, r < rows ? r : 0);
    const float* Q = static_cast<const float*>(a.Q) + x.b * a.qs.b + x.h * a.qs.h + x.n * a.qs.n + 4 * t;
#pragma unroll
    for (int p = 0; p < P; ++p)
      q[i][p] = r < rows ? __ldg(reinterpret_cast<const float4*>(Q + 32 * p)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float c2 = a.scale * kLog2e;
  float m = -INFINITY, z = 0.f;  // row t / 2 of the group's keys
  float2 o[kRows][2 * P];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int p = 0; p < 2 * P; ++p) o[i][p] = fm::f2(0.f, 0.f);
  for (int step = t0; step < t1; ++step) {
    fetch(step + R::kStages - 1);  // into the place that the last step read
    tc::cp_async_wait<R::kStages - 1>();
    const int stage = (step - t0) % R::kStages;
    const float4* at = ring + stage * R::kStage + threadIdx.x;
    const bool seen = on >> stage & 1;
    float s[kRows];
    {
      float2 acc[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) acc[i] = fm::f2(0.f, 0.f);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float4 k = at[p * kThreads];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          acc[i] = fm::fma2(fm::f2(q[i][p].x, q[i][p].y), fm::f2(k.x, k.y), acc[i]);
          acc[i] = fm::fma2(fm::f2(q[i][p].z, q[i][p].w), fm::f2(k.z, k.w), acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) s[i] = acc[i].x + acc[i].y;
    }
    float x;
    {
      const bool up = lane & 4, odd = lane & 2;
      const float s0 = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 4);
      const float s1 = (up ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 4);
      x = (odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
    }
    if (!seen) x = -INFINITY;  // the ring's place holds what was there before
    // the scale in use is kept until a score is more than 2^8 above it; NaN must reach the output
    const bool grown = x != -INFINITY && !((x - m) * c2 <= 8.f);
    if (__any_sync(0xffffffffu, grown)) {
      const float keep = grown ? exp2f((m - x) * c2) : 1.f;
      if (grown) m = x;
      z *= keep;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float f = __shfl_sync(0xffffffffu, keep, (lane & 24) + 2 * i);
#pragma unroll
        for (int p = 0; p < 2 * P; ++p) o[i][p] = fm::mul2(o[i][p], fm::f2(f, f));
      }
    }
    const float w = exp2f((x - (m == -INFINITY ? 0.f : m)) * c2);
    z += w;
    float pr[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) pr[i] = __shfl_sync(0xffffffffu, w, (lane & 24) + 2 * i);
    if (seen) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float4 v = at[(P + p) * kThreads];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          o[i][2 * p] = fm::fma2(fm::f2(pr[i], pr[i]), fm::f2(v.x, v.y), o[i][2 * p]);
          o[i][2 * p + 1] = fm::fma2(fm::f2(pr[i], pr[i]), fm::f2(v.z, v.w), o[i][2 * p + 1]);
        }
      }
    }
  }
  // the groups' results, over one scale
  __syncthreads();  // the ring is read; no copy is in flight past the last step
  float* sO = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<float4*>(sO + (group * kRows + i) * D + 32 * p + 4 * t) =
          make_float4(o[i][2 * p].x, o[i][2 * p].y, o[i][2 * p + 1].x, o[i][2 * p + 1].y);
  if (t % 2 == 0) {
    sM[group][t / 2] = m;
    sZ[group][t / 2] = z;
  }
  __syncthreads();
  const int i = threadIdx.x / (D / 4), c = threadIdx.x % (D / 4) * 4, r = chunk * kRows + i;
  if (i >= kRows || r >= rows) return;
  float top = -INFINITY;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) top = fm::max3_nan(top, top, sM[g][i]);
  float sum = 0.f, out[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g = 0; g < kGroups; ++g) {
    const float mg = sM[g][i];
    if (mg == -INFINITY) continue;  // no key of this group
    const float f = exp2f((mg - top) * c2);
    const float4 v = *reinterpret_cast<const float4*>(sO + (g * kRows + i) * D + c);
    sum += f * sZ[g][i];
    out[0] += f * v.x, out[1] += f * v.y, out[2] += f * v.z, out[3] += f * v.w;
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
  for (int u = 0; u < 4; ++u) out[u] *= inv;
  const float lse = sum == 0.f ? -INFINITY : a.scale * top + logf(sum);
  const RowAt x = row_at(a, kb, kh, r);
  const size_t row = ((size_t)x.b * a.Hq + x.h) * a.Nq + x.n;
  const size_t all = (size_t)a.B * a.Hq * a.Nq;
  if (a.splits > 1) {
    put4(a.part + ((size_t)split * all + row) * D + c, out);
    if (c == 0) a.part_lse[(size_t)split * all + row] = lse;
  } else {
    put4(static_cast<float*>(a.O) + x.b * a.os.b + x.h * a.os.h + x.n * a.os.n + c, out);
    if (c == 0 && a.lse != nullptr) a.lse[row] = lse;
  }
}

template <int D>
cudaError_t run(const CrossArgs& a, cudaStream_t st) {
  const int chunks = (a.per_b * a.per_h * a.Nq + kRows - 1) / kRows;
  const cudaError_t e = allow_smem<cross_few_f32_kernel<D>>(Ring<D>::kBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.Bk * a.Hk * chunks, a.splits);
  return launch_after(cross_few_f32_kernel<D>, grid, dim3(kThreads), Ring<D>::kBytes, st, a, chunks);
}

}  // namespace

cudaError_t launch_cross_few_f32(const CrossArgs& a, cudaStream_t st, LaunchLog& log) {
  log.add("cross_few_f32");
  return a.d == 64 ? run<64>(a, st) : run<128>(a, st);
}

}  // namespace avq
