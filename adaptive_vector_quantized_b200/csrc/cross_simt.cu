// Exact attention over another sequence's keys and values, and its gradients,
// on the CUDA cores: both element types, every supported shape, and the path
// of 32-bit inputs (tensor-core products would round them to 11 bits).
//
//   S = scale Q K^T over the keys that are looked at, P = softmax(S), O = P V,
//   lse = log sum exp(S);
//   with delta = rowsum(dO O):  dS = scale P (dO V^T - delta),
//   dQ = dS K,  dK = dS^T Q,  dV = P^T dO  (dK, dV over every query head and
//   sequence that shares the key head).
// A row with no key gives O = 0, lse = -inf and dQ = 0.
//
// Tiles of 64 rows x 64 keys in shared memory as fp32; 256 threads, each 4 x 4
// scores, in fma.f32x2 (two products an instruction).  All five products read
// the tiles as they were loaded: rows against rows (S, dO V^T), rows against
// columns (P V, dS K) and columns against columns (P^T dO, dS^T Q).  Keys that
// are left out are loaded as zeros, so that infinities and NaN there meet no
// product.
//
// Bound by what shared memory hands to registers (32 values a clock and SM, each
// used by 4 of 128 products a clock: half the FMA pipe's rate).  The loads of 32-bit
// inputs run beside the products: V's beside Q K^T, the next K's beside P V, for dK
// and dV the next step's rows beside this one's (in dQ V and K take one place, one
// after the other, so that another block of the SM covers them).  24 heads of 1000
// rows and keys of 128: 406 us (30 TFLOP/s; 463 with K and V in one place, 549 with
// loads that nothing covers), gradients 1.39 ms.  8 x 4 scores a thread, with half the
// threads: 511 us where 4 x 4 took 463, as too few warps are left to cover anything.
#include "cross.cuh"
#include "fastmath.cuh"

namespace avq {

namespace {

constexpr int kT = 64;  // rows and keys of a tile
constexpr int kThreads = 256;

// 16-byte piece c of row r of a [64][W] tile: pieces of neighbouring rows lie on
// different banks
template <int W>
__device__ __forceinline__ int place(int r, int c) {
  return r * W + ((c ^ (r & 7)) << 2);
}
template <int W>
__device__ __forceinline__ float4 get4(const float* tile, int r, int c) {
  return *reinterpret_cast<const float4*>(tile + place<W>(r, c));
}

// Thread (ty, tx) of 16 x 16 has the rows ty + 16 i (in cols_cols 4 ty + i) and the
// keys tx + 16 j, or 4 columns of each 64.
constexpr int kM = 4;

// rows [first, first + 64) of a [.., n, d] tensor; rows that are not wanted are zeros
template <typename T, int D, typename F>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int64_t row_stride, int first, F&& want) {
#pragma unroll 4
  for (int e = threadIdx.x; e < kT * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (want(r)) loadE<4>(src + (int64_t)(first + r) * row_stride + 4 * c, v);
    *reinterpret_cast<float4*>(dst + place<D>(r, c)) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// load_tile under way: complete after cp_async_wait and a barrier (bf16 has to be
// converted, so its loads are complete at the barrier).
template <typename T, int D, typename F>
__device__ __forceinline__ void fetch_tile(float* dst, const T* src, int64_t row_stride, int first, F&& want) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll 4
    for (int e = threadIdx.x; e < kT * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4);
      float* to = dst + place<D>(r, c);
      if (want(r))
        tc::cp_async16(to, src + (int64_t)(first + r) * row_stride + 4 * c);
      else
        *reinterpret_cast<float4*>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  } else {
    load_tile<T, D>(dst, src, row_stride, first, want);
  }
  tc::cp_async_commit();
}

// acc[i][j] = sum_k A[ty + 16 i][k] B[tx + 16 j][k]
template <int D>
__device__ __forceinline__ void rows_rows(const float* A, const float* B, int ty, int tx, float acc[][4]) {
  float2 s[kM][4];
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = fm::f2(0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < D / 4; ++k) {
    float4 a[kM], b[4];
#pragma unroll
    for (int i = 0; i < kM; ++i) a[i] = get4<D>(A, ty + 16 * i, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = get4<D>(B, tx + 16 * j, k);
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fm::fma2(fm::f2(a[i].x, a[i].y), fm::f2(b[j].x, b[j].y), s[i][j]);
        s[i][j] = fm::fma2(fm::f2(a[i].z, a[i].w), fm::f2(b[j].z, b[j].w), s[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// A score of the tile: row r, key j
__device__ __forceinline__ float& score(float* tile, int r, int j) { return tile[place<kT>(r, j >> 2) + (j & 3)]; }

// acc[i][c] += sum_k A[ty + 16 i][k] B[k][4 tx + 64 c ..]  (A: score tile)
template <int D>
__device__ __forceinline__ void rows_cols(const float* A, const float* B, int ty, int tx, float2 acc[][D / 32]) {
#pragma unroll 2
  for (int k = 0; k < kT / 4; ++k) {
    float4 a[kM];
#pragma unroll
    for (int i = 0; i < kM; ++i) a[i] = get4<kT>(A, ty + 16 * i, k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 v = get4<D>(B, 4 * k + kk, tx + 16 * c);
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          const float x = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
          acc[i][2 * c] = fm::fma2(fm::f2(x, x), fm::f2(v.x, v.y), acc[i][2 * c]);
          acc[i][2 * c + 1] = fm::fma2(fm::f2(x, x), fm::f2(v.z, v.w), acc[i][2 * c + 1]);
        }
      }
    }
  }
}

// acc[i][c] += sum_k A[k][kM ty + i] B[k][4 tx + 64 c ..]  (A: score tile)
template <int D>
__device__ __forceinline__ void cols_cols(const float* A, const float* B, int ty, int tx, float2 acc[][D / 32]) {
#pragma unroll 4
  for (int k = 0; k < kT; ++k) {
    const float4 a = get4<kT>(A, k, ty);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float4 v = get4<D>(B, k, tx + 16 * c);
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        const float x = i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : a.w;
        acc[i][2 * c] = fm::fma2(fm::f2(x, x), fm::f2(v.x, v.y), acc[i][2 * c]);
        acc[i][2 * c + 1] = fm::fma2(fm::f2(x, x), fm::f2(v.z, v.w), acc[i][2 * c + 1]);
      }
    }
  }
}

template <int C>
__device__ __forceinline__ void clear(float2 (&acc)[kM][C]) {
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[i][c] = fm::f2(0.f, 0.f);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) cross_simt_kernel(const CrossArgs a) {
  grid_dependency_wait();
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sQ + kT * D;
  float* sV = sK + kT * D;
  float* sP = sV + kT * D;
  __shared__ unsigned char seen[2][kT];
  const int tiles = (a.Nq + kT - 1) / kT;
  const int rt = blockIdx.x % tiles, bh = blockIdx.x / tiles, split = blockIdx.y;
  const int b = bh / a.Hq, h = bh % a.Hq;
  const int kb = b / a.per_b, kh = h / a.per_h;
  const int count = key_count(a, kb);
  const int ktiles = (count + kT - 1) / kT;
  const int t0 = part_begin(ktiles, split, a.splits), t1 = part_begin(ktiles, split + 1, a.splits);
  const int row0 = rt * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const T* Q = static_cast<const T*>(a.Q) + b * a.qs.b + h * a.qs.h;
  const T* K = static_cast<const T*>(a.K) + kb * a.ks.b + kh * a.ks.h;
  const T* V = static_cast<const T*>(a.V) + kb * a.vs.b + kh * a.vs.h;
  fetch_tile<T, D>(sQ, Q, a.qs.n, row0, [&](int r) { return row0 + r < a.Nq; });
  auto look = [&](int t) {
    if (threadIdx.x < kT && t < t1) seen[t & 1][threadIdx.x] = key_seen(a, kb, t * kT + threadIdx.x, count);
  };
  look(t0);
  __syncthreads();
  if (t0 < t1) fetch_tile<T, D>(sK, K, a.ks.n, t0 * kT, [&](int r) { return seen[t0 & 1][r] != 0; });
  const float c2 = a.scale * kLog2e;
  float m[kM], z[kM];
  float2 o[kM][D / 32];
  clear(o);
#pragma unroll
  for (int i = 0; i < kM; ++i) m[i] = -INFINITY, z[i] = 0.f;
  for (int t = t0; t < t1; ++t) {
    const unsigned char* on = seen[t & 1];
    tc::cp_async_wait<0>();
    __syncthreads();  // K is here; the last trip has read V and P
    fetch_tile<T, D>(sV, V, a.vs.n, t * kT, [&](int r) { return on[r] != 0; });
    look(t + 1);
    float s[kM][4];
    rows_rows<D>(sQ, sK, ty, tx, s);
#pragma unroll
    for (int i = 0; i < kM; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!on[tx + 16 * j]) s[i][j] = -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mn = fmaxf(m[i], top);
      const float base = mn == -INFINITY ? 0.f : mn * c2;
      const float keep = m[i] == -INFINITY ? 0.f : exp2f(m[i] * c2 - base);
      z[i] *= keep;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(fmaf(s[i][j], c2, -base));
        z[i] += s[i][j];
        score(sP, ty + 16 * i, tx + 16 * j) = s[i][j];
      }
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[i][c] = fm::mul2(o[i][c], fm::f2(keep, keep));
    }
    tc::cp_async_wait<0>();
    __syncthreads();  // V and P are here; K has been read
    if (t + 1 < t1)
      fetch_tile<T, D>(sK, K, a.ks.n, (t + 1) * kT, [&](int r) { return seen[(t + 1) & 1][r] != 0; });
    rows_cols<D>(sP, sV, ty, tx, o);
  }
  tc::cp_async_wait<0>();  // without steps Q is still under way
#pragma unroll
  for (int i = 0; i < kM; ++i)
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) z[i] += __shfl_xor_sync(0xffffffffu, z[i], w);
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int r = row0 + ty + 16 * i;
    if (r >= a.Nq) continue;
    const float inv = z[i] > 0.f ? 1.f / z[i] : (z[i] == 0.f ? 0.f : z[i]);  // NaN stays NaN
    const float lse = z[i] == 0.f ? -INFINITY : a.scale * m[i] + logf(z[i]);
    const size_t row = ((size_t)b * a.Hq + h) * a.Nq + r;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float v[4] = {o[i][2 * c].x * inv, o[i][2 * c].y * inv, o[i][2 * c + 1].x * inv, o[i][2 * c + 1].y * inv};
      if (a.splits > 1)
        put4(a.part + ((size_t)split * a.B * a.Hq * a.Nq + row) * D + 4 * tx + 64 * c, v);
      else
        put4(static_cast<T*>(a.O) + b * a.os.b + h * a.os.h + r * a.os.n + 4 * tx + 64 * c, v);
    }
    if (tx == 0) {
      if (a.splits > 1)
        a.part_lse[(size_t)split * a.B * a.Hq * a.Nq + row] = lse;
      else if (a.lse != nullptr)
        a.lse[row] = lse;
    }
  }
}

// From Q K^T and dO V^T of a tile pair: P and dS of the rows ty + 16 i, keys tx + 16 j.
__device__ __forceinline__ void scores_back(const float* sL, const float* sDelta, const unsigned char* seen, int ty,
                                            int tx, float c2, float scale, float p[][4], float ds[][4]) {
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const float l = sL[ty + 16 * i], dl = sDelta[ty + 16 * i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool on = seen[tx + 16 * j] != 0 && l != -INFINITY;
      p[i][j] = on ? exp2f(fmaf(p[i][j], c2, -l)) : 0.f;
      ds[i][j] = on ? p[i][j] * (ds[i][j] - dl) * scale : 0.f;
    }
  }
}

// log-sum-exp (in base 2) and delta of a row tile; rows past the end get +inf (P = 0)
__device__ __forceinline__ void load_rows(const CrossArgs& a, float* sL, float* sDelta, size_t head_row, int row0) {
  if (threadIdx.x < kT) {
    const int r = row0 + threadIdx.x;
    sL[threadIdx.x] = r < a.Nq ? a.lse[head_row + r] * kLog2e : INFINITY;
    sDelta[threadIdx.x] = r < a.Nq ? a.delta[head_row + r] : 0.f;
  }
}

// At d = 128 one block fits an SM either way, with room for the next step's rows; at
// 64 two blocks do without it.
template <int D>
constexpr int kRowBufs = D == 64 ? 1 : 2;

// block, split: of the key tiles and of their ranges of rows
template <typename T, int D>
__device__ __forceinline__ void form_dkv(float* sm, const CrossArgs& a, int block, int split) {
  float* sK = sm;
  float* sV = sK + kT * D;
  constexpr int N = kRowBufs<D>;
  float* rows = sV + kT * D;  // Q and dO, of this step and with two places of the next
  float* sP = rows + N * 2 * kT * D;
  float* sD = sP + kT * kT;
  __shared__ float sL[N][kT], sDelta[N][kT];
  __shared__ unsigned char seen[kT];
  const int tiles = (a.Nk + kT - 1) / kT;
  const int kt = block % tiles, bh = block / tiles;
  const int kb = bh / a.Hk, kh = bh % a.Hk;
  const int R = a.per_b, G = a.per_h;
  const int k0 = kt * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int count = key_count(a, kb);
  if (threadIdx.x < kT) seen[threadIdx.x] = key_seen(a, kb, k0 + threadIdx.x, count);
  __syncthreads();
  fetch_tile<T, D>(sK, static_cast<const T*>(a.K) + kb * a.ks.b + kh * a.ks.h, a.ks.n, k0,
                  [&](int r) { return seen[r] != 0; });
  fetch_tile<T, D>(sV, static_cast<const T*>(a.V) + kb * a.vs.b + kh * a.vs.h, a.vs.n, k0,
                  [&](int r) { return seen[r] != 0; });
  const float c2 = a.scale * kLog2e;
  float2 dk[kM][D / 32], dv[kM][D / 32];
  clear(dk);
  clear(dv);
  const int rtiles = (a.Nq + kT - 1) / kT;
  const int all = R * G * rtiles;
  const int i0 = part_begin(all, split, a.splits), i1 = k0 < count ? part_begin(all, split + 1, a.splits) : i0;
  auto fetch = [&](int it) {
    if (it >= i1) return;
    const int row0 = it % rtiles * kT, rg = it / rtiles, place = (it - i0) % N;
    const int b = kb * R + rg / G, h = kh * G + rg % G;
    float* to = rows + place * 2 * kT * D;
    auto in = [&](int r) { return row0 + r < a.Nq; };
    fetch_tile<T, D>(to, static_cast<const T*>(a.Q) + b * a.qs.b + h * a.qs.h, a.qs.n, row0, in);
    fetch_tile<T, D>(to + kT * D, static_cast<const T*>(a.G) + b * a.gs.b + h * a.gs.h, a.gs.n, row0, in);
    load_rows(a, sL[place], sDelta[place], ((size_t)b * a.Hq + h) * a.Nq, row0);
  };
  if (N > 1) fetch(i0);
  for (int it = i0; it < i1; ++it) {
    const int place = (it - i0) % N;
    const float *sQ = rows + place * 2 * kT * D, *sG = sQ + kT * D;
    if (N == 1) {
      __syncthreads();  // the last trip has read the rows
      fetch(it);
    }
    tc::cp_async_wait<0>();
    __syncthreads();  // this step's rows are here; the last trip has read its own and P and dS
    if (N > 1) fetch(it + 1);
    float p[kM][4], ds[kM][4];
    rows_rows<D>(sQ, sK, ty, tx, p);
    rows_rows<D>(sG, sV, ty, tx, ds);
    scores_back(sL[place], sDelta[place], seen, ty, tx, c2, a.scale, p, ds);
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        score(sP, ty + 16 * i, tx + 16 * j) = p[i][j];
        score(sD, ty + 16 * i, tx + 16 * j) = ds[i][j];
      }
    __syncthreads();
    cols_cols<D>(sP, sG, ty, tx, dv);
    cols_cols<D>(sD, sQ, ty, tx, dk);
  }
  tc::cp_async_wait<0>();  // without steps K and V are still under way
  const size_t elems = (size_t)a.Bk * a.Hk * a.Nk * D;
  const bool lone = lone_key(a, kb, count);
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int r = k0 + kM * ty + i;
    if (r >= a.Nk) continue;
    const size_t at = (((size_t)kb * a.Hk + kh) * a.Nk + r) * D;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float k4[4] = {dk[i][2 * c].x, dk[i][2 * c].y, dk[i][2 * c + 1].x, dk[i][2 * c + 1].y};
      float v4[4] = {dv[i][2 * c].x, dv[i][2 * c].y, dv[i][2 * c + 1].x, dv[i][2 * c + 1].y};
      if (!seen[kM * ty + i]) {  // whatever the rows held
#pragma unroll
        for (int e = 0; e < 4; ++e) k4[e] = v4[e] = 0.f;
      }
      if (lone) {
#pragma unroll
        for (int e = 0; e < 4; ++e) k4[e] *= 0.f;  // NaN stays
      }
      if (a.splits > 1) {
        put4(a.part + (size_t)split * 2 * elems + at + 4 * tx + 64 * c, k4);
        put4(a.part + ((size_t)split * 2 + 1) * elems + at + 4 * tx + 64 * c, v4);
      } else {
        put4(static_cast<T*>(a.dK) + at + 4 * tx + 64 * c, k4);
        put4(static_cast<T*>(a.dV) + at + 4 * tx + 64 * c, v4);
      }
    }
  }
}

// block, split: of the row tiles and of their ranges of keys
template <typename T, int D>
__device__ __forceinline__ void form_dq(float* sm, const CrossArgs& a, int block, int split) {
  float* sKV = sm;  // V, then K
  float* sQ = sKV + kT * D;
  float* sG = sQ + kT * D;
  float* sD = sG + kT * D;
  __shared__ float sL[kT], sDelta[kT];
  __shared__ unsigned char seen[kT];
  const int tiles = (a.Nq + kT - 1) / kT;
  const int rt = block % tiles, bh = block / tiles;
  const int b = bh / a.Hq, h = bh % a.Hq;
  const int kb = b / a.per_b, kh = h / a.per_h;
  const int row0 = rt * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int count = key_count(a, kb);
  const int ktiles = (count + kT - 1) / kT;
  const int t0 = part_begin(ktiles, split, a.splits), t1 = part_begin(ktiles, split + 1, a.splits);
  load_tile<T, D>(sQ, static_cast<const T*>(a.Q) + b * a.qs.b + h * a.qs.h, a.qs.n, row0,
                  [&](int r) { return row0 + r < a.Nq; });
  load_tile<T, D>(sG, static_cast<const T*>(a.G) + b * a.gs.b + h * a.gs.h, a.gs.n, row0,
                  [&](int r) { return row0 + r < a.Nq; });
  const size_t head_row = ((size_t)b * a.Hq + h) * a.Nq;
  load_rows(a, sL, sDelta, head_row, row0);
  const T* K = static_cast<const T*>(a.K) + kb * a.ks.b + kh * a.ks.h;
  const T* V = static_cast<const T*>(a.V) + kb * a.vs.b + kh * a.vs.h;
  const float c2 = a.scale * kLog2e;
  float2 dq[kM][D / 32];
  clear(dq);
  for (int t = t0; t < t1; ++t) {
    const int k0 = t * kT;
    __syncthreads();
    if (threadIdx.x < kT) seen[threadIdx.x] = key_seen(a, kb, k0 + threadIdx.x, count);
    __syncthreads();
    load_tile<T, D>(sKV, V, a.vs.n, k0, [&](int r) { return seen[r] != 0; });
    __syncthreads();
    float p[kM][4], ds[kM][4];
    rows_rows<D>(sG, sKV, ty, tx, ds);
    __syncthreads();
    load_tile<T, D>(sKV, K, a.ks.n, k0, [&](int r) { return seen[r] != 0; });
    __syncthreads();
    rows_rows<D>(sQ, sKV, ty, tx, p);
    scores_back(sL, sDelta, seen, ty, tx, c2, a.scale, p, ds);
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) score(sD, ty + 16 * i, tx + 16 * j) = ds[i][j];
    __syncthreads();
    rows_cols<D>(sD, sKV, ty, tx, dq);
  }
  const bool lone = lone_key(a, kb, count);
#pragma unroll
  for (int i = 0; i < kM; ++i) {
    const int r = row0 + ty + 16 * i;
    if (r >= a.Nq) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float v[4] = {dq[i][2 * c].x, dq[i][2 * c].y, dq[i][2 * c + 1].x, dq[i][2 * c + 1].y};
      if (lone) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= 0.f;  // NaN stays
      }
      const size_t at = (head_row + r) * D + 4 * tx + 64 * c;
      if (a.splits > 1)
        put4(a.part + (size_t)split * a.B * a.Hq * a.Nq * D + at, v);
      else
        put4(static_cast<T*>(a.dQ) + at, v);
    }
  }
}

// d = 64: the first `keys` blocks form dK and dV (key_tiles of them to a split), the
// others dQ with the arguments q (row_tiles to a split), on the places that those
// leave.  One launch, since a kernel for dQ that started beside the other would read
// delta before its own wait for the work before it, and nothing else makes another
// kernel's writes visible.  12 heads of 1001 rows over 333 keys: 96 us, 134 with a
// launch for each.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) cross_simt_backward_kernel(const CrossArgs a, const CrossArgs q,
                                                                         int key_tiles, int keys, int row_tiles) {
  grid_dependency_wait();
  extern __shared__ __align__(16) float sm[];
  const int block = blockIdx.x;
  if (block < keys)
    form_dkv<T, 64>(sm, a, block % key_tiles, block / key_tiles);
  else
    form_dq<T, 64>(sm, q, (block - keys) % row_tiles, (block - keys) / row_tiles);
}
// d = 128: dK and dV take all of an SM's shared memory, dQ half of it, so that one
// launch would leave dQ one block an SM: a launch for each.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1) cross_simt_dkv_kernel(const CrossArgs a) {
  grid_dependency_wait();
  allow_dependents();
  extern __shared__ __align__(16) float sm[];
  form_dkv<T, 128>(sm, a, blockIdx.x, blockIdx.y);
}
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) cross_simt_dq_kernel(const CrossArgs a) {
  grid_dependency_wait();
  extern __shared__ __align__(16) float sm[];
  form_dq<T, 128>(sm, a, blockIdx.x, blockIdx.y);
}

template <typename T, int D>
cudaError_t forward(const CrossArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(3 * kT * D + kT * kT) * sizeof(float);
  cudaError_t e = allow_smem<cross_simt_kernel<T, D>>((int)smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)a.B * a.Hq * ((a.Nq + kT - 1) / kT)), a.splits);
  return launch_after(cross_simt_kernel<T, D>, grid, dim3(kThreads), smem, st, a);
}
template <typename T, int D>
cudaError_t backward(const CrossArgs& a, const CrossArgs& q, cudaStream_t st, LaunchLog& log) {
  const int dkv_smem = ((2 + 2 * kRowBufs<D>) * kT * D + 2 * kT * kT) * (int)sizeof(float);
  const int dq_smem = (3 * kT * D + kT * kT) * (int)sizeof(float);
  const unsigned key_tiles = (unsigned)((long long)a.Bk * a.Hk * ((a.Nk + kT - 1) / kT));
  const unsigned row_tiles = (unsigned)((long long)a.B * a.Hq * ((a.Nq + kT - 1) / kT));
  cudaError_t e;
  if constexpr (D == 64) {
    static_assert(kRowBufs<64> == 1, "dK and dV take more shared memory than dQ");
    log.add("cross_simt_backward");
    e = allow_smem<cross_simt_backward_kernel<T>>(dkv_smem);
    if (e != cudaSuccess) return e;
    const unsigned keys = key_tiles * a.splits;
    return launch_after(cross_simt_backward_kernel<T>, dim3(keys + row_tiles * q.splits), dim3(kThreads), dkv_smem,
                        st, a, q, (int)(key_tiles > 0 ? key_tiles : 1), (int)keys, (int)row_tiles);
  } else {
    if (key_tiles > 0) {
      log.add("cross_simt_dkv");
      e = allow_smem<cross_simt_dkv_kernel<T>>(dkv_smem);
      if (e == cudaSuccess)
        e = launch_after(cross_simt_dkv_kernel<T>, dim3(key_tiles, a.splits), dim3(kThreads), dkv_smem, st, a);
      if (e != cudaSuccess) return e;
    }
    log.add("cross_simt_dq");
    e = allow_smem<cross_simt_dq_kernel<T>>(dq_smem);
    if (e != cudaSuccess) return e;
    return launch_after(cross_simt_dq_kernel<T>, dim3(row_tiles, q.splits), dim3(kThreads), dq_smem, st, q);
  }
}

}  // namespace

cudaError_t launch_cross_simt(const CrossArgs& a, avq_dtype dt, cudaStream_t st, LaunchLog& log) {
  log.add("cross_simt");
  if (dt == AVQ_F32) return a.d == 64 ? forward<float, 64>(a, st) : forward<float, 128>(a, st);
  return a.d == 64 ? forward<bf16, 64>(a, st) : forward<bf16, 128>(a, st);
}
cudaError_t launch_cross_simt_backward(const CrossArgs& a, const CrossArgs& q, avq_dtype dt, cudaStream_t st,
                                       LaunchLog& log) {
  if (dt == AVQ_F32) return a.d == 64 ? backward<float, 64>(a, q, st, log) : backward<float, 128>(a, q, st, log);
  return a.d == 64 ? backward<bf16, 64>(a, q, st, log) : backward<bf16, 128>(a, q, st, log);
}

}  // namespace avq
