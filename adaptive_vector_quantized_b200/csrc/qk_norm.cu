// Norms of queries and keys per head with the rotation by position in the same
// pass, the rotation alone, and the gradients.
//
// For one head vector x of d elements (RMS or LayerNorm, then the rotation):
//   u = x / sqrt(mean(x^2) + eps)            (RMS)
//   u = (x - mean(x)) / sqrt(var(x) + eps)   (LayerNorm)
//   y = R (u w + b)
// R turns each of rot / 2 pairs of elements by the angle position * frequency
// and scales it by mscale; elements past rot stay.  Backwards, with z = R^T dy
// and g = z w:
//   dw = sum z u,  db = sum z,
//   dx = (g - u mean(g u) [- mean(g) for LayerNorm]) / sqrt(...),
// u recomputed from x, so the forward pass keeps nothing.
//
// Angles are products in 64 bits, reduced to a fraction of a turn before the
// rounding to 32 bits: at position 10^6 a 32-bit angle would be off by 0.06.
//
// The kernels are bound by memory: each element is read once and written
// once.  A head is spread over d / 8 lanes of 8 elements, as two groups of 4
// that hold both elements of every pair in either layout, so the rotation
// needs no exchange between lanes and the norm 3 or 4 butterfly shuffles.
// Sine and cosine are computed once per token and block (a table in shared
// memory) and kept in registers over the token's heads.
#include "common.cuh"
#include "internal.h"

namespace avq {

namespace {

constexpr int kThreads = 256;
// Heads of a token that a lane group has under way at a time: 64 bytes of each
// lane's loads, requested while the heads before are worked on.
template <typename T>
constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;

struct Params {
  const void* x[2];  // queries, keys
  const void* g[2];  // their outputs' gradients (backward)
  void* y[2];        // outputs, or the gradients of x
  const void* w[2];
  const void* b[2];
  Strides xs[2], gs[2];
  int H[2];
  const int32_t* pos;
  const double* freqs;
  float* part;  // weight gradients per block: [2][blocks][2][d]
  int tokens, N, rot, axes, pos_batch;
  int tb;  // tokens of one block's tile (a power of two)
  float eps, mscale, sign;
};

template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v);
template <>
__device__ __forceinline__ void store4<float>(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store4<bf16>(bf16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// A lane's 8 elements of a head as they stand in memory, each group of 4 by itself.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x, int ia, int ib) {
    a = __ldg(reinterpret_cast<const float4*>(x + ia));
    b = __ldg(reinterpret_cast<const float4*>(x + ib));
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw<bf16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const bf16* x, int ia, int ib) {
    a = __ldg(reinterpret_cast<const uint2*>(x + ia));
    b = __ldg(reinterpret_cast<const uint2*>(x + ib));
  }
  __device__ __forceinline__ void clear() { a = b = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(b.x), v[5] = bf16_hi(b.x), v[6] = bf16_lo(b.y), v[7] = bf16_hi(b.y);
  }
};

// Weights and biases of queries and keys in shared memory as fp32 (1 and 0 where absent).
template <typename T, int D>
__device__ __forceinline__ void fill_weights(const Params& p, float* sw, float* sb) {
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const int which = i / D, c = i % D;
    const T* w = static_cast<const T*>(p.w[which]);
    const T* b = static_cast<const T*>(p.b[which]);
    sw[i] = w != nullptr ? static_cast<float>(w[c]) : 1.f;
    sb[i] = b != nullptr ? static_cast<float>(b[c]) : 0.f;
  }
}
__device__ __forceinline__ void get8(const float* s, int ia, int ib, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(s + ia), b = *reinterpret_cast<const float4*>(s + ib);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosine and sine (times mscale; sine with the rotation's sign) of every
// pair of the tile's tokens.
__device__ __forceinline__ void fill_table(const Params& p, float2* tab, int first) {
  const int half = p.rot >> 1;
  const int per_axis = p.axes == 2 ? half >> 1 : half;
  for (int e = threadIdx.x; e < p.tb * half; e += kThreads) {
    const int t = e / half, i = e - t * half;
    const int tok = first + t;
    if (tok >= p.tokens) break;
    const int n = tok % p.N;
    int at = n;
    if (p.pos != nullptr) {
      const long long row = p.pos_batch ? tok : n;
      at = __ldg(p.pos + row * p.axes + (i >= per_axis ? 1 : 0));
    }
    const double turns = (double)at * (__ldg(p.freqs + i) * 0.15915494309189533577);  // / 2 pi
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    tab[e] = make_float2(c * p.mscale, s * p.mscale * p.sign);
  }
}

// Places of a lane's two groups of 4 elements and whether they are rotated.
template <bool kHalf>
__device__ __forceinline__ bool places(int lane, int rot, int& a, int& b) {
  const bool turned = lane < (rot >> 3);
  if (kHalf && turned) {
    a = 4 * lane;
    b = (rot >> 1) + 4 * lane;
  } else {
    a = 8 * lane;
    b = a + 4;
  }
  return turned;
}

// v: the lane's elements (group a, then group b); cs: its four pairs' cosine and sine.
template <bool kHalf>
__device__ __forceinline__ void turn(float* v, const float2* cs) {
  if constexpr (kHalf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[i], b = v[4 + i];
      v[i] = a * cs[i].x - b * cs[i].y;
      v[4 + i] = b * cs[i].x + a * cs[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * cs[i].x - b * cs[i].y;
      v[2 * i + 1] = b * cs[i].x + a * cs[i].y;
    }
  }
}

// v <- u, returns 1 / sqrt(...)
template <int D, int kNorm>
__device__ __forceinline__ float normalise(float* v, float eps) {
  constexpr int L = D / 8;
  if constexpr (kNorm == AVQ_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
    const float mean = group_sum<L>(s) * (1.f / D);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) q += v[i] * v[i];
  const float r = rsqrtf(group_sum<L>(q) * (1.f / D) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= r;
  return r;
}

template <typename T, int D, int kNorm, bool kHalf>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_kernel(const Params p) {
  constexpr int L = D / 8, G = kThreads / L, U = kBatch<T>;
  __shared__ __align__(16) float2 tab[G * D / 2];
  __shared__ __align__(16) float sw[kNorm == AVQ_NORM_NONE ? 4 : 2 * D], sb[kNorm == AVQ_NORM_NONE ? 4 : 2 * D];
  const int first = blockIdx.x * p.tb;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int t = group & (p.tb - 1), slot = group / p.tb, slots = G / p.tb;
  const int tok = first + t;
  const bool in = tok < p.tokens;  // whole groups: the shuffles still run
  const int b = in ? tok / p.N : 0, n = in ? tok % p.N : 0;
  int ia, ib;
  const bool turned = places<kHalf>(lane, p.rot, ia, ib);
  // batches of U heads: the queries' first, then the keys' (the same number for every group)
  const int per = slots * U;
  const int qb = (p.H[0] + per - 1) / per, all = qb + (p.H[1] + per - 1) / per;
  Raw<T> raw[2][U];
  auto request = [&](int i, Raw<T>* r) {
    const int which = i >= qb, h0 = (which ? i - qb : i) * per + slot;
    const T* x = static_cast<const T*>(p.x[which]) + b * p.xs[which].b + n * p.xs[which].n;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + k * slots;
      if (in && h < p.H[which]) r[k].load(x + h * p.xs[which].h, ia, ib);
      else r[k].clear();
    }
  };
  float2 cs[4];
  auto finish = [&](int i, const Raw<T>* r) {
    const int which = i >= qb, h0 = (which ? i - qb : i) * per + slot;
    const int H = p.H[which];
    T* y = static_cast<T*>(p.y[which]) + ((long long)b * H * p.N + n) * D;
    float w[8], bias[8];
    if constexpr (kNorm != AVQ_NORM_NONE) {
      get8(sw + which * D, ia, ib, w);
      get8(sb + which * D, ia, ib, bias);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + k * slots;
      float v[8];
      r[k].get(v);
      if constexpr (kNorm != AVQ_NORM_NONE) {
        normalise<D, kNorm>(v, p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * w[e] + bias[e];
      }
      if (turned) turn<kHalf>(v, cs);
      if (in && h < H) {
        store4(y + (long long)h * p.N * D + ia, v);
        store4(y + (long long)h * p.N * D + ib, v + 4);
      }
    }
  };
  request(0, raw[0]);  // under way while the table is made
  fill_table(p, tab, first);
  if constexpr (kNorm != AVQ_NORM_NONE) fill_weights<T, D>(p, sw, sb);
  __syncthreads();
  if (turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = tab[t * (p.rot >> 1) + 4 * lane + i];
  }
  for (int i = 0; i < all; i += 2) {
    if (i + 1 < all) request(i + 1, raw[1]);
    finish(i, raw[0]);
    if (i + 1 < all) {
      if (i + 2 < all) request(i + 2, raw[0]);
      finish(i + 1, raw[1]);
    }
  }
}

// Gradients.  blockIdx.y: queries or keys; each block walks tiles and keeps
// its share of the weight gradients in registers, summed over its groups at
// the end in a fixed order.
template <typename T, int D, int kNorm, bool kHalf>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_backward_kernel(const Params p, int tiles) {
  constexpr int L = D / 8, G = kThreads / L, U = kBatch<T> / 2;
  __shared__ __align__(16) float2 tab[2][G * D / 2];
  __shared__ float sums[G][D];
  const int which = blockIdx.y;
  const int H = p.H[which];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int t = group & (p.tb - 1), slot = group / p.tb, slots = G / p.tb;
  int ia, ib;
  const bool turned = places<kHalf>(lane, p.rot, ia, ib);
  const Strides xs = p.xs[which], gs = p.gs[which];
  float w[8], dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, dw[i] = 0.f, db[i] = 0.f;
  if (p.w[which] != nullptr) {
    loadE<4>(static_cast<const T*>(p.w[which]) + ia, w);
    loadE<4>(static_cast<const T*>(p.w[which]) + ib, w + 4);
  }
  // batches of U heads of a tile's tokens, tile after tile
  const int per = slots * U, batches = (H + per - 1) / per;
  Raw<T> rx[2][U], rg[2][U];
  auto request = [&](int tile, int i, Raw<T>* x, Raw<T>* g) {
    const int tok = tile * p.tb + t;
    const bool in = tok < p.tokens;
    const int b = in ? tok / p.N : 0, n = in ? tok % p.N : 0;
    const T* px = static_cast<const T*>(p.x[which]) + b * xs.b + n * xs.n;
    const T* pg = static_cast<const T*>(p.g[which]) + b * gs.b + n * gs.n;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = i * per + k * slots + slot;
      if (in && h < H) {
        x[k].load(px + h * xs.h, ia, ib);
        g[k].load(pg + h * gs.h, ia, ib);
      } else {
        x[k].clear();
        g[k].clear();
      }
    }
  };
  float2 cs[4];
  auto finish = [&](int tile, int i, const Raw<T>* rx, const Raw<T>* rg) {
    const int tok = tile * p.tb + t;
    const bool in = tok < p.tokens;
    const int b = in ? tok / p.N : 0, n = in ? tok % p.N : 0;
    T* y = static_cast<T*>(p.y[which]) + ((long long)b * H * p.N + n) * D;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = i * per + k * slots + slot;
      const bool live = in && h < H;
      float u[8], z[8];
      rx[k].get(u);
      rg[k].get(z);
      if (turned) turn<kHalf>(z, cs);
      const float r = normalise<D, kNorm>(u, p.eps);
      float gu = 0.f, gm = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (live) {  // an absent row's u is 0 / 0 when eps is 0
          dw[e] += z[e] * u[e];
          db[e] += z[e];
        }
        z[e] *= w[e];
        gu += z[e] * u[e];
        gm += z[e];
      }
      gu = group_sum<L>(gu) * (1.f / D);
      gm = kNorm == AVQ_NORM_LAYER ? group_sum<L>(gm) * (1.f / D) : 0.f;
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = (z[e] - gm - u[e] * gu) * r;
        store4(y + (long long)h * p.N * D + ia, z);
        store4(y + (long long)h * p.N * D + ib, z + 4);
      }
    }
  };
  // the batch after (tile, i)
  auto next = [&](int& tile, int& i) {
    if (++i == batches) {
      i = 0;
      tile += gridDim.x;
    }
  };
  int tile = blockIdx.x, i = 0, made = 0;
  if (tile < tiles) request(tile, i, rx[0], rg[0]);
  // one turn of the loop handles two batches, so that the buffers' places are known
  auto turn_of = [&](int cur) {
    int nt = tile, ni = i;
    next(nt, ni);
    if (nt < tiles) request(nt, ni, rx[cur ^ 1], rg[cur ^ 1]);
    if (i == 0) {  // a new tile: its sines and cosines, in the table that no one reads any more
      fill_table(p, tab[made & 1], tile * p.tb);
      __syncthreads();
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = tab[made & 1][t * (p.rot >> 1) + 4 * lane + e];
      }
      ++made;
    }
    finish(tile, i, rx[cur], rg[cur]);
    tile = nt;
    i = ni;
  };
  while (tile < tiles) {
    turn_of(0);
    if (tile < tiles) turn_of(1);
  }
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sums[group][ia + i] = kind == 0 ? dw[i] : db[i];
      sums[group][ib + i] = kind == 0 ? dw[4 + i] : db[4 + i];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
      for (int k = 0; k < G; ++k) s += sums[k][threadIdx.x];
      p.part[(((size_t)which * gridDim.x + blockIdx.x) * 2 + kind) * D + threadIdx.x] = s;
    }
  }
}

// Weight gradients: the blocks' shares added up in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float* part, int blocks, float* dwq, float* dbq,
                                                          float* dwk, float* dbk) {
  __shared__ float s[1024 / D][D];
  grid_dependency_wait();
  float* const outs[4] = {dwq, dbq, dwk, dbk};
  float* out = outs[blockIdx.x];
  if (out == nullptr) return;
  const int which = blockIdx.x >> 1, kind = blockIdx.x & 1;
  const int c = threadIdx.x % D, r = threadIdx.x / D;
  float v = 0.f;
  for (int i = r; i < blocks; i += 1024 / D) v += part[(((size_t)which * blocks + i) * 2 + kind) * D + c];
  s[r][c] = v;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 1024 / D; ++i) v += s[i][c];
    out[c] = v;
  }
}

int groups_of(int d) { return kThreads / (d / 8); }

// Tokens per tile: as many as fit the block's lane groups (sine and cosine
// are then shared by the token's heads alone), fewer while the tiles would
// leave SMs idle; the freed groups share the token's heads.
int tile_tokens(int d, int tokens) {
  int tb = groups_of(d);
  while (tb > 1 && (tokens + tb - 1) / tb < 2 * num_sms()) tb >>= 1;
  return tb;
}

Params params_of(const avq_qk_dims& s, const Strides* xs, const int32_t* pos, const double* freqs) {
  Params p{};
  p.H[0] = s.Hq;
  p.H[1] = s.Hk;
  p.xs[0] = xs[0];
  p.xs[1] = xs[1];
  p.pos = pos;
  p.freqs = freqs;
  p.tokens = s.B * s.N;
  p.N = s.N;
  p.rot = s.rot;
  p.axes = s.axes;
  p.pos_batch = s.pos_batch;
  p.eps = s.eps;
  p.mscale = s.mscale;
  p.sign = 1.f;
  p.tb = tile_tokens(s.d, p.tokens);
  return p;
}

template <typename T, int D, int kNorm>
void launch_fwd(const Params& p, bool half, int tiles, cudaStream_t st) {
  if (half)
    qk_norm_kernel<T, D, kNorm, true><<<tiles, kThreads, 0, st>>>(p);
  else
    qk_norm_kernel<T, D, kNorm, false><<<tiles, kThreads, 0, st>>>(p);
}
template <typename T, int D>
void launch_fwd_norm(const Params& p, int norm, bool half, int tiles, cudaStream_t st) {
  if (norm == AVQ_NORM_NONE) return launch_fwd<T, D, AVQ_NORM_NONE>(p, half, tiles, st);
  if (norm == AVQ_NORM_RMS) return launch_fwd<T, D, AVQ_NORM_RMS>(p, half, tiles, st);
  return launch_fwd<T, D, AVQ_NORM_LAYER>(p, half, tiles, st);
}
template <typename T, int D, int kNorm>
void launch_bwd(const Params& p, bool half, int tiles, dim3 grid, cudaStream_t st) {
  if (half)
    qk_norm_backward_kernel<T, D, kNorm, true><<<grid, kThreads, 0, st>>>(p, tiles);
  else
    qk_norm_backward_kernel<T, D, kNorm, false><<<grid, kThreads, 0, st>>>(p, tiles);
}
template <typename T, int D>
void launch_bwd_norm(const Params& p, int norm, bool half, int tiles, dim3 grid, cudaStream_t st) {
  if (norm == AVQ_NORM_RMS) return launch_bwd<T, D, AVQ_NORM_RMS>(p, half, tiles, grid, st);
  return launch_bwd<T, D, AVQ_NORM_LAYER>(p, half, tiles, grid, st);
}

int backward_blocks(const avq_qk_dims& s) {
  const int tokens = s.B * s.N;
  const int tb = tile_tokens(s.d, tokens);
  const int tiles = (tokens + tb - 1) / tb;
  const int most = 2 * num_sms();  // for each of queries and keys: four blocks per SM in all
  return tiles < most ? tiles : most;
}

}  // namespace

cudaError_t launch_qk_norm(const avq_qk_dims& s, avq_dtype dt, const void* const* x, const Strides* xs,
                           const void* const* w, const void* const* b, const int32_t* pos, const double* freqs,
                           bool inverse, void* const* y, cudaStream_t st, LaunchLog& log) {
  Params p = params_of(s, xs, pos, freqs);
  for (int i = 0; i < 2; ++i) p.x[i] = x[i], p.w[i] = w[i], p.b[i] = b[i], p.y[i] = y[i];
  if (inverse) p.sign = -1.f;
  const int tiles = (p.tokens + p.tb - 1) / p.tb;
  const bool half = s.layout == AVQ_ROTARY_HALF;
  if (dt == AVQ_F32) {
    if (s.d == 64) launch_fwd_norm<float, 64>(p, s.norm, half, tiles, st);
    else launch_fwd_norm<float, 128>(p, s.norm, half, tiles, st);
  } else {
    if (s.d == 64) launch_fwd_norm<bf16, 64>(p, s.norm, half, tiles, st);
    else launch_fwd_norm<bf16, 128>(p, s.norm, half, tiles, st);
  }
  log.add(s.norm == AVQ_NORM_NONE ? "rotary" : "qk_norm");
  return cudaGetLastError();
}

size_t qk_norm_backward_workspace(const avq_qk_dims& s) {
  return (size_t)2 * backward_blocks(s) * 2 * s.d * sizeof(float);
}

cudaError_t launch_qk_norm_backward(const avq_qk_dims& s, avq_dtype dt, const void* const* g, const Strides* gs,
                                    const void* const* x, const Strides* xs, const void* const* w,
                                    const int32_t* pos, const double* freqs, void* const* dx, float* const* dw,
                                    float* const* db, void* ws, cudaStream_t st, LaunchLog& log) {
  Params p = params_of(s, xs, pos, freqs);
  for (int i = 0; i < 2; ++i) p.x[i] = x[i], p.w[i] = w[i], p.g[i] = g[i], p.gs[i] = gs[i], p.y[i] = dx[i];
  p.sign = -1.f;
  p.part = static_cast<float*>(ws);
  const int tiles = (p.tokens + p.tb - 1) / p.tb;
  const bool half = s.layout == AVQ_ROTARY_HALF;
  const int blocks = backward_blocks(s);
  const dim3 grid(blocks, s.Hk > 0 ? 2 : 1);
  if (dt == AVQ_F32) {
    if (s.d == 64) launch_bwd_norm<float, 64>(p, s.norm, half, tiles, grid, st);
    else launch_bwd_norm<float, 128>(p, s.norm, half, tiles, grid, st);
  } else {
    if (s.d == 64) launch_bwd_norm<bf16, 64>(p, s.norm, half, tiles, grid, st);
    else launch_bwd_norm<bf16, 128>(p, s.norm, half, tiles, grid, st);
  }
  log.add("qk_norm_backward");
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  bool any = false;
  for (int i = 0; i < 2; ++i) any = any || dw[i] != nullptr || db[i] != nullptr;
  if (!any) return cudaSuccess;
  const int outs = s.Hk > 0 ? 4 : 2;
  if (s.d == 64)
    e = launch_after(weight_sum_kernel<64>, dim3(outs), dim3(1024), 0, st, (const float*)p.part, blocks, dw[0],
                     db[0], dw[1], db[1]);
  else
    e = launch_after(weight_sum_kernel<128>, dim3(outs), dim3(1024), 0, st, (const float*)p.part, blocks, dw[0],
                     db[0], dw[1], db[1]);
  log.add("weight_sum");
  return e;
}

}  // namespace avq
