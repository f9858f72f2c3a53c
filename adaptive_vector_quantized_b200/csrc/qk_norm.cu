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
// Angles are formed in 64-bit fixed point: a frequency as a fraction of a turn
// in units of 2^-64, times the position as integers, where whole turns drop
// off by themselves; only the remaining fraction becomes fp32.  That is off by at
// most 2^-26 of a turn, and the frequency's product with 1 / (2 pi), in fp64, by
// 2^-52 of the whole angle.  (At position 10^6 a 32-bit product would be off by
// 0.06.)
//
// The kernels are bound by memory: each element is read once and written
// once.  A head is spread over d / 8 lanes of 8 elements, as two groups of 4
// that hold both elements of every pair in either layout, so the rotation
// needs no exchange between lanes and the norm 3 or 4 butterfly shuffles.
// A lane works out the sine and cosine of its own four pairs once per token and
// keeps them over the token's heads: no table, no barrier.
#include "common.cuh"
#include "fastmath.cuh"
#include "internal.h"
#include "tc_util.cuh"

namespace avq {

namespace {

constexpr int kThreads = 256;
// Heads of a token that a lane group has under way at a time: 64 bytes of each
// lane's loads, in each of two batches.  They are copied asynchronously into
// places of shared memory that belong to one thread each, so that they take no
// registers and need no barrier.  Measured for RMS norm with rotation of 65536
// tokens of 32 heads of 64 (537 MB): 107 us with the batches in registers, where
// the loads' latency bound it, 88 us like this (6.1 TB/s).
template <typename T>
constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
constexpr int kStages = 2;

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

__device__ __forceinline__ void store4(float* p, const float2* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
__device__ __forceinline__ void store4(bf16* p, const float2* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
}

// A lane's 8 elements of a head as they stand in memory, each group of 4 by itself.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  typedef float4 Four;
  static __device__ __forceinline__ void get(float4 a, float4 b, float2* v) {
    v[0] = fm::f2(a.x, a.y), v[1] = fm::f2(a.z, a.w), v[2] = fm::f2(b.x, b.y), v[3] = fm::f2(b.z, b.w);
  }
};
template <>
struct Raw<bf16> {
  typedef uint2 Four;
  static __device__ __forceinline__ void get(uint2 a, uint2 b, float2* v) {
    v[0] = fm::f2(bf16_lo(a.x), bf16_hi(a.x)), v[1] = fm::f2(bf16_lo(a.y), bf16_hi(a.y));
    v[2] = fm::f2(bf16_lo(b.x), bf16_hi(b.x)), v[3] = fm::f2(bf16_lo(b.y), bf16_hi(b.y));
  }
};
// This thread's places for heads under way: [place][group][thread].
template <typename T>
struct Places {
  typedef typename Raw<T>::Four Four;
  Four* s;  // the thread's first
  uint32_t addr;
  __device__ __forceinline__ explicit Places(Four* ring) : s(ring + threadIdx.x), addr(tc::smem_u32(s)) {}
  // x: the lane's first group, the second `apart` elements on
  __device__ __forceinline__ void request(int k, const T* x, int apart) const {
    copy(addr + (2 * k) * kThreads * (int)sizeof(Four), x);
    copy(addr + (2 * k + 1) * kThreads * (int)sizeof(Four), x + apart);
  }
  __device__ __forceinline__ void get(int k, float2* v) const {
    Raw<T>::get(s[(2 * k) * kThreads], s[(2 * k + 1) * kThreads], v);
  }
  static __device__ __forceinline__ void copy(uint32_t dst, const T* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"((int)sizeof(Four)) : "memory");
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
__device__ __forceinline__ void get8(const float* s, int ia, int ib, float2* v) {
  const float4 a = *reinterpret_cast<const float4*>(s + ia), b = *reinterpret_cast<const float4*>(s + ib);
  v[0] = fm::f2(a.x, a.y), v[1] = fm::f2(a.z, a.w), v[2] = fm::f2(b.x, b.y), v[3] = fm::f2(b.z, b.w);
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// A lane's four rotations.  In the half layout pairs are neighbours in each of the
// two groups: two at a time, c = (c0, c1).  Interleaved, an element's partner is its
// neighbour: one at a time, since (c, c) and (-s, s) would take twice the registers
// and the swap two moves.
template <bool kHalf>
struct Turn {
  float2 c[2], s[2];
  // of the angles with cosines x and sines y
  __device__ __forceinline__ void set(const float* x, const float* y) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = fm::f2(x[2 * i], x[2 * i + 1]);
      s[i] = fm::f2(y[2 * i], y[2 * i + 1]);
    }
  }
  // v: the lane's elements two by two, group a then group b
  __device__ __forceinline__ void apply(float2* v) const {
    if constexpr (kHalf) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = v[i], b = v[2 + i];
        const float2 bs = fm::mul2(b, s[i]);
        v[i] = fm::fma2(a, c[i], fm::f2(-bs.x, -bs.y));
        v[2 + i] = fm::fma2(b, c[i], fm::mul2(a, s[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ci = i & 1 ? c[i >> 1].y : c[i >> 1].x, si = i & 1 ? s[i >> 1].y : s[i >> 1].x;
        const float2 x = v[i];
        v[i] = fm::f2(fmaf(x.x, ci, -(x.y * si)), fmaf(x.y, ci, x.x * si));
      }
    }
  }
};

// Angles of the lane's four pairs.
struct Angles {
  unsigned long long freq[4];  // turns per position, in units of 2^-64
  int axis;
  __device__ __forceinline__ void init(const Params& p, int lane) {
    const int half = p.rot >> 1;
    axis = p.axes == 2 && 4 * lane >= half >> 1 ? 1 : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double turns = __ldg(p.freqs + 4 * lane + e) * 0.15915494309189533577;  // / 2 pi
      freq[e] = (unsigned long long)__double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
    }
  }
  // the position of token `tok` along the lane's axis
  __device__ __forceinline__ int position(const Params& p, int tok, int n) const {
    if (p.pos == nullptr) return n;
    return __ldg(p.pos + (long long)(p.pos_batch ? tok : n) * p.axes + axis);
  }
  template <typename T, bool kHalf>
  __device__ __forceinline__ void turn(const Params& p, int at, Turn<kHalf>* out) const {
    float c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned long long turns = (unsigned long long)(long long)at * freq[e];  // modulo one turn
      const float part = (float)(int)(turns >> 32);                                  // in units of 2^-32
      // CUDA bounds the fast forms by 2^-21.19 in [-pi, pi]; with the argument's
      // rounding 2^-20.7 in all, a 6000th of a bf16 rounding
      if constexpr (sizeof(T) == 2)
        __sincosf(part * 1.46291807926715968e-9f, &s[e], &c[e]);  // 2 pi 2^-32
      else
        sincospif(part * 4.656612873077392578125e-10f, &s[e], &c[e]);  // 2^-31
      c[e] *= p.mscale;
      s[e] *= p.mscale * p.sign;
    }
    out->set(c, s);
  }
};

__device__ __forceinline__ float2 both(float x) { return fm::f2(x, x); }

// v <- u, returns 1 / sqrt(...)
template <int D, int kNorm>
__device__ __forceinline__ float normalise(float2* v, float eps) {
  constexpr int L = D / 8;
  if constexpr (kNorm == AVQ_NORM_LAYER) {
    const float2 s = fm::add2(fm::add2(v[0], v[1]), fm::add2(v[2], v[3]));
    const float mean = group_sum<L>(s.x + s.y) * (1.f / D);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fm::add2(v[i], both(-mean));
  }
  float2 q = fm::mul2(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) q = fm::fma2(v[i], v[i], q);
  const float r = rsqrtf(group_sum<L>(q.x + q.y) * (1.f / D) + eps);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fm::mul2(v[i], both(r));
  return r;
}

template <typename T, int D, int kNorm, bool kHalf>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_kernel(const Params p) {
  constexpr int L = D / 8, G = kThreads / L, U = kBatch<T>;
  __shared__ __align__(16) typename Raw<T>::Four ring[kStages * U * 2 * kThreads];
  __shared__ __align__(16) float sw[kNorm == AVQ_NORM_NONE ? 4 : 2 * D], sb[kNorm == AVQ_NORM_NONE ? 4 : 2 * D];
  const int first = blockIdx.x * p.tb;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int t = group & (p.tb - 1), slot = group / p.tb, slots = G / p.tb;
  const int tok = first + t;
  const bool in = tok < p.tokens;  // whole groups: the shuffles still run
  const int b = in ? tok / p.N : 0, n = in ? tok - b * p.N : 0;
  int ia, ib;
  const bool turned = places<kHalf>(lane, p.rot, ia, ib);
  // batches of U heads: the queries' first, then the keys' (the same number for every group)
  const int per = slots * U;
  const int qb = (p.H[0] + per - 1) / per, all = qb + (p.H[1] + per - 1) / per;
  const Places<T> places(ring);
  const int apart = ib - ia;
  auto request = [&](int i) {
    const int which = i >= qb, h0 = (which ? i - qb : i) * per + slot;
    const int64_t sh = slots * p.xs[which].h;
    const T* x = static_cast<const T*>(p.x[which]) + b * p.xs[which].b + n * p.xs[which].n + h0 * p.xs[which].h + ia;
    const int left = in && i < all ? p.H[which] - h0 : 0;
#pragma unroll
    for (int k = 0; k < U; ++k, x += sh)
      if (k * slots < left) places.request((i & 1) * U + k, x, apart);
    tc::cp_async_commit();
  };
  grid_dependency_wait();
  request(0);  // under way while the angles are made
  request(1);
  if constexpr (kNorm != AVQ_NORM_NONE) fill_weights<T, D>(p, sw, sb);
  Turn<kHalf> rotation;
  if (turned) {
    Angles angles;
    angles.init(p, lane);
    angles.turn<T>(p, angles.position(p, in ? tok : 0, n), &rotation);
  }
  if constexpr (kNorm != AVQ_NORM_NONE) __syncthreads();
  const long long step = (long long)slots * p.N * D;
  for (int i = 0; i < all; ++i) {
    tc::cp_async_wait<1>();
    const int which = i >= qb, h0 = (which ? i - qb : i) * per + slot;
    const int H = p.H[which], left = in ? H - h0 : 0;
    T* y = static_cast<T*>(p.y[which]) + (((long long)b * H + h0) * p.N + n) * D + ia;
    float2 w[4], bias[4];
    if constexpr (kNorm != AVQ_NORM_NONE) {
      get8(sw + which * D, ia, ib, w);
      get8(sb + which * D, ia, ib, bias);
    }
    float2 v[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      places.get((i & 1) * U + k, v[k]);  // of an absent head: anything, never stored
      if constexpr (kNorm != AVQ_NORM_NONE) {
        normalise<D, kNorm>(v[k], p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = fm::fma2(v[k][e], w[e], bias[e]);
      }
    }
    if (turned) {
#pragma unroll
      for (int k = 0; k < U; ++k) rotation.apply(v[k]);
    }
    if ((U - 1) * slots < left) {
#pragma unroll
      for (int k = 0; k < U; ++k, y += step) {
        store4(y, v[k]);
        store4(y + apart, v[k] + 2);
      }
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k, y += step)
        if (k * slots < left) {
          store4(y, v[k]);
          store4(y + apart, v[k] + 2);
        }
    }
    request(i + 2);
  }
}

// Gradients.  blockIdx.y: queries or keys; each block walks tiles and keeps
// its share of the weight gradients in registers, summed over its groups at
// the end in a fixed order.
template <typename T, int D, int kNorm, bool kHalf, bool kBias>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_backward_kernel(const Params p, int tiles) {
  constexpr int L = D / 8, G = kThreads / L, U = kBatch<T> / 2;
  __shared__ __align__(16) typename Raw<T>::Four ring[kStages * U * 4 * kThreads];
  float* sums = reinterpret_cast<float*>(ring);  // [G][D], at the end
  grid_dependency_wait();
  allow_dependents();
  const int which = blockIdx.y;
  const int H = p.H[which];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int t = group & (p.tb - 1), slot = group / p.tb, slots = G / p.tb;
  int ia, ib;
  const bool turned = places<kHalf>(lane, p.rot, ia, ib);
  const Strides xs = p.xs[which], gs = p.gs[which];
  float2 w[4], dw[4], db[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = both(1.f), dw[i] = db[i] = both(0.f);
  if (p.w[which] != nullptr) {
    const T* pw = static_cast<const T*>(p.w[which]);
    typedef typename Raw<T>::Four Four;
    Raw<T>::get(*reinterpret_cast<const Four*>(pw + ia), *reinterpret_cast<const Four*>(pw + ib), w);
  }
  // batches of U heads of a tile's tokens, tile after tile
  const int per = slots * U, batches = (H + per - 1) / per;
  const int apart = ib - ia;
  const int64_t x_step = slots * xs.h, g_step = slots * gs.h;
  const long long y_step = (long long)slots * p.N * D;
  const Places<T> places(ring);
  Angles angles;
  if (turned) angles.init(p, lane);
  // a batch: where the group's token stands at the group's first head of it
  struct At {
    const T *x, *g;
    T* y;
    int left;  // heads from there on, 0 for a token past the end
    int tile, i, pos;
  };
  auto first_of = [&](int tile) {
    const int tok = tile * p.tb + t;
    const bool in = tile < tiles && tok < p.tokens;
    const int b = in ? tok / p.N : 0, n = in ? tok - b * p.N : 0;
    At at;
    at.x = static_cast<const T*>(p.x[which]) + b * xs.b + n * xs.n + slot * xs.h + ia;
    at.g = static_cast<const T*>(p.g[which]) + b * gs.b + n * gs.n + slot * gs.h + ia;
    at.y = static_cast<T*>(p.y[which]) + (((long long)b * H + slot) * p.N + n) * D + ia;
    at.left = in ? H - slot : 0;
    at.tile = tile;
    at.i = 0;
    at.pos = turned ? angles.position(p, in ? tok : 0, n) : 0;
    return at;
  };
  auto advance = [&](At& at) {
    if (++at.i == batches) {
      at = first_of(at.tile + gridDim.x);
    } else {
      at.x += U * x_step;
      at.g += U * g_step;
      at.y += U * y_step;
      at.left -= U * slots;
    }
  };
  auto request = [&](const At& at, int stage) {
    const T *px = at.x, *pg = at.g;
#pragma unroll
    for (int k = 0; k < U; ++k, px += x_step, pg += g_step) {
      if (k * slots >= at.left) continue;
      places.request((stage * U + k) * 2, px, apart);
      places.request((stage * U + k) * 2 + 1, pg, apart);
    }
    tc::cp_async_commit();
  };
  Turn<kHalf> rotation;
  auto finish = [&](T* y, int left, int stage) {
    float2 u[U][4], z[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      places.get((stage * U + k) * 2, u[k]);
      places.get((stage * U + k) * 2 + 1, z[k]);
    }
    const bool whole = (U - 1) * slots < left;
    if (!whole) {  // an absent row is 0 throughout
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k * slots >= left) {
#pragma unroll
          for (int e = 0; e < 4; ++e) u[k][e] = z[k][e] = both(0.f);
        }
    }
    if (turned) {
#pragma unroll
      for (int k = 0; k < U; ++k) rotation.apply(z[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float r = normalise<D, kNorm>(u[k], whole || k * slots < left ? p.eps : 1.f);
      float2 gu = both(0.f), gm = both(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dw[e] = fm::fma2(z[k][e], u[k][e], dw[e]);
        if constexpr (kBias) db[e] = fm::add2(db[e], z[k][e]);
        z[k][e] = fm::mul2(z[k][e], w[e]);
        gu = fm::fma2(z[k][e], u[k][e], gu);
        if constexpr (kNorm == AVQ_NORM_LAYER) gm = fm::add2(gm, z[k][e]);
      }
      const float mu = group_sum<L>(gu.x + gu.y) * (-1.f / D);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[k][e] = fm::fma2(u[k][e], both(mu), z[k][e]);
      if constexpr (kNorm == AVQ_NORM_LAYER) {
        const float mean = group_sum<L>(gm.x + gm.y) * (-1.f / D);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[k][e] = fm::add2(z[k][e], both(mean));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) z[k][e] = fm::mul2(z[k][e], both(r));
    }
    if (whole) {
#pragma unroll
      for (int k = 0; k < U; ++k, y += y_step) {
        store4(y, z[k]);
        store4(y + apart, z[k] + 2);
      }
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k, y += y_step)
        if (k * slots < left) {
          store4(y, z[k]);
          store4(y + apart, z[k] + 2);
        }
    }
  };
  // the batch that is worked on is two behind the one that is requested
  At ahead = first_of(blockIdx.x);
  T* y[2];
  int left[2], pos[2], state[2];  // state: 0 further batch of a tile, 1 its first, 2 past the end
  auto ask = [&](int stage) {
    request(ahead, stage);
    y[stage] = ahead.y;
    left[stage] = ahead.left;
    pos[stage] = ahead.pos;
    state[stage] = ahead.tile >= tiles ? 2 : ahead.i == 0;
    advance(ahead);
  };
  auto turn_of = [&](int stage) {
    if (state[stage] == 1 && turned) angles.turn<T>(p, pos[stage], &rotation);
    tc::cp_async_wait<1>();
    finish(y[stage], left[stage], stage);
    ask(stage);
  };
  ask(0);
  ask(1);
  while (state[0] < 2) {
    turn_of(0);
    if (state[1] == 2) break;
    turn_of(1);
  }
  tc::cp_async_wait<0>();
  for (int kind = 0; kind < (kBias ? 2 : 1); ++kind) {
    __syncthreads();
    store4(sums + group * D + ia, kind == 0 ? dw : db);
    store4(sums + group * D + ib, kind == 0 ? dw + 2 : db + 2);
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
      for (int k = 0; k < G; ++k) s += sums[k * D + threadIdx.x];
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

// Tokens per tile (forward): as many as fit the block's lane groups (sine and
// cosine are then shared by the token's heads alone), fewer while the tiles would
// leave SMs idle; the freed groups share the token's heads.  12 heads of 64: 784
// tokens 5.6 us, 8.0 with whole tiles, 6.9 with two tiles an SM; 2048 tokens 6.1,
// 8.1, 9.2.  The gradients take whole tiles: 300 tokens of 8 heads of 128 8.2 us,
// 8.9 with a tile an SM, 1568 tokens 11.3 and 12.2 (each block adds its own sums).
int tile_tokens(int d, int tokens) {
  int tb = groups_of(d);
  while (tb > 1 && (tokens + tb - 1) / tb < num_sms()) tb >>= 1;
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
cudaError_t launch_fwd(const Params& p, bool half, int tiles, cudaStream_t st) {
  return launch_after(half ? qk_norm_kernel<T, D, kNorm, true> : qk_norm_kernel<T, D, kNorm, false>, dim3(tiles),
                      dim3(kThreads), 0, st, p);
}
template <typename T, int D>
cudaError_t launch_fwd_norm(const Params& p, int norm, bool half, int tiles, cudaStream_t st) {
  if (norm == AVQ_NORM_NONE) return launch_fwd<T, D, AVQ_NORM_NONE>(p, half, tiles, st);
  if (norm == AVQ_NORM_RMS) return launch_fwd<T, D, AVQ_NORM_RMS>(p, half, tiles, st);
  return launch_fwd<T, D, AVQ_NORM_LAYER>(p, half, tiles, st);
}
template <typename T, int D, int kNorm, bool kBias>
cudaError_t launch_bwd(const Params& p, bool half, int tiles, dim3 grid, cudaStream_t st) {
  return launch_after(half ? qk_norm_backward_kernel<T, D, kNorm, true, kBias>
                           : qk_norm_backward_kernel<T, D, kNorm, false, kBias>,
                      grid, dim3(kThreads), 0, st, p, tiles);
}
// bias: whether a bias gradient is asked for
template <typename T, int D>
cudaError_t launch_bwd_norm(const Params& p, int norm, bool bias, bool half, int tiles, dim3 grid, cudaStream_t st) {
  if (norm == AVQ_NORM_RMS)
    return bias ? launch_bwd<T, D, AVQ_NORM_RMS, true>(p, half, tiles, grid, st)
                : launch_bwd<T, D, AVQ_NORM_RMS, false>(p, half, tiles, grid, st);
  return bias ? launch_bwd<T, D, AVQ_NORM_LAYER, true>(p, half, tiles, grid, st)
              : launch_bwd<T, D, AVQ_NORM_LAYER, false>(p, half, tiles, grid, st);
}

int backward_blocks(const avq_qk_dims& s) {
  const int tokens = s.B * s.N;
  const int tb = groups_of(s.d);
  const int tiles = (tokens + tb - 1) / tb;
  const int most = s.Hk > 0 ? num_sms() : 2 * num_sms();  // the two blocks that an SM holds
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
  cudaError_t e;
  if (dt == AVQ_F32) {
    e = s.d == 64 ? launch_fwd_norm<float, 64>(p, s.norm, half, tiles, st)
                  : launch_fwd_norm<float, 128>(p, s.norm, half, tiles, st);
  } else {
    e = s.d == 64 ? launch_fwd_norm<bf16, 64>(p, s.norm, half, tiles, st)
                  : launch_fwd_norm<bf16, 128>(p, s.norm, half, tiles, st);
  }
  log.add(s.norm == AVQ_NORM_NONE ? "rotary" : "qk_norm");
  return e;
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
  p.tb = groups_of(s.d);
  p.part = static_cast<float*>(ws);
  const int tiles = (p.tokens + p.tb - 1) / p.tb;
  const bool half = s.layout == AVQ_ROTARY_HALF;
  const int blocks = backward_blocks(s);
  const bool bias = db[0] != nullptr || db[1] != nullptr;
  const dim3 grid(blocks, s.Hk > 0 ? 2 : 1);
  cudaError_t e;
  if (dt == AVQ_F32) {
    e = s.d == 64 ? launch_bwd_norm<float, 64>(p, s.norm, bias, half, tiles, grid, st)
                  : launch_bwd_norm<float, 128>(p, s.norm, bias, half, tiles, grid, st);
  } else {
    e = s.d == 64 ? launch_bwd_norm<bf16, 64>(p, s.norm, bias, half, tiles, grid, st)
                  : launch_bwd_norm<bf16, 128>(p, s.norm, bias, half, tiles, grid, st);
  }
  log.add("qk_norm_backward");
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
