// C ABI of the exact operators beside the quantised path (norms and rotation
// of queries and keys, attention over another sequence): host-side validation
// and dispatch.  Every check runs on the host before anything is enqueued.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace avq {

namespace {

constexpr long long kMaxRows = 1ll << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t elem(avq_dtype dt) { return dt == AVQ_F32 ? 4 : 2; }
bool known(avq_dtype dt) { return dt == AVQ_F32 || dt == AVQ_BF16; }

avq_status need_ptr(const void* p, const char* name) {
  if (p == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return api_fail(AVQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return AVQ_OK;
}

// What a view is for: its tokens may repeat (stride 0), it is read by tensor
// copies (which cannot repeat rows), or it is written.
enum Use { kRead, kCopied, kWritten };

// Strides of a [B,H,N,d] view, those of dimensions of size 1 set to 0; the
// tensor's extent in bytes in *span.
avq_status view(const avq_strides* s, int B, int H, int N, int d, avq_dtype dt, Use use, const char* name,
                Strides* out, size_t* span) {
  if (s == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "%s: strides are NULL", name);
  const int64_t v[3] = {B > 1 ? s->b : 0, H > 1 ? s->h : 0, N > 1 ? s->n : 0};
  const int n[3] = {B, H, N};
  const int64_t es = (int64_t)elem(dt);
  int64_t last = d;
  for (int i = 0; i < 3; ++i) {
    if (v[i] < 0 || v[i] >= (int64_t)1 << 38)  // bytes below 2^40, a tensor map's limit
      return api_fail(AVQ_ERR_INVALID_ARG, "%s: strides must be in [0, 2^38)", name);
    if (v[i] * es % 16 != 0)
      return api_fail(AVQ_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", name);
    if (use == kCopied && i == 2 && N > 1 && v[i] == 0)
      return api_fail(AVQ_ERR_INVALID_ARG, "%s: tokens must not repeat (stride 0)", name);
    last += v[i] * (int64_t)(n[i] > 0 ? n[i] - 1 : 0);
  }
  // of what is written, each dimension steps over what those with shorter strides span
  for (int i = 0; i < 3 && use == kWritten; ++i) {
    int64_t inner = d;
    for (int j = 0; j < 3; ++j)
      if (j != i && n[j] > 1 && (v[j] < v[i] || (v[j] == v[i] && j < i))) inner += v[j] * (int64_t)(n[j] - 1);
    if (n[i] > 1 && v[i] < inner)
      return api_fail(AVQ_ERR_INVALID_ARG, "%s: an output's rows must not overlap", name);
  }
  *out = Strides{v[0], v[1], v[2]};
  if (span != nullptr) *span = (size_t)(last * es);
  return AVQ_OK;
}

// Memory that a call reads or writes; of 0 bytes where it does not.
struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};
// Every output apart from every input and every other output.
template <size_t kOuts, size_t kIns>
avq_status apart(const Range (&outs)[kOuts], const Range (&ins)[kIns]) {
  auto meet = [](const Range& x, const Range& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return x.p != nullptr && y.p != nullptr && x.bytes > 0 && y.bytes > 0 && a < b + y.bytes && b < a + x.bytes;
  };
  for (size_t o = 0; o < kOuts; ++o) {
    for (const Range& in : ins)
      if (meet(outs[o], in)) return api_fail(AVQ_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, in.name);
    for (size_t i = 0; i < o; ++i)
      if (meet(outs[o], outs[i])) return api_fail(AVQ_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, outs[i].name);
  }
  return AVQ_OK;
}

avq_status check_ws(size_t need, const void* ws, size_t bytes) {
  if (need == 0) return AVQ_OK;
  if (ws == nullptr || bytes < need)
    return api_fail(AVQ_ERR_WORKSPACE, "workspace of %zu bytes required (got %zu at %p)", need, bytes, ws);
  if (!aligned(ws, 256)) return api_fail(AVQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return AVQ_OK;
}

#define AVQ_TRY(call)                       \
  do {                                      \
    const avq_status try_st = (call);       \
    if (try_st != AVQ_OK) return try_st;    \
  } while (0)

// ---- norms and rotation ------------------------------------------------------

avq_status check_qk(const avq_qk_dims* s, avq_dtype dt) {
  if (s == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "dims is NULL");
  if (!known(dt)) return api_fail(AVQ_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (s->B < 1 || s->N < 1 || s->Hq < 1 || s->Hk < 0)
    return api_fail(AVQ_ERR_INVALID_ARG, "B, N and Hq must be >= 1 and Hk >= 0 (got %d, %d, %d, %d)", s->B, s->N,
                    s->Hq, s->Hk);
  if (s->d != 64 && s->d != 128) return api_fail(AVQ_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", s->d);
  const long long tokens = (long long)s->B * s->N;
  if (tokens >= kMaxRows || tokens * s->Hq >= kMaxRows || tokens * s->Hk >= kMaxRows)
    return api_fail(AVQ_ERR_UNSUPPORTED, "B*H*N must be below 2^30");
  if (s->axes != 1 && s->axes != 2) return api_fail(AVQ_ERR_INVALID_ARG, "axes must be 1 or 2 (got %d)", s->axes);
  if (s->rot < 0 || s->rot > s->d || s->rot % (8 * s->axes) != 0)
    return api_fail(AVQ_ERR_INVALID_ARG, "rot must be a multiple of %d in [0, d] (got %d)", 8 * s->axes, s->rot);
  if (s->layout != AVQ_ROTARY_HALF && s->layout != AVQ_ROTARY_INTERLEAVED)
    return api_fail(AVQ_ERR_INVALID_ARG, "unknown rotary layout %d", s->layout);
  if (s->norm < AVQ_NORM_NONE || s->norm > AVQ_NORM_LAYER)
    return api_fail(AVQ_ERR_INVALID_ARG, "unknown norm %d", s->norm);
  if (!(s->eps >= 0.f) || !isfinite(s->eps)) return api_fail(AVQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!isfinite(s->mscale)) return api_fail(AVQ_ERR_INVALID_ARG, "mscale must be finite");
  return AVQ_OK;
}

avq_status check_turn(const avq_qk_dims& s, const int32_t* positions, const double* freqs) {
  if (s.rot == 0) return AVQ_OK;
  if (!aligned(positions, 4)) return api_fail(AVQ_ERR_INVALID_ARG, "positions is not 4-byte aligned");
  if (freqs == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "freqs is NULL");
  if (!aligned(freqs, 8)) return api_fail(AVQ_ERR_INVALID_ARG, "freqs is not 8-byte aligned");
  return AVQ_OK;
}

avq_status optional_vector(const void* p, const char* name) {
  return p == nullptr ? AVQ_OK : need_ptr(p, name);
}

struct Pair {
  const void* x[2];
  Strides s[2];
  size_t span[2];
};
avq_status pair_of(const avq_qk_dims& s, avq_dtype dt, const void* q, const avq_strides* qs, const char* qn,
                   const void* k, const avq_strides* ks, const char* kn, Pair* out) {
  *out = Pair{};
  AVQ_TRY(need_ptr(q, qn));
  AVQ_TRY(view(qs, s.B, s.Hq, s.N, s.d, dt, kRead, qn, &out->s[0], &out->span[0]));
  out->x[0] = q;
  if (s.Hk > 0) {
    AVQ_TRY(need_ptr(k, kn));
    AVQ_TRY(view(ks, s.B, s.Hk, s.N, s.d, dt, kRead, kn, &out->s[1], &out->span[1]));
    out->x[1] = k;
  }
  return AVQ_OK;
}
avq_status outputs_of(const avq_qk_dims& s, void* q, const char* qn, void* k, const char* kn, void** out) {
  AVQ_TRY(need_ptr(q, qn));
  out[0] = q;
  out[1] = nullptr;
  if (s.Hk > 0) {
    AVQ_TRY(need_ptr(k, kn));
    out[1] = k;
  }
  return AVQ_OK;
}
// The memory of dense outputs, of a vector [d], of positions and frequencies.
Range dense_of(const avq_qk_dims& s, avq_dtype dt, const void* p, int H, const char* name) {
  return Range{p, (size_t)s.B * H * s.N * s.d * elem(dt), name};
}
Range vector_of(const avq_qk_dims& s, size_t size, const void* p, const char* name) {
  return Range{p, (size_t)s.d * size, name};
}
Range positions_of(const avq_qk_dims& s, const int32_t* p) {
  return Range{p, s.rot > 0 ? (size_t)(s.pos_batch ? s.B : 1) * s.N * s.axes * sizeof(int32_t) : 0, "positions"};
}
Range freqs_of(const avq_qk_dims& s, const double* p) { return Range{p, (size_t)s.rot / 2 * sizeof(double), "freqs"}; }

// ---- attention over another sequence -------------------------------------------

avq_status check_cross(const avq_cross_dims* s, avq_dtype dt) {
  if (s == nullptr) return api_fail(AVQ_ERR_INVALID_ARG, "dims is NULL");
  if (!known(dt)) return api_fail(AVQ_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (s->B < 1 || s->Bk < 1 || s->Hq < 1 || s->Hk < 1 || s->Nq < 1 || s->Nk < 0)
    return api_fail(AVQ_ERR_INVALID_ARG, "B, Bk, Hq, Hk and Nq must be >= 1 and Nk >= 0");
  if (s->B % s->Bk != 0) return api_fail(AVQ_ERR_INVALID_ARG, "B must be a multiple of Bk (got %d, %d)", s->B, s->Bk);
  if (s->Hq % s->Hk != 0)
    return api_fail(AVQ_ERR_INVALID_ARG, "Hq must be a multiple of Hk (got %d, %d)", s->Hq, s->Hk);
  if (s->d != 64 && s->d != 128) return api_fail(AVQ_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", s->d);
  const long long qh = (long long)s->B * s->Hq, kh = (long long)s->Bk * s->Hk;
  if (qh >= kMaxRows || qh * s->Nq >= kMaxRows || kh >= kMaxRows || kh * s->Nk >= kMaxRows)
    return api_fail(AVQ_ERR_UNSUPPORTED, "B*Hq*Nq and Bk*Hk*Nk must be below 2^30");
  if (!(s->scale > 0.f) || !isfinite(s->scale)) return api_fail(AVQ_ERR_INVALID_ARG, "scale must be finite and > 0");
  return AVQ_OK;
}

// Ranges of the long axis (`units` tiles of it) when `items` blocks alone
// would leave SMs idle: as many as bring the blocks to `target`, none shorter
// than one tile.
int split_count(long long items, long long units, long long target) {
  long long n = items >= target ? 1 : target / items;
  if (n > units) n = units;
  if (n > 64) n = 64;
  return n < 1 ? 1 : (int)n;
}
long long tiles64(long long n) { return (n + 63) / 64; }

// Parts for the items of the CUDA-core kernels, each a walk over `units` tiles, on
// `slots` resident blocks: as many as make the rounds shortest, where a part costs
// about half a tile more (its own tile's load, its result's way to memory and back).
// 12 heads of 1001 rows over 333 keys of 64 (192 items of up to 6 tiles): 45 us, 55 with
// as many parts as the slots hold at once (41 us now).
int even_split(long long items, long long units, long long slots) {
  int best = 1;
  double least = 0;
  for (int n = 1; n <= 64 && (n == 1 || n <= units); ++n) {
    const double cost = (double)((items * n + slots - 1) / slots) * ((double)((units + n - 1) / n) + 0.5);
    if (n == 1 || cost < least) best = n, least = cost;
  }
  return best;
}

// Rows per key head up to which mma.sync on 16 rows at a time beats the 128-row
// tiles of tcgen05: with 32 sequences of 4096 keys, 8 key heads, 16 rows take 53
// against 93 us at d = 64 and 91 against 99 at d = 128, 32 rows 78 against 93 and
// 125 against 99.
constexpr long long few_rows(int d) { return d == 64 ? 32 : 16; }

// The same for 32-bit inputs, four rows at a time against 64-row tiles: 8 sequences of
// 4096 keys, 8 heads, 8 rows take 46 against 144 us at d = 64 and 63 against 270 at
// d = 128, 24 rows 115 against 145 and 161 against 270, 32 rows 181 and 258.
constexpr long long kFewRowsF32 = 24;

// How the items of a kernel with one block per SM, each a walk over `units` key
// tiles, fill its rounds: the items of full rounds stay whole, those of the last
// round are split where two or more parts of at least four tiles each fit it.
// 64 pairs of row tiles of each of 8 heads of 128 over 16384 keys (3.46 rounds): 990
// us whole, 909 us with the last round split in two (captured, in bursts).  64 parts at
// most, as in split_count: not measured.
struct Rounds {
  int whole = 0, splits = 1;
  long long parts = 0;  // partial results
};
Rounds rounds_of(long long items, long long units, long long sms) {
  Rounds r;
  const long long rest = items % sms;
  long long n = rest > 0 ? sms / rest : 1;
  if (n > units / 4) n = units / 4;
  if (n > 64) n = 64;
  if (n < 2) {
    r.whole = (int)items;
    return r;
  }
  r.whole = (int)(items - rest);
  r.splits = (int)n;
  r.parts = rest * n;
  return r;
}

// How a call is carried out, from its sizes, type and path alone.
struct CrossPlan {
  bool tc = false;   // tensor-core kernels
  bool few = false;  // the one for few rows per key head
  int splits = 1;    // forward, except for tc
  Rounds rounds;     // tc: forward, or dQ
  int dkv_splits = 1, dq_splits = 1;
  size_t part = 0, part_lse = 0, delta = 0, lone = 0;  // bytes, each a multiple of 256
  size_t dq_part = 0;                        // where dQ's begin in part
  size_t total() const { return part + part_lse + delta + lone; }
};

CrossPlan plan_cross(const avq_cross_dims& s, avq_dtype dt, bool backward) {
  CrossPlan p;
  const long long slots = 2ll * num_sms();  // blocks of the CUDA-core kernels
  const long long rows = (long long)s.B * s.Hq * s.Nq, keys = (long long)s.Bk * s.Hk * s.Nk;
  const long long row_items = (long long)s.B * s.Hq * tiles64(s.Nq), key_items = (long long)s.Bk * s.Hk * tiles64(s.Nk);
  const long long shared = (long long)(s.B / s.Bk) * (s.Hq / s.Hk);  // query heads that read one key head
  const long long key_tiles = (s.Nk + 127) / 128;
  p.tc = dt == AVQ_BF16 && api_path() != AVQ_PATH_SIMT && s.Nk > 0;
  if (!backward) {
    p.few = p.tc ? shared * s.Nq <= few_rows(s.d) : dt == AVQ_F32 && shared * s.Nq <= kFewRowsF32;
    if (p.tc && !p.few) {  // pairs of 128-row tiles
      p.rounds = rounds_of((long long)s.B * s.Hq * ((s.Nq + 255) / 256), key_tiles, num_sms());
      p.part = up256((size_t)p.rounds.parts * 256 * s.d * 4);
      p.part_lse = up256((size_t)p.rounds.parts * 256 * 4);
      return p;
    }
    // few: two rounds of the resident blocks, since lengths differ (32 sequences
    // of 4096 to 8191 keys took 68 us with 1 or 2 rounds, 71 with 4, 78 with 8)
    const long long pairs = (long long)s.Bk * s.Hk;
    if (!p.few)
      p.splits = even_split(row_items, tiles64(s.Nk), slots);
    else if (p.tc)
      p.splits = split_count(pairs * ((shared * s.Nq + 15) / 16), s.Nk / 128, 4ll * num_sms());
    else
      p.splits = split_count(pairs * ((shared * s.Nq + 3) / 4), s.Nk / 64, 6ll * num_sms());
    if (p.splits > 1) {
      p.part = up256((size_t)p.splits * rows * s.d * 4);
      p.part_lse = up256((size_t)p.splits * rows * 4);
    }
    return p;
  }
  p.delta = up256((size_t)rows * 4);
  p.lone = up256((size_t)s.Bk * 4);
  // dQ may be formed while dK and dV are: each in a place of its own
  size_t dq;
  if (p.tc) {
    const long long kb = (long long)s.Bk * s.Hk * key_tiles, qb = (long long)s.B * s.Hq * ((s.Nq + 127) / 128);
    const long long sms = num_sms();
    // Where the items of both halves fit the SMs, neither is cut into more than leave
    // the other its place, and they run side by side: 300 rows and keys, 24 heads of
    // 128: 19.5 us, 32.5 with both over all SMs, one after the other; 1024 rows and
    // keys, 8 heads of 64: 23.5 and 33.6.  dK and dV have 4 of the 7 products.
    const bool beside = kb + qb <= sms && !cross_tc_dkv_forms_dq(s.Nk, s.d);
    p.dkv_splits = split_count(kb, shared * ((s.Nq + 127) / 128), beside ? sms * 4 / 7 : sms);
    p.rounds = rounds_of(qb, key_tiles, beside ? sms - kb * p.dkv_splits : sms);
    dq = (size_t)p.rounds.parts * 128 * s.d * 4;
  } else {
    p.dq_splits = even_split(row_items, tiles64(s.Nk), slots);
    dq = p.dq_splits > 1 ? (size_t)p.dq_splits * rows * s.d * 4 : 0;
    if (key_items > 0) p.dkv_splits = even_split(key_items, shared * tiles64(s.Nq), s.d == 64 ? slots : slots / 2);
  }
  const size_t dkv = p.dkv_splits > 1 ? (size_t)p.dkv_splits * 2 * keys * s.d * 4 : 0;
  p.dq_part = up256(dkv);
  p.part = p.dq_part + up256(dq);
  return p;
}

avq_status cross_inputs(const avq_cross_dims& s, avq_dtype dt, const void* Q, const avq_strides* qs, const void* K,
                        const avq_strides* ks, const void* V, const avq_strides* vs, const int32_t* kv_lens,
                        const uint8_t* key_mask, CrossArgs* a, size_t* spans) {
  AVQ_TRY(need_ptr(Q, "Q"));
  AVQ_TRY(view(qs, s.B, s.Hq, s.Nq, s.d, dt, kCopied, "Q", &a->qs, &spans[0]));
  if (s.Nk > 0) {
    AVQ_TRY(need_ptr(K, "K"));
    AVQ_TRY(need_ptr(V, "V"));
    AVQ_TRY(view(ks, s.Bk, s.Hk, s.Nk, s.d, dt, kCopied, "K", &a->ks, &spans[1]));
    AVQ_TRY(view(vs, s.Bk, s.Hk, s.Nk, s.d, dt, kCopied, "V", &a->vs, &spans[2]));
  } else {
    spans[1] = spans[2] = 0;
  }
  if (!aligned(kv_lens, 4)) return api_fail(AVQ_ERR_INVALID_ARG, "kv_lens is not 4-byte aligned");
  a->B = s.B, a->Bk = s.Bk, a->Hq = s.Hq, a->Hk = s.Hk, a->Nq = s.Nq, a->Nk = s.Nk, a->d = s.d;
  a->per_b = s.B / s.Bk, a->per_h = s.Hq / s.Hk;
  a->scale = s.scale;
  a->splits = 1;
  a->Q = Q, a->K = K, a->V = V;
  a->kv_lens = kv_lens, a->key_mask = key_mask;
  return AVQ_OK;
}

Range lens_of(const avq_cross_dims& s, const int32_t* p) { return Range{p, (size_t)s.Bk * sizeof(int32_t), "kv_lens"}; }
Range mask_of(const avq_cross_dims& s, const uint8_t* p) { return Range{p, (size_t)s.Bk * s.Nk, "key_mask"}; }

}  // namespace
}  // namespace avq

using namespace avq;

extern "C" {

avq_status avq_rotary(const avq_qk_dims* dims, avq_dtype dtype, const void* Q, const avq_strides* q_strides,
                      const void* K, const avq_strides* k_strides, const int32_t* positions, const double* freqs,
                      int inverse, void* Yq, void* Yk, avq_stream_t stream) {
  api_begin();
  AVQ_TRY(check_qk(dims, dtype));
  if (dims->norm != AVQ_NORM_NONE) return api_fail(AVQ_ERR_INVALID_ARG, "norm must be AVQ_NORM_NONE");
  AVQ_TRY(check_turn(*dims, positions, freqs));
  Pair in;
  void* out[2];
  AVQ_TRY(pair_of(*dims, dtype, Q, q_strides, "Q", K, k_strides, "K", &in));
  AVQ_TRY(outputs_of(*dims, Yq, "Yq", Yk, "Yk", out));
  AVQ_TRY(apart({dense_of(*dims, dtype, out[0], dims->Hq, "Yq"), dense_of(*dims, dtype, out[1], dims->Hk, "Yk")},
                {{in.x[0], in.span[0], "Q"}, {in.x[1], in.span[1], "K"}, positions_of(*dims, positions),
                 freqs_of(*dims, freqs)}));
  if (api_injected("rotary")) return api_fail(AVQ_ERR_CUDA, "injected failure before launch (avq_rotary)");
  const void* none[2] = {nullptr, nullptr};
  LaunchLog log{};
  const cudaError_t e = launch_qk_norm(*dims, dtype, in.x, in.s, none, none, positions, freqs, inverse != 0, out,
                                       reinterpret_cast<cudaStream_t>(stream), log);
  return api_finish(e, "rotary launch", log);
}

avq_status avq_qk_norm(const avq_qk_dims* dims, avq_dtype dtype, const void* Q, const avq_strides* q_strides,
                       const void* K, const avq_strides* k_strides, const void* wq, const void* wk, const void* bq,
                       const void* bk, const int32_t* positions, const double* freqs, void* Yq, void* Yk,
                       avq_stream_t stream) {
  api_begin();
  AVQ_TRY(check_qk(dims, dtype));
  if (dims->norm == AVQ_NORM_NONE) return api_fail(AVQ_ERR_INVALID_ARG, "norm must be RMS or LAYER");
  AVQ_TRY(check_turn(*dims, positions, freqs));
  Pair in;
  void* out[2];
  AVQ_TRY(pair_of(*dims, dtype, Q, q_strides, "Q", K, k_strides, "K", &in));
  AVQ_TRY(optional_vector(wq, "wq"));
  AVQ_TRY(optional_vector(wk, "wk"));
  AVQ_TRY(optional_vector(bq, "bq"));
  AVQ_TRY(optional_vector(bk, "bk"));
  AVQ_TRY(outputs_of(*dims, Yq, "Yq", Yk, "Yk", out));
  const size_t es = elem(dtype);
  AVQ_TRY(apart({dense_of(*dims, dtype, out[0], dims->Hq, "Yq"), dense_of(*dims, dtype, out[1], dims->Hk, "Yk")},
                {{in.x[0], in.span[0], "Q"}, {in.x[1], in.span[1], "K"}, vector_of(*dims, es, wq, "wq"),
                 vector_of(*dims, es, wk, "wk"), vector_of(*dims, es, bq, "bq"), vector_of(*dims, es, bk, "bk"),
                 positions_of(*dims, positions), freqs_of(*dims, freqs)}));
  if (api_injected("qk_norm")) return api_fail(AVQ_ERR_CUDA, "injected failure before launch (avq_qk_norm)");
  const void* w[2] = {wq, wk};
  const void* b[2] = {bq, bk};
  LaunchLog log{};
  const cudaError_t e = launch_qk_norm(*dims, dtype, in.x, in.s, w, b, positions, freqs, false, out,
                                       reinterpret_cast<cudaStream_t>(stream), log);
  return api_finish(e, "qk_norm launch", log);
}

size_t avq_qk_norm_workspace_size(const avq_qk_dims* dims, avq_dtype dtype) {
  if (dims == nullptr || dims->B < 1 || dims->N < 1 || !known(dtype) || (dims->d != 64 && dims->d != 128)) return 0;
  if ((long long)dims->B * dims->N >= kMaxRows) return 0;
  return up256(qk_norm_backward_workspace(*dims));
}

avq_status avq_qk_norm_backward(const avq_qk_dims* dims, avq_dtype dtype, const void* dYq,
                                const avq_strides* dyq_strides, const void* dYk, const avq_strides* dyk_strides,
                                const void* Q, const avq_strides* q_strides, const void* K,
                                const avq_strides* k_strides, const void* wq, const void* wk,
                                const int32_t* positions, const double* freqs, void* dQ, void* dK, float* dwq,
                                float* dwk, float* dbq, float* dbk, void* ws, size_t ws_bytes,
                                avq_stream_t stream) {
  api_begin();
  AVQ_TRY(check_qk(dims, dtype));
  if (dims->norm == AVQ_NORM_NONE) return api_fail(AVQ_ERR_INVALID_ARG, "norm must be RMS or LAYER");
  AVQ_TRY(check_turn(*dims, positions, freqs));
  Pair in[2];
  void* out[2];
  AVQ_TRY(pair_of(*dims, dtype, dYq, dyq_strides, "dYq", dYk, dyk_strides, "dYk", &in[0]));
  AVQ_TRY(pair_of(*dims, dtype, Q, q_strides, "Q", K, k_strides, "K", &in[1]));
  AVQ_TRY(optional_vector(wq, "wq"));
  AVQ_TRY(optional_vector(wk, "wk"));
  AVQ_TRY(outputs_of(*dims, dQ, "dQ", dK, "dK", out));
  float* dw[2] = {dwq, dims->Hk > 0 ? dwk : nullptr};  // without keys theirs are ignored
  float* db[2] = {dbq, dims->Hk > 0 ? dbk : nullptr};
  AVQ_TRY(optional_vector(dw[0], "dwq"));
  AVQ_TRY(optional_vector(dw[1], "dwk"));
  AVQ_TRY(optional_vector(db[0], "dbq"));
  AVQ_TRY(optional_vector(db[1], "dbk"));
  const size_t es = elem(dtype), need = up256(qk_norm_backward_workspace(*dims));
  AVQ_TRY(check_ws(need, ws, ws_bytes));
  AVQ_TRY(apart({dense_of(*dims, dtype, out[0], dims->Hq, "dQ"), dense_of(*dims, dtype, out[1], dims->Hk, "dK"),
                 vector_of(*dims, 4, dw[0], "dwq"), vector_of(*dims, 4, dw[1], "dwk"),
                 vector_of(*dims, 4, db[0], "dbq"), vector_of(*dims, 4, db[1], "dbk"), {ws, need, "the workspace"}},
                {{in[0].x[0], in[0].span[0], "dYq"}, {in[0].x[1], in[0].span[1], "dYk"},
                 {in[1].x[0], in[1].span[0], "Q"}, {in[1].x[1], in[1].span[1], "K"},
                 vector_of(*dims, es, wq, "wq"), vector_of(*dims, es, wk, "wk"),
                 positions_of(*dims, positions), freqs_of(*dims, freqs)}));
  if (api_injected("qk_norm_backward"))
    return api_fail(AVQ_ERR_CUDA, "injected failure before launch (avq_qk_norm_backward)");
  const void* w[2] = {wq, wk};
  LaunchLog log{};
  const cudaError_t e = launch_qk_norm_backward(*dims, dtype, in[0].x, in[0].s, in[1].x, in[1].s, w, positions, freqs,
                                                out, dw, db, ws, reinterpret_cast<cudaStream_t>(stream), log);
  return api_finish(e, "qk_norm_backward launch", log);
}

size_t avq_cross_workspace_size(const avq_cross_dims* dims, avq_dtype dtype, int backward) {
  api_begin();
  if (check_cross(dims, dtype) != AVQ_OK) return 0;
  return plan_cross(*dims, dtype, backward != 0).total();
}

avq_status avq_cross_attention(const avq_cross_dims* dims, avq_dtype dtype, const void* Q,
                               const avq_strides* q_strides, const void* K, const avq_strides* k_strides,
                               const void* V, const avq_strides* v_strides, const int32_t* kv_lens,
                               const uint8_t* key_mask, void* O, const avq_strides* o_strides, float* lse, void* ws,
                               size_t ws_bytes, avq_stream_t stream) {
  api_begin();
  AVQ_TRY(check_cross(dims, dtype));
  const avq_cross_dims& s = *dims;
  CrossArgs a{};
  size_t spans[3], ospan;
  AVQ_TRY(cross_inputs(s, dtype, Q, q_strides, K, k_strides, V, v_strides, kv_lens, key_mask, &a, spans));
  AVQ_TRY(need_ptr(O, "O"));
  AVQ_TRY(view(o_strides, s.B, s.Hq, s.Nq, s.d, dtype, kWritten, "O", &a.os, &ospan));
  AVQ_TRY(optional_vector(lse, "lse"));
  const CrossPlan p = plan_cross(s, dtype, false);
  AVQ_TRY(check_ws(p.total(), ws, ws_bytes));
  AVQ_TRY(apart({{O, ospan, "O"},
                 {lse, (size_t)s.B * s.Hq * s.Nq * sizeof(float), "lse"},
                 {ws, p.total(), "the workspace"}},
                {{Q, spans[0], "Q"}, {K, spans[1], "K"}, {V, spans[2], "V"}, lens_of(s, kv_lens),
                 mask_of(s, key_mask)}));
  if (api_path() == AVQ_PATH_TC && dtype != AVQ_BF16)
    return api_fail(AVQ_ERR_UNSUPPORTED, "no tensor-core kernel for this type");
  if (api_injected("cross_attention"))
    return api_fail(AVQ_ERR_CUDA, "injected failure before launch (avq_cross_attention)");
  a.O = O;
  a.lse = lse;
  const bool items = p.tc && !p.few;
  a.splits = items ? p.rounds.splits : p.splits;
  a.whole = p.rounds.whole;
  a.part = static_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  LaunchLog log{};
  cudaError_t e;
  if (p.tc) {
    unsigned int* err = error_word();
    if (err == nullptr) return api_fail(AVQ_ERR_CUDA, "cannot resolve the device error word");
    e = p.few ? launch_cross_few(a, err, cs, log) : launch_cross_tc(a, err, cs, log);
  } else {
    e = p.few ? launch_cross_few_f32(a, cs, log) : launch_cross_simt(a, dtype, cs, log);
  }
  if (e == cudaSuccess && !items && a.splits > 1) e = launch_cross_join(a, dtype, cs, log);
  return api_finish(e, "cross attention launch", log);
}

avq_status avq_cross_attention_backward(const avq_cross_dims* dims, avq_dtype dtype, const void* dO,
                                        const avq_strides* do_strides, const void* Q, const avq_strides* q_strides,
                                        const void* K, const avq_strides* k_strides, const void* V,
                                        const avq_strides* v_strides, const void* O, const avq_strides* o_strides,
                                        const float* lse, const int32_t* kv_lens, const uint8_t* key_mask, void* dQ,
                                        void* dK, void* dV, void* ws, size_t ws_bytes, avq_stream_t stream) {
  api_begin();
  AVQ_TRY(check_cross(dims, dtype));
  const avq_cross_dims& s = *dims;
  CrossArgs a{};
  size_t spans[5];
  AVQ_TRY(cross_inputs(s, dtype, Q, q_strides, K, k_strides, V, v_strides, kv_lens, key_mask, &a, spans));
  AVQ_TRY(need_ptr(dO, "dO"));
  AVQ_TRY(view(do_strides, s.B, s.Hq, s.Nq, s.d, dtype, kCopied, "dO", &a.gs, &spans[3]));
  AVQ_TRY(need_ptr(O, "O"));
  AVQ_TRY(view(o_strides, s.B, s.Hq, s.Nq, s.d, dtype, kCopied, "O", &a.os, &spans[4]));
  AVQ_TRY(need_ptr(lse, "lse"));
  AVQ_TRY(need_ptr(dQ, "dQ"));
  if (s.Nk > 0) {
    AVQ_TRY(need_ptr(dK, "dK"));
    AVQ_TRY(need_ptr(dV, "dV"));
  }
  const size_t qn = (size_t)s.B * s.Hq * s.Nq * s.d, kn = (size_t)s.Bk * s.Hk * s.Nk * s.d, es = elem(dtype);
  const CrossPlan p = plan_cross(s, dtype, true);
  AVQ_TRY(check_ws(p.total(), ws, ws_bytes));
  AVQ_TRY(apart({{dQ, qn * es, "dQ"}, {dK, kn * es, "dK"}, {dV, kn * es, "dV"}, {ws, p.total(), "the workspace"}},
                {{Q, spans[0], "Q"}, {K, spans[1], "K"}, {V, spans[2], "V"}, {dO, spans[3], "dO"}, {O, spans[4], "O"},
                 {lse, (size_t)s.B * s.Hq * s.Nq * sizeof(float), "lse"}, lens_of(s, kv_lens), mask_of(s, key_mask)}));
  if (api_path() == AVQ_PATH_TC && dtype != AVQ_BF16)
    return api_fail(AVQ_ERR_UNSUPPORTED, "no tensor-core kernel for this type");
  if (api_injected("cross_attention_backward"))
    return api_fail(AVQ_ERR_CUDA, "injected failure before launch (avq_cross_attention_backward)");
  a.G = dO;
  a.O = const_cast<void*>(O);
  a.lse = const_cast<float*>(lse);
  a.dQ = dQ, a.dK = dK, a.dV = dV;
  a.part = static_cast<float*>(ws);
  a.delta = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
  if (key_mask != nullptr) a.lone = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + p.part + p.delta);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  unsigned int* err = error_word();
  if (err == nullptr) return api_fail(AVQ_ERR_CUDA, "cannot resolve the device error word");
  LaunchLog log{};
  CrossArgs q = a;
  a.splits = p.dkv_splits;
  q.splits = p.tc ? p.rounds.splits : p.dq_splits;
  q.whole = p.rounds.whole;
  q.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.dq_part);
  cudaError_t e = launch_cross_delta(a, dtype, cs, log);
  if (p.tc) {
    if (e == cudaSuccess) e = launch_cross_tc_backward(a, q, err, cs, log);
  } else {
    if (e == cudaSuccess) e = launch_cross_simt_backward(a, q, dtype, cs, log);
    if (e == cudaSuccess && p.dq_splits > 1) e = launch_partial_sum(dtype, q.part, p.dq_splits, &dQ, 1, qn, cs, log);
  }
  if (e == cudaSuccess && s.Nk > 0 && p.dkv_splits > 1) {
    void* const both[2] = {dK, dV};
    e = launch_partial_sum(dtype, a.part, p.dkv_splits, both, 2, kn, cs, log);
  }
  return api_finish(e, "cross attention backward launch", log);
}

}  // extern "C"
