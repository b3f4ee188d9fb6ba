// medusa_rope and medusa_paged_append: the rotary embedding in the forms
// backbones use, and the entry of a chunk's keys and values into the paged
// cache with the rotation on the way.
//
// Pair (x0, x1) of a head at position p turns by a = p f_i:
//   y0 = m (x0 cos a - x1 sin a),  y1 = m (x1 cos a + x0 sin a).
// The gradient of the inputs is the same turn by -a.
//
// The angle is formed in whole numbers: f_i / 2 pi modulo 1 as a 64-bit
// fraction (host, from double), times the int32 position modulo 2^64, is the
// angle in turns with an error of at most |p| 2^-64 turns beyond that of the
// double frequency.  The nearest quarter turn is split off in the integer, so
// sincospif sees at most an eighth of a turn, rounded to 24 bits.
//
// Bandwidth bounds both calls (each element is read and written once, about 10
// instructions a pair).  Many small CTAs hide the loads: 128 threads, a token each
// (more when a token has fewer than 128 tasks of two vectors), one task in flight a
// thread, its angles formed once into shared memory while the first loads are on
// their way.  Measured, 10782 prompt tokens with 32 + 8 + 8 heads entered into
// the cache: 44 us (6.0 TB/s), in sixteen CTAs an SM (32 registers); with 256 threads 56 us, with two, three or four
// tasks in flight 49 to 52 us, with the next task's loads ahead of the turn 48 us
// (registers: fewer CTAs on an SM), with a thread's angles kept in registers over its
// heads 51 us (the same).  32 layers of 64 tokens with 32 + 32 heads: 13.1
// us; 16384 fp32 tokens with 32 + 8 heads: 99 us (6.8 TB/s).
#include <cmath>

#include "divide.h"
#include "host_util.h"
#include "paged.cuh"

namespace medusa {
namespace paged {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxTokens = 8;  // tokens per CTA

struct RopeArgs {
  const void *q, *k, *v;  // q, k, v may be NULL
  long long ldq, ldk, ldv;
  void *q_out, *k_out;  // dense; k_out NULL when keys enter the cache
  void *k_pages, *v_pages;
  const int32_t *pos, *q_start, *prefix_len;
  int32_t* d_status;
  Cache cache;
  int nl, T, B, Hq, Hkv, d, rotary, inverse;
  int tokens;  // per CTA
  unsigned per_tok_inv;   // the reciprocal of a token's tasks; 0 where a CTA has one token
  unsigned per_head_inv;  // floor(2^32 / n) + 1: the high word of a product divides by n > 1
  float magnitude;
  unsigned long long turn[MEDUSA_MAX_HEAD_DIM / 2];
};

template <int BYTES>
struct Vec;
template <>
struct Vec<16> { using type = uint4; };
template <>
struct Vec<8> { using type = uint2; };
template <>
struct Vec<4> { using type = uint32_t; };
template <>
struct Vec<2> { using type = uint16_t; };

// W elements as one load or store.
template <typename T, int W>
using Chunk = typename Vec<W * sizeof(T)>::type;

template <int W>
__device__ __forceinline__ void unpack(const Chunk<float, W>& c, float* f) {
  const float* e = reinterpret_cast<const float*>(&c);
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = e[i];
}
template <int W>
__device__ __forceinline__ void unpack(const Chunk<uint16_t, W>& c, float* f) {
  if constexpr (W == 1) {
    f[0] = bf16_bits_to_f32(c);
  } else {
    const uint32_t* e = reinterpret_cast<const uint32_t*>(&c);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      f[2 * i] = __uint_as_float(e[i] << 16);
      f[2 * i + 1] = __uint_as_float(e[i] & 0xffff0000u);
    }
  }
}
template <int W>
__device__ __forceinline__ void pack(const float* f, Chunk<float, W>& c) {
  float* e = reinterpret_cast<float*>(&c);
#pragma unroll
  for (int i = 0; i < W; ++i) e[i] = f[i];
}
template <int W>
__device__ __forceinline__ void pack(const float* f, Chunk<uint16_t, W>& c) {
  if constexpr (W == 1) {
    c = (uint16_t)bf16x2_rn(f[0], 0.f);
  } else {
    uint32_t* e = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) e[i] = bf16x2_rn(f[2 * i], f[2 * i + 1]);
  }
}

// (cos, sin) of p turns of `turn` 2^-64, times m.
__device__ __forceinline__ float2 turn_of(int p, unsigned long long turn, int inverse, float m) {
  unsigned long long v = (unsigned long long)(long long)p * turn;
  if (inverse) v = 0ull - v;
  const unsigned quarter = (unsigned)((v + (1ull << 61)) >> 62);           // nearest quarter turn, modulo 4
  const long long rest = (long long)(v - ((unsigned long long)quarter << 62));  // [-2^61, 2^61)
  float s, c;
  sincospif((float)(int)(rest >> 31) * 2.3283064365386963e-10f, &s, &c);  // rest 2^-63 half turns, in units of 2^-32
  float cc = (quarter & 1) ? -s : c, ss = (quarter & 1) ? c : s;
  if (quarter & 2) {
    cc = -cc;
    ss = -ss;
  }
  return make_float2(cc * m, ss * m);
}

// Sixteen CTAs an SM, 32 registers: with 40, which the look for a token's sequence would take,
// the prompts' 44 us are 48.
template <typename T, int W, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 16) rope_kernel(const __grid_constant__ RopeArgs a) {
  using C = Chunk<T, W>;
  // Angle e of the W that vector c needs lies at (e / 2, c, e % 2): lanes with
  // neighbouring vectors then read neighbouring words.
  __shared__ __align__(16) float2 cs[kRopeMaxTokens][MEDUSA_MAX_HEAD_DIM / 2];
  __shared__ int s_slot[kRopeMaxTokens];  // pool row, -1: not entered, -2: nothing of the token is written
  __shared__ int s_pos[kRopeMaxTokens];
  pdl_wait();
  pdl_trigger();
  const unsigned per_head = a.d / (2 * W), turned = a.rotary / (2 * W), half = a.rotary / 2;
  const unsigned hq = a.q ? a.Hq : 0, hk = a.k ? a.Hkv : 0, hv = a.v ? a.Hkv : 0;
  const unsigned per_tok = (hq + hk + hv) * per_head;
  const long long tok0 = (long long)blockIdx.x * a.tokens, all = (long long)a.nl * a.T;
  const int n_tok = (int)(all - tok0 < a.tokens ? all - tok0 : a.tokens);
  const unsigned tasks = per_tok * (unsigned)n_tok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // One task: 2 W elements of one head, the two members of W pairs or a plain copy.
  struct Task {
    const T *s0, *s1;
    unsigned tok, head, c;
  };
  auto find = [&](unsigned id) {
    Task t;
    t.tok = quotient(id, a.per_tok_inv);
    const unsigned r = id - t.tok * per_tok;
    t.head = per_head == 1 ? r : __umulhi(r, a.per_head_inv);
    t.c = r - t.head * per_head;
    const long long at = tok0 + t.tok;
    const T* base;
    const bool value = t.head >= hq + hk;
    if (t.head < hq) base = static_cast<const T*>(a.q) + at * a.ldq + (long long)t.head * a.d;
    else if (!value) base = static_cast<const T*>(a.k) + at * a.ldk + (long long)(t.head - hq) * a.d;
    else base = static_cast<const T*>(a.v) + at * a.ldv + (long long)(t.head - hq - hk) * a.d;
    const bool split = !INTER && !value && t.c < turned;
    t.s0 = base + (split ? t.c * W : !INTER && !value && t.c >= turned ? a.rotary + (t.c - turned) * 2 * W : t.c * 2 * W);
    t.s1 = split ? t.s0 + half : t.s0 + W;
    return t;
  };

  Task t;
  C x0, x1;
  auto load = [&](unsigned id) {
    t = find(id);
    x0 = *reinterpret_cast<const C*>(t.s0);
    x1 = *reinterpret_cast<const C*>(t.s1);
  };
  if (threadIdx.x < tasks) load(threadIdx.x);  // in flight while the angles are formed

  if (a.k_pages) {
    // Token tok's sequence is the first whose starts hold it.
    for (int tk = warp; tk < n_tok; tk += kRopeThreads / 32) {
      const int t = (int)((tok0 + tk) % a.T);
      int b = a.B;
      bool odd = false;  // some starts decrease or lie outside the tokens
#pragma unroll 1
      for (int j = lane; j < a.B; j += 32) {
        const int q0 = a.q_start[j], q1 = a.q_start[j + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.T) odd = true;
        else if (q0 <= t && t < q1) b = min(b, j);
      }
      b = __reduce_min_sync(0xffffffffu, b);
      int slot = -2, p = 0;
      int err = MEDUSA_DEV_OK, top = -1;
      if (__any_sync(0xffffffffu, odd)) {
        if (lane == 0) set_status(a.d_status, MEDUSA_DEV_BAD_LENGTH);
#pragma unroll 1
        for (int j = lane; j < b; j += 32) top = max(top, end_of(a.q_start, a.T, j));
        top = __reduce_max_sync(0xffffffffu, top);
      }
      if (b < a.B) {
        const int q0 = a.q_start[b], n = a.q_start[b + 1] - q0, L = a.prefix_len[b];
        if (L < 0 || L > a.cache.rows() || q0 < top) {
          err = MEDUSA_DEV_BAD_LENGTH;
        } else {
          const int row = L + (t - q0);
          p = row;
          slot = -1;
          if (L > a.cache.rows() - n) err = MEDUSA_DEV_CACHE_OVERFLOW;
          else if ((slot = pool_row(a.cache, b, row)) < 0) err = MEDUSA_DEV_BAD_INDEX;
        }
      }
      if (err && lane == 0) set_status(a.d_status, err);
      if (lane == 0) {
        s_slot[tk] = slot;
        s_pos[tk] = a.pos ? a.pos[t] : p;
      }
    }
    __syncthreads();
  }
  for (unsigned j = threadIdx.x; j < half * n_tok; j += kRopeThreads) {
    const unsigned tk = j / half, i = j - tk * half;
    const int p = a.k_pages ? s_pos[tk] : a.pos[(tok0 + tk) % a.T];
    const unsigned c = i / W, e = i % W;
    cs[tk][W == 1 ? c : ((e >> 1) * turned + c) * 2 + (e & 1)] = turn_of(p, a.turn[i], a.inverse, a.magnitude);
  }
  __syncthreads();

  for (unsigned id = threadIdx.x; id < tasks; id += kRopeThreads) {
    if (id != threadIdx.x) load(id);
    const long long at = tok0 + t.tok;
    const int slot = a.k_pages ? s_slot[t.tok] : 0;
    if (slot == -2) continue;
    T* dst;
    if (t.head < hq) {
      dst = static_cast<T*>(a.q_out) + (at * a.Hq + t.head) * a.d;
    } else {
      const bool value = t.head >= hq + hk;
      const unsigned h = t.head - hq - (value ? hk : 0u);
      if (a.k_pages) {
        if (slot < 0) continue;
        const long long row = (at / a.T) * ((long long)a.cache.n_pages * a.cache.page_size) + slot;
        dst = static_cast<T*>(value ? a.v_pages : a.k_pages) + (row * a.Hkv + h) * a.d;
      } else {
        dst = static_cast<T*>(a.k_out) + (at * a.Hkv + h) * a.d;
      }
      if (value) {
        dst += t.c * 2 * W;
        *reinterpret_cast<C*>(dst) = x0;
        *reinterpret_cast<C*>(dst + W) = x1;
        continue;
      }
    }
    if (t.c >= turned) {  // behind the turned part
      dst += a.rotary + (t.c - turned) * 2 * W;
      *reinterpret_cast<C*>(dst) = x0;
      *reinterpret_cast<C*>(dst + W) = x1;
      continue;
    }
    float x[2 * W], y[2 * W];
    unpack<W>(x0, x);
    unpack<W>(x1, x + W);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float2 f = cs[t.tok][W == 1 ? t.c : ((e >> 1) * turned + t.c) * 2 + (e & 1)];
      const int i0 = INTER ? 2 * e : e, i1 = INTER ? 2 * e + 1 : W + e;
      y[i0] = x[i0] * f.x - x[i1] * f.y;
      y[i1] = x[i1] * f.x + x[i0] * f.y;
    }
    C y0, y1;
    pack<W>(y, y0);
    pack<W>(y + W, y1);
    dst += INTER ? t.c * 2 * W : t.c * W;
    *reinterpret_cast<C*>(dst) = y0;
    *reinterpret_cast<C*>(dst + (INTER ? W : half)) = y1;
  }
}

// Elements per vector: the widest of 16 bytes and below that divides every
// offset the kernel forms.
static int rope_width(const RopeArgs& a, size_t es) {
  for (int w = (int)(16 / es); w > 1; w /= 2) {
    auto fits = [&](const void* p) { return (reinterpret_cast<uintptr_t>(p) & (w * es - 1)) == 0; };
    if (a.d % (2 * w) || a.rotary % (2 * w)) continue;
    if (!fits(a.q) || !fits(a.k) || !fits(a.v) || !fits(a.q_out) || !fits(a.k_out) || !fits(a.k_pages) || !fits(a.v_pages))
      continue;
    if ((a.q && a.ldq % w) || (a.k && a.ldk % w) || (a.v && a.ldv % w)) continue;
    return w;
  }
  return 1;
}

template <typename T, int W>
static void rope_go(const RopeArgs& a, bool inter, unsigned grid, cudaStream_t s) {
  if (inter) launch_pdl(rope_kernel<T, W, true>, dim3(grid), dim3(kRopeThreads), 0, s, a);
  else launch_pdl(rope_kernel<T, W, false>, dim3(grid), dim3(kRopeThreads), 0, s, a);
}

static medusa_status rope_launch(RopeArgs& a, const medusa_rope_plan* plan, medusa_dtype dt, cudaStream_t s) {
  if (plan) {
    a.rotary = plan->rotary_dim;
    a.magnitude = plan->magnitude;
    for (int i = 0; i < a.rotary / 2; ++i) a.turn[i] = plan->turn[i];
  }
  const int w = rope_width(a, dtype_bytes(dt));
  const long long all = (long long)a.nl * a.T;
  const long long per_tok = (long long)((a.q ? a.Hq : 0) + (a.k ? a.Hkv : 0) + (a.v ? a.Hkv : 0)) * (a.d / (2 * w));
  // Tokens per CTA: as many as give every thread a task, but first two CTAs per SM.
  long long n = kRopeThreads / per_tok;
  const long long spread = all / (2 * device_sm_count());
  if (n > spread) n = spread;
  a.tokens = n < 1 ? 1 : n > kRopeMaxTokens ? kRopeMaxTokens : (int)n;
  // Exact: with several tokens there are at most kRopeThreads tasks, of one or more to a
  // token; a vector's number within its token times the vectors of a head stays below 2^32
  // (3 x 65535 heads of at most 128 vectors).
  const unsigned per_head = (unsigned)(a.d / (2 * w));
  a.per_tok_inv = a.tokens == 1 ? 0u : reciprocal((unsigned)per_tok);
  a.per_head_inv = (unsigned)((1ull << 32) / per_head) + 1;
  const unsigned grid = (unsigned)((all + a.tokens - 1) / a.tokens);
  const bool inter = plan && plan->interleaved;
  if (dt == MEDUSA_BF16) {
    if (w == 8) rope_go<uint16_t, 8>(a, inter, grid, s);
    else if (w == 4) rope_go<uint16_t, 4>(a, inter, grid, s);
    else if (w == 2) rope_go<uint16_t, 2>(a, inter, grid, s);
    else rope_go<uint16_t, 1>(a, inter, grid, s);
  } else {
    if (w == 4) rope_go<float, 4>(a, inter, grid, s);
    else if (w == 2) rope_go<float, 2>(a, inter, grid, s);
    else rope_go<float, 1>(a, inter, grid, s);
  }
  return launch_status();
}

// Bytes from the first to behind the last element of [nl][T][H][d] with token stride ld.
static size_t span(int nl, int T, long long ld, int H, int d, size_t es) {
  return ((size_t)((long long)nl * T - 1) * (size_t)ld + (size_t)H * d) * es;
}

static bool plan_ok(const medusa_rope_plan* p, int d) {
  return p->rotary_dim >= 2 && p->rotary_dim % 2 == 0 && p->rotary_dim <= d && std::isfinite(p->magnitude);
}

}  // namespace paged
}  // namespace medusa

using namespace medusa;
using namespace medusa::paged;

extern "C" medusa_status medusa_rope_plan_init(int rotary_dim, int interleaved, double base, medusa_rope_scaling scaling,
                                               double factor, double low, double high, int original_len,
                                               double magnitude, medusa_rope_plan* out) {
  if (!out || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > MEDUSA_MAX_HEAD_DIM) return MEDUSA_ERR_INVALID_ARG;
  if (!(base > 0.0) || !std::isfinite(base) || !std::isfinite(magnitude)) return MEDUSA_ERR_INVALID_ARG;
  const int kind = (int)scaling;
  if (kind < MEDUSA_ROPE_PLAIN || kind > MEDUSA_ROPE_RAMP) return MEDUSA_ERR_INVALID_ARG;
  if (kind != MEDUSA_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor))) return MEDUSA_ERR_INVALID_ARG;
  const bool bands = kind == MEDUSA_ROPE_BANDS, ramp = kind == MEDUSA_ROPE_RAMP;
  if ((bands || ramp) && !(low > 0.0 && high > low && std::isfinite(high) && original_len >= 1)) return MEDUSA_ERR_INVALID_ARG;
  if (ramp && !(base > 1.0)) return MEDUSA_ERR_INVALID_ARG;
  const double kTwoPi = 6.283185307179586476925286766559;
  double from = 0.0, to = 1.0;
  if (ramp) {
    auto pair = [&](double turns) { return rotary_dim * std::log(original_len / (kTwoPi * turns)) / (2.0 * std::log(base)); };
    from = std::fmax(std::floor(pair(high)), 0.0);
    to = std::fmin(std::ceil(pair(low)), (double)(rotary_dim - 1));
  }
  *out = medusa_rope_plan{};
  out->rotary_dim = rotary_dim;
  out->interleaved = interleaved ? 1 : 0;
  out->magnitude = (float)magnitude;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0, g = f;
    if (kind == MEDUSA_ROPE_LINEAR) {
      g = f / factor;
    } else if (bands || ramp) {
      keep = bands ? (original_len * f / kTwoPi - low) / (high - low) : 1.0 - (i - from) / std::fmax(to - from, 0.001);
      keep = std::fmin(std::fmax(keep, 0.0), 1.0);
      g = keep * f + (1.0 - keep) * f / factor;
    }
    const double turns = g / kTwoPi;
    if (!std::isfinite(turns)) return MEDUSA_ERR_INVALID_ARG;
    out->turn[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
  }
  return MEDUSA_OK;
}

extern "C" medusa_status medusa_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, const int32_t* pos,
                                     const medusa_rope_plan* plan, int inverse, int n_layers, int T, int Hq, int Hkv,
                                     int d, medusa_dtype dt, void* q_out, void* k_out, medusa_stream_t stream) {
  if (!q || !q_out || !pos || !plan || (k != nullptr) != (k_out != nullptr) || !dtype_ok(dt)) return MEDUSA_ERR_INVALID_ARG;
  if (n_layers < 1 || T < 1 || Hq < 1 || (k && Hkv < 1) || d < 2 || d % 2 || d > MEDUSA_MAX_HEAD_DIM) return MEDUSA_ERR_INVALID_ARG;
  if ((long long)n_layers * T > 0x7fffffffll || Hq > 65535 || Hkv > 65535 || !plan_ok(plan, d)) return MEDUSA_ERR_INVALID_ARG;
  if (ldq < (int64_t)Hq * d || (k && ldk < (int64_t)Hkv * d)) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt);
  const uintptr_t all = (uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out;
  if ((all & (es - 1)) || ((uintptr_t)pos & 3)) return MEDUSA_ERR_INVALID_ARG;
  const size_t nq = span(n_layers, T, ldq, Hq, d, es), nk = k ? span(n_layers, T, ldk, Hkv, d, es) : 0;
  const size_t oq = span(n_layers, T, (long long)Hq * d, Hq, d, es), ok = k ? span(n_layers, T, (long long)Hkv * d, Hkv, d, es) : 0;
  const size_t np = (size_t)T * 4;
  if (!(q_out == q && ldq == (int64_t)Hq * d) && overlaps(q, nq, q_out, oq)) return MEDUSA_ERR_ALIAS;
  if (overlaps(q_out, oq, pos, np)) return MEDUSA_ERR_ALIAS;
  if (k) {
    if (!(k_out == k && ldk == (int64_t)Hkv * d) && overlaps(k, nk, k_out, ok)) return MEDUSA_ERR_ALIAS;
    if (overlaps(q_out, oq, k, nk) || overlaps(q_out, oq, k_out, ok) || overlaps(k_out, ok, q, nq) || overlaps(k_out, ok, pos, np))
      return MEDUSA_ERR_ALIAS;
  }
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.ldq = ldq;
  a.ldk = ldk;
  a.q_out = q_out;
  a.k_out = k_out;
  a.pos = pos;
  a.nl = n_layers;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.inverse = inverse ? 1 : 0;
  return rope_launch(a, plan, dt, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" medusa_status medusa_paged_append(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                                             int64_t ldv, const int32_t* pos, const medusa_rope_plan* plan,
                                             const int32_t* page_table, const int32_t* q_start, const int32_t* prefix_len,
                                             int n_layers, int T, int B, int Hq, int Hkv, int d, int n_pages,
                                             int page_size, int max_pages, medusa_dtype dt, void* q_out, void* k_pages,
                                             void* v_pages, int32_t* d_status, medusa_stream_t stream) {
  if (!k || !v || !page_table || !q_start || !prefix_len || !k_pages || !v_pages || (q != nullptr) != (q_out != nullptr))
    return MEDUSA_ERR_INVALID_ARG;
  if (!dtype_ok(dt) || n_layers < 1 || T < 1 || B < 1 || (q && Hq < 1) || Hkv < 1 || d < 2 || d % 2 || d > MEDUSA_MAX_HEAD_DIM)
    return MEDUSA_ERR_INVALID_ARG;
  if (!cache_sizes_ok(n_layers, B, n_pages, page_size, max_pages) || (long long)n_layers * T > 0x7fffffffll) return MEDUSA_ERR_INVALID_ARG;
  if (Hq > 65535 || Hkv > 65535 || (plan && !plan_ok(plan, d))) return MEDUSA_ERR_INVALID_ARG;
  if ((q && ldq < (int64_t)Hq * d) || ldk < (int64_t)Hkv * d || ldv < (int64_t)Hkv * d) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt);
  const uintptr_t all = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_pages | (uintptr_t)v_pages;
  const uintptr_t words = (uintptr_t)pos | (uintptr_t)page_table | (uintptr_t)q_start | (uintptr_t)prefix_len | (uintptr_t)d_status;
  if ((all & (es - 1)) || (words & 3)) return MEDUSA_ERR_INVALID_ARG;
  const size_t np = (size_t)n_layers * n_pages * page_size * Hkv * d * es;
  const size_t nk = span(n_layers, T, ldk, Hkv, d, es), nv = span(n_layers, T, ldv, Hkv, d, es);
  const size_t nq = q ? span(n_layers, T, ldq, Hq, d, es) : 0, oq = q ? span(n_layers, T, (long long)Hq * d, Hq, d, es) : 0;
  if (overlaps(k_pages, np, v_pages, np)) return MEDUSA_ERR_ALIAS;
  for (const void* pool : {(const void*)k_pages, (const void*)v_pages})
    if (overlaps(pool, np, k, nk) || overlaps(pool, np, v, nv) || (q && (overlaps(pool, np, q, nq) || overlaps(pool, np, q_out, oq))))
      return MEDUSA_ERR_ALIAS;
  if (q) {
    if (!(q_out == q && ldq == (int64_t)Hq * d) && overlaps(q, nq, q_out, oq)) return MEDUSA_ERR_ALIAS;
    if (overlaps(q_out, oq, k, nk) || overlaps(q_out, oq, v, nv)) return MEDUSA_ERR_ALIAS;
  }
  const size_t nb = (size_t)B * 4;
  for (const Region& r : {Region{page_table, nb * max_pages}, Region{q_start, nb + 4}, Region{prefix_len, nb}, Region{pos, (size_t)T * 4}})
    if (overlaps_any(r, {{q_out, oq}, {k_pages, np}, {v_pages, np}})) return MEDUSA_ERR_ALIAS;
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.q_out = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.pos = pos;
  a.q_start = q_start;
  a.prefix_len = prefix_len;
  a.d_status = d_status;
  a.cache = Cache{page_table, n_pages, page_size, max_pages};
  a.nl = n_layers;
  a.T = T;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.magnitude = 1.f;
  return rope_launch(a, plan, dt, reinterpret_cast<cudaStream_t>(stream));
}
