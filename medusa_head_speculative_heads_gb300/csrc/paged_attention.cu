// medusa_paged_attention and medusa_paged_tree_attention: entry points, the
// CUDA-core kernel (fp32, and what the tensor-core kernel does not take) and
// the merge of items that several CTAs share.
//
// Paper review ("Medusa: Simple LLM Inference Acceleration Framework with
// Multiple Decoding Heads"), section "Medusa 的三个核心组件": each token attends
// to its own predecessors; "局限性": the cache grows with batch and length, so
// it is kept in pages here.
//
// One pass over the keys with a running maximum m and sum l per row:
//   m' = max(m, max s), f = 2^(m - m'), l' = f l + sum 2^(s - m'),
//   O' = f O + sum 2^(s - m') v,
// s in the log2 domain (scale log2 e folded in); at the end O / l.  Two parts
// of a row combine the same way.
#include "host_util.h"
#include "medusa_test_hooks.h"
#include "paged_attn.cuh"

namespace medusa {
namespace paged {

constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
}

// A tile is 16 RM rows x 64 keys; thread (ty, tx) of 16 x 16 holds rows
// ty RM .. + RM - 1: their scores of keys tx + 16 j and their columns
// 4 tx + 64 j .. + 3 of O, in registers.  Q is fp32 in shared memory, K and V as
// they are stored, rows padded by four elements, so the sixteen rows a quarter
// or half warp reads lie in different banks.  Probabilities pass through shared
// memory between threads of one half warp.  K and V have one buffer each, filled by
// asynchronous copies: the next K under the products with V, V under the scores.
// A warp none of whose rows exists takes part in the copies only.
// Products are taken two at a time (fma.rn.f32x2: over even and odd columns in the
// scores, over pairs of columns in the sums).  Measured, fp32, 5 ragged sequences of
// up to 331 tokens behind up to 1338 rows, 8 + 4 heads of 64: the kernel 86 us, with the
// merge 90 to 98 us, 21 TFLOP/s (with single products and loads between two barriers 114 us).
// Shared memory's pipe bounds it, busy for 64 % of the clocks (the FMA pipe for 47 %): a
// 16-byte load takes four of them when lanes read several rows and two as a broadcast,
// 24 for the 64 products of four columns.  A warp of 8 rows x 64 keys, each K row
// read once and Q as broadcasts, takes as many and measured 101 us; 128 threads with 8 x
// 4 scores each take 16 and measured 98 to 101 (too few warps, or registers spilled).
template <int DC>
__host__ __device__ constexpr int simt_pitch() { return 16 * DC + 4; }
template <typename T, int DC, int RM>
constexpr size_t simt_smem() {
  return (size_t)16 * RM * (simt_pitch<DC>() + kSimtKeys + 4) * sizeof(float) + (size_t)2 * kSimtKeys * simt_pitch<DC>() * sizeof(T);
}

// Four elements into shared memory; `some` false: zeros, and `from` is not read.
template <typename T>
__device__ __forceinline__ void copy4_async(T* to, const T* from, bool some) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(from), "n"(4 * sizeof(T)),
               "r"(some ? (int)(4 * sizeof(T)) : 0)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// CTAs that fit an SM, by registers and shared memory.
constexpr int simt_ctas(int DC, int RM) { return RM == 1 ? (DC <= 4 ? 3 : DC <= 8 ? 2 : 1) : DC <= 4 ? 2 : 1; }

template <typename T, int DC, int RM>
__global__ void __launch_bounds__(kSimtThreads, simt_ctas(DC, RM)) paged_attn_simt_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int R = 16 * RM, DP = simt_pitch<DC>(), PP = kSimtKeys + 4;
  extern __shared__ float4 smem4[];
  float* Qs = reinterpret_cast<float*>(smem4);
  float* Ps = Qs + R * DP;
  T* Ks = reinterpret_cast<T*>(Ps + R * PP);
  T* Vs = Ks + kSimtKeys * DP;
  __shared__ long long sh[70];
  __shared__ const T *s_k[2][kSimtKeys], *s_v[2][kSimtKeys];  // row starts of a tile's keys (NULL: zeros)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (blockIdx.x == 0)
    for (int b = tid; b < a.w.B; b += kSimtThreads)
      if (!seq_of(a.w, b).ok) set_status(a.d_status, MEDUSA_DEV_BAD_LENGTH);
  Plan pl;
  Item it;
  const bool any = plan_find(a.w, pl, it, sh, blockIdx.x);
  if (tid == 0) note_shared(a, pl, it, any);
  if (!any) return;
  const long long u0 = pl.Q * blockIdx.x, u1 = u0 + pl.Q < pl.U ? u0 + pl.Q : pl.U;
  const int dv = a.d / 4;

  for (long long u = u0; u < u1;) {
    const long long end = it.first + it.tiles < u1 ? it.first + it.tiles : u1;
    const int t0 = (int)(u - it.first), t1 = (int)(end - it.first);
    const int l = it.lg / a.w.nh, kvh = it.lg % a.w.nh / a.nsub;
    const int pre = a.w.N ? (it.s.L + kSimtKeys - 1) / kSimtKeys : it.tiles;  // tiles of cache rows
    const int rows_end = a.w.N ? it.s.L : it.s.L + min(it.s.len, (it.i + 1) * a.w.ctok);
    // Where the keys of tile t lie.
    auto find_rows = [&](int t) {
      if (tid >= kSimtKeys) return;
      const T *k = nullptr, *v = nullptr;
      if (t < pre) {
        const int j = t * kSimtKeys + tid;
        if (j < rows_end) {
          const int slot = pool_row(a.cache, it.b, j);
          if (slot >= 0) {
            const size_t at = (((size_t)l * a.cache.n_pages * a.cache.page_size + slot) * a.Hkv + kvh) * a.d;
            k = static_cast<const T*>(a.k_pages) + at;
            v = static_cast<const T*>(a.v_pages) + at;
          } else {
            set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
          }
        }
      } else {
        const int j = (t - pre) * kSimtKeys + tid;
        if (j < a.w.N) {
          const size_t at = (((size_t)l * a.w.T + it.s.q0 + j) * a.Hkv + kvh) * a.d;
          k = static_cast<const T*>(a.kt) + at;
          v = static_cast<const T*>(a.vt) + at;
        }
      }
      s_k[t & 1][tid] = k;
      s_v[t & 1][tid] = v;
    };
    // Brings a tile's rows into Ks or Vs.
    auto bring = [&](T* to, const T* const* from) {
#pragma unroll
      for (int i = 0; i < DC; ++i) {
        const int idx = tid + i * kSimtThreads, r = idx / (4 * DC), c = idx - r * (4 * DC);
        const T* x = from[r];
        const bool some = x && c < dv;
        copy4_async(to + r * DP + 4 * c, some ? x + 4 * c : static_cast<const T*>(a.k_pages), some);
      }
    };
    find_rows(t0);
    __syncthreads();  // Qs and Ks of the item before are no longer read
    bring(Ks, s_k[t0 & 1]);
    {
      constexpr int kAtOnce = 4;
      for (int i0 = tid; i0 < R * 4 * DC; i0 += kAtOnce * kSimtThreads) {
        float4 v[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          const int idx = i0 + e * kSimtThreads, r = idx / (4 * DC), c = idx - r * (4 * DC);
          v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (idx >= R * 4 * DC) continue;
          const Row x = row_of(a, it, r);
          if (x.ok && c < dv)
            v[e] = load4(static_cast<const T*>(a.q) + ((long long)l * a.w.T + it.s.q0 + x.tok) * a.ldq + (long long)x.h * a.d + 4 * c);
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          const int idx = i0 + e * kSimtThreads, r = idx / (4 * DC), c = idx - r * (4 * DC);
          if (idx < R * 4 * DC) store4(Qs + r * DP + 4 * c, v[e]);
        }
      }
    }
    Row row[RM];
    float m[RM], sum[RM];
    uint64_t o[RM][DC / 4][2];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      row[i] = row_of(a, it, ty * RM + i);
      m[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int c = 0; c < DC / 4; ++c) o[i][c][0] = o[i][c][1] = 0;
    }

    bool live = false;
#pragma unroll
    for (int i = 0; i < RM; ++i) live |= row[i].ok;
    live = __any_sync(0xffffffffu, live);

    for (int t = t0; t < t1; ++t) {
      copies_done();
      __syncthreads();  // K has arrived, V of the tile before is no longer read
      bring(Vs, s_v[t & 1]);
      if (t + 1 < t1) find_rows(t + 1);
      uint64_t s2[RM][4];  // sums over even and over odd columns
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = 0;
      for (int c = 0; live && c < dv; ++c) {
        float4 kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = load4(Ks + (tx + 16 * j) * DP + 4 * c);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const float4 qq = load4(Qs + (ty * RM + i) * DP + 4 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s2[i][j] = fma2(pack2(qq.z, qq.w), pack2(kk[j].z, kk[j].w), fma2(pack2(qq.x, qq.y), pack2(kk[j].x, kk[j].y), s2[i][j]));
        }
      }
      float s[RM][4];
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = (t < pre ? t : t - pre) * kSimtKeys + tx + 16 * j;
          bool see;
          if (t >= pre) see = row[i].ok && key < a.w.N && ((a.mask[(size_t)row[i].tok * a.W + (key >> 5)] >> (key & 31)) & 1u);
          else see = row[i].ok && key < (a.w.N ? it.s.L : it.s.L + row[i].tok + 1);
          const float2 z = unpack2(s2[i][j]);
          s[i][j] = see ? (z.x + z.y) * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int e = 8; e; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
        const float mn = fmaxf(m[i], mx), off = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[i] - off);  // 0 for the first keys seen
        m[i] = mn;
        float rs = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - off);
          rs += p;
          Ps[(ty * RM + i) * PP + tx + 16 * j] = p;
        }
        sum[i] = fmaf(sum[i], f, rs);  // this thread's share; its sixteen are added at the end
#pragma unroll
        for (int c = 0; c < DC / 4; ++c) {
          o[i][c][0] = fma2(o[i][c][0], pack2(f, f), 0);
          o[i][c][1] = fma2(o[i][c][1], pack2(f, f), 0);
        }
      }
      copies_done();
      __syncthreads();  // V has arrived, K is no longer read, the probabilities are written
      if (t + 1 < t1) bring(Ks, s_k[(t + 1) & 1]);
      if (!live) continue;
#pragma unroll 2
      for (int j = 0; j < kSimtKeys; j += 4) {
        float4 p[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) p[i] = load4(Ps + (ty * RM + i) * PP + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int c = 0; c < DC / 4; ++c) {
            const float4 v = load4(Vs + (j + e) * DP + 4 * tx + 64 * c);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
              const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
              o[i][c][0] = fma2(pack2(pe, pe), pack2(v.x, v.y), o[i][c][0]);
              o[i][c][1] = fma2(pack2(pe, pe), pack2(v.z, v.w), o[i][c][1]);
            }
          }
        }
      }
      __syncwarp();
    }

    const bool whole = t0 == 0 && t1 == it.tiles;
    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      float ls = sum[i];
#pragma unroll
      for (int e = 8; e; e >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, e);
      if (!row[i].ok) continue;
      const size_t at = whole ? out_row(a, it, row[i]) : (size_t)slot * a.R + ty * RM + i;  // in lse or part_ml
      const float f = whole ? row_scale(a, it.s.L, row[i].tok, ls) : 1.f;
#pragma unroll
      for (int c = 0; c < DC / 4; ++c) {
        const int col = 4 * tx + 64 * c;
        if (col >= a.d) continue;
        const float2 lo = unpack2(o[i][c][0]), hi = unpack2(o[i][c][1]);
        const float4 v = make_float4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
        if (whole) store4(static_cast<T*>(a.out) + at * a.d + col, v);
        else store4(part_at(a, slot, ty * RM + i, col / 4), v);
      }
      if (tx == 0) {
        if (!whole) a.part_ml[at] = make_float2(m[i], ls);
        else if (a.lse) a.lse[at] = lse_of(m[i], ls);
      }
    }
    u = end;
    if (u < u1 && !next_item(a.w, sh[63] != 0, it)) break;
  }
}

// Adds the parts of every item that several CTAs share.  The CTA boundary c
// (tile c Q, c = 1 .. C - 1) belongs to the item it falls inside; the first
// boundary inside an item merges all of its parts, in the order of the CTAs:
// O = sum 2^(m_p - M) O_p, l = sum 2^(m_p - M) l_p, M = max m_p.  The attention
// kernel's CTAs have left the items they found.  Latency bounds it, so it is spread
// over all SMs.  Slots of up to 64 rows: one warp per row (its lanes share the
// columns, there may be one row and a hundred parts), eight warps a CTA, eight CTAs a boundary.
template <typename T>
__global__ void __launch_bounds__(256) paged_attn_merge_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const Shared sd = a.shared[blockIdx.x + 1];
  if (sd.first < 0) return;
  const Item& it = sd.it;
  const int first = sd.first, last = sd.last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = blockIdx.y * 8 + warp; r < a.R; r += gridDim.y * 8) {
    const Row x = row_of(a, it, r);
    if (!x.ok) continue;
    // CTA p's part: slot 1 of the CTA the item starts in, slot 0 of the others.
    auto at = [&](int p) { return (size_t)(2 * p + (p == first ? 1 : 0)) * a.R + r; };
    float M = -INFINITY;
    for (int p = first + lane; p <= last; p += 32) M = fmaxf(M, a.part_ml[at(p)].x);
    M = warp_max(M);
    const float off = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int p = first + lane; p <= last; p += 32) {
      const float2 q = a.part_ml[at(p)];
      l = fmaf(exp2f(q.x - off), q.y, l);
    }
    l = warp_sum(l);
    const float inv = row_scale(a, it.s.L, x.tok, l);
    const size_t to = out_row(a, it, x);
    for (int col = 4 * lane; col < a.d; col += 128) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = first; p <= last; ++p) {
        const size_t w = at(p);
        const float2 ml = a.part_ml[w];
        const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - off);
        const float4 v = *reinterpret_cast<const float4*>(a.part_o + w * a.d + col);  // as part_at
        if (f != 0.f) {  // a part that saw no key may hold anything
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
        }
      }
      store4(static_cast<T*>(a.out) + to * a.d + col, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
    if (a.lse && lane == 0) a.lse[to] = lse_of(M, l);
  }
}


// Slots of more rows (few parts): a lane takes one row's sixteen columns, a CTA a
// group of 32 rows.  151 boundaries in blocks of 32 tokens x 7 heads, cold caches: 24 us with a
// warp per row, 12.6 us so.
__global__ void __launch_bounds__(256) paged_attn_merge_wide_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const Shared sd = a.shared[blockIdx.x + 1];
  if (sd.first < 0) return;
  const int lane = threadIdx.x & 31, c0 = 4 * (threadIdx.x >> 5), r = blockIdx.y * 32 + lane;
  if (4 * c0 >= a.d) return;
  const Row x = row_of(a, sd.it, r);
  if (!__any_sync(0xffffffffu, x.ok)) return;
  float M = -INFINITY, l = 0.f;
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int p = sd.first; p <= sd.last; ++p) {
    // CTA p's part: slot 1 of the CTA the item starts in, slot 0 of the others.
    const int slot = 2 * p + (p == sd.first ? 1 : 0);
    const float4* from = reinterpret_cast<const float4*>(part_at(a, slot, r, c0));
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (4 * (c0 + k) < a.d) v[k] = from[k * part_rows(256)];
    const float2 q = x.ok ? a.part_ml[(size_t)slot * a.R + r] : make_float2(-INFINITY, 0.f);
    const float m = fmaxf(M, q.x), off = m == -INFINITY ? 0.f : m;
    const float f = exp2f(M - off), g = q.y == 0.f ? 0.f : exp2f(q.x - off);
    M = m;
    l = fmaf(l, f, g * q.y);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (g == 0.f || 4 * (c0 + k) >= a.d) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);  // a part that saw no key may hold anything
      o[k].x = fmaf(o[k].x, f, g * v[k].x);
      o[k].y = fmaf(o[k].y, f, g * v[k].y);
      o[k].z = fmaf(o[k].z, f, g * v[k].z);
      o[k].w = fmaf(o[k].w, f, g * v[k].w);
    }
  }
  if (!x.ok) return;
  const float inv = row_scale(a, sd.it.s.L, x.tok, l);
  const size_t to = out_row(a, sd.it, x);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (4 * (c0 + k) < a.d)
      store4(static_cast<uint16_t*>(a.out) + to * a.d + 4 * (c0 + k), make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
  if (a.lse && c0 == 0) a.lse[to] = lse_of(M, l);
}

// ------------------------------------------------------------------ host side

// How a call is divided: which kernel, its block of rows and its CTAs.
struct Division {
  bool tc;
  int R, ctas, KT, sub, nsub, tile_rows, tile_tok, ctok;
};

static int log2_of(int p) {
  int n = 0;
  while (p >> (n + 1)) ++n;
  return n;
}

static int pow2_at_most(int x) {
  int p = 1;
  while (2 * p <= x) p *= 2;
  return p;
}

static bool tc_shape(int G, int d, int page_size, medusa_dtype dt) {
  return dt == MEDUSA_BF16 && d >= 8 && d <= 128 && d % 8 == 0 && page_size % 8 == 0 && G <= 128;
}

static Division divide(int T, int B, int Hq, int Hkv, int d, int page_size, medusa_dtype dt) {
  Division v{};
  const int G = Hq / Hkv, sms = device_sm_count();
  v.tc = tc_shape(G, d, page_size, dt);
  if (v.tc) {
    // Blocks of up to 64 rows where a sequence has no more on average (decoding, trees), else of
    // two tiles of 128.  The first streams keys faster (a decoding token of 64 sequences 194 us, in the
    // wide blocks 200; a 64-node verify pass of 32 layers 113 and 120), the second reads a
    // prompt's keys a quarter as often.  The mean decides for the whole call: a prompt among so many
    // decoding sequences that it stays low runs in narrow blocks, which fill half of each product
    // (32 + 8 heads; 60 sequences 106 us and 512 tokens 23, in one call 139; with 2048 tokens, 70 us,
    // the wide blocks take both: 193).
    const bool narrow = (long long)T * G <= 64ll * B && G <= 64;
    v.R = narrow ? 64 : 256;
    v.tile_rows = narrow ? 64 : 128;
    v.ctas = sms;
    v.KT = 128;
    v.sub = G;
    v.nsub = 1;
    v.tile_tok = pow2_at_most(v.tile_rows / G);
    v.ctok = narrow ? v.tile_tok : 2 * v.tile_tok;
    return v;
  }
  // Rows of a tile: 16 when a sequence has at most 32 on average, else 64.  A tile of 16 takes about
  // half as long as one of 64 (fp32, 7 heads x 3 nodes: 15 us, in tiles of 64 22 us; 7 heads x 94 nodes 501 and 262 us).
  v.R = (long long)T * G <= 32ll * B || d > 128 ? 16 : 64;
  v.tile_rows = v.R;
  v.ctas = sms * simt_ctas(d <= 64 ? 4 : d <= 128 ? 8 : 16, v.R / 16);
  v.KT = kSimtKeys;
  v.nsub = (G + v.R - 1) / v.R;
  v.sub = (G + v.nsub - 1) / v.nsub;
  v.tile_tok = v.ctok = pow2_at_most(v.R / v.sub);
  return v;
}

static size_t ws_bytes_of(const Division& v, int d) {
  return (size_t)v.ctas * (2 * v.R * (d + 2) * sizeof(float) + sizeof(Shared));
}

template <typename T, int DC, int RM>
static medusa_status simt_go(const AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem = simt_smem<T, DC, RM>();
  auto kern = paged_attn_simt_kernel<T, DC, RM>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return MEDUSA_ERR_CUDA;
  launch_pdl(kern, dim3(a.w.ctas), dim3(kSimtThreads), smem, s, a);
  return MEDUSA_OK;
}

template <typename T>
static medusa_status simt_launch(const AttnArgs& a, cudaStream_t s) {
  if (a.R == 16) return a.d <= 64 ? simt_go<T, 4, 1>(a, s) : a.d <= 128 ? simt_go<T, 8, 1>(a, s) : simt_go<T, 16, 1>(a, s);
  return a.d <= 64 ? simt_go<T, 4, 4>(a, s) : simt_go<T, 8, 4>(a, s);
}

// Arguments that both entry points check and fill alike.
static medusa_status attend(AttnArgs& a, int n_layers, int T, int B, int Hq, int Hkv, int d, int n_pages, int page_size,
                            int max_pages, int64_t ldq, float scale, medusa_dtype dt, void* ws, size_t ws_bytes,
                            cudaStream_t s) {
  const Division v = divide(T, B, Hq, Hkv, d, page_size, dt);
  a.cache.n_pages = n_pages;
  a.cache.page_size = page_size;
  a.cache.max_pages = max_pages;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.G = Hq / Hkv;
  a.ldq = ldq;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (!ws || !aligned16(ws) || ws_bytes < ws_bytes_of(v, d)) return MEDUSA_ERR_WORKSPACE;
  // The entry points have compared out and lse with the big inputs.
  const size_t es = dtype_bytes(dt), tokens = (size_t)n_layers * T, pool = (size_t)n_layers * n_pages * page_size * Hkv * d * es;
  const size_t tree = a.w.N ? tokens * Hkv * d * es : 0, nb = (size_t)B * 4;
  const Region small[] = {{a.cache.page_table, nb * max_pages}, {a.w.q_start, nb + 4}, {a.w.prefix_len, nb}, {a.mask, (size_t)a.w.N * a.W * 4}};
  const Region out{a.out, tokens * Hq * d * es}, lse{a.lse, tokens * Hq * 4}, scratch{ws, ws_bytes_of(v, d)};
  for (const Region& r : small)
    if (overlaps_any(r, {out, lse, scratch})) return MEDUSA_ERR_ALIAS;
  if (overlaps_any(scratch, {out, lse, {a.q, ((tokens - 1) * (size_t)ldq + (size_t)Hq * d) * es}, {a.k_pages, pool}, {a.v_pages, pool}, {a.kt, tree}, {a.vt, tree}}))
    return MEDUSA_ERR_ALIAS;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)v.ctas * 2 * v.R * d);
  a.shared = reinterpret_cast<Shared*>(a.part_ml + (size_t)v.ctas * 2 * v.R);
  a.R = v.R;
  a.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && d % 16 == 0;
  a.tile_rows = v.tile_rows;
  a.tile_tok = v.tile_tok;
  a.sub = v.sub;
  a.nsub = v.nsub;
  a.w.nl = n_layers;
  a.w.nh = Hkv * v.nsub;
  a.w.cap = max_pages * page_size;
  a.w.ctok = v.ctok;
  a.w.KT = v.KT;
  a.w.ctok_log2 = log2_of(v.ctok);
  a.w.KT_log2 = log2_of(v.KT);
  // No more CTAs than there can be tiles (but two, for the reciprocal): idle ones delay a small call
  // (3 heads x 10 nodes of 4 sequences 12.7 us, on all SMs 14.1; fp32, 21 short sequences 9.0 and 11.7).
  const long long blocks = a.w.N ? (long long)B * ((a.w.N + v.ctok - 1) / v.ctok) : (long long)B + T / v.ctok;
  const long long tiles = (a.w.cap + v.KT - 1) / v.KT + (a.w.N + v.KT - 1) / v.KT;
  const double most = (double)a.w.nl * a.w.nh * blocks * tiles;
  a.w.ctas = most >= v.ctas ? v.ctas : most <= 2 ? 2 : (int)most;
  a.w.ctas_inv = ~0ull / a.w.ctas + 1;
  a.w.B = B;
  a.w.T = T;
  const medusa_status st = v.tc ? paged_attention_tc(a, s) : dt == MEDUSA_BF16 ? simt_launch<uint16_t>(a, s) : simt_launch<float>(a, s);
  if (st != MEDUSA_OK) return st;
  // Sequences that can hold one tile of keys at most leave no item to share (2 to 3 us of a call's 10 to 13).
  if (!a.w.N && a.w.cap <= v.KT) return launch_status();
  if (v.R > 64) launch_pdl(paged_attn_merge_wide_kernel, dim3(a.w.ctas - 1, v.R / 32), dim3(256), 0, s, a);
  else if (dt == MEDUSA_BF16) launch_pdl(paged_attn_merge_kernel<uint16_t>, dim3(a.w.ctas - 1, v.R / 8), dim3(256), 0, s, a);
  else launch_pdl(paged_attn_merge_kernel<float>, dim3(a.w.ctas - 1, v.R / 8), dim3(256), 0, s, a);
  return launch_status();
}

static bool sizes_ok(int n_layers, int T, int B, int Hq, int Hkv, int d, int n_pages, int page_size, int max_pages,
                     float scale, int dt) {
  if (n_layers < 1 || T < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq > 65535) return false;
  if (d < 4 || d % 4 || d > MEDUSA_MAX_HEAD_DIM || !(scale > 0.f) || !(scale < INFINITY) || !dtype_ok(dt)) return false;
  if ((long long)n_layers * T > 0x7fffffffll || (long long)n_layers * Hq > 0x7fffffffll) return false;
  return cache_sizes_ok(n_layers, B, n_pages, page_size, max_pages);
}

}  // namespace paged
}  // namespace medusa

using namespace medusa;
using namespace medusa::paged;

extern "C" size_t medusa_paged_attention_workspace_size(int n_layers, int T, int B, int Hq, int Hkv, int d, int page_size,
                                                        medusa_dtype dt) {
  if (n_layers < 1 || T < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || d < 4 || d > MEDUSA_MAX_HEAD_DIM || page_size < 1 || !dtype_ok(dt))
    return 0;
  return ws_bytes_of(divide(T, B, Hq, Hkv, d, page_size, dt), d);
}

static medusa_status chunk_attention(const void* q, int64_t ldq, const void* k_pages, const void* v_pages,
                                     const int32_t* page_table, const int32_t* q_start,
                                     const int32_t* prefix_len, int n_layers, int T, int B, int Hq, int Hkv,
                                     int d, int n_pages, int page_size, int max_pages, float scale,
                                     medusa_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                     int32_t* d_status, medusa_stream_t stream, int withhold) {
  if (!q || !k_pages || !v_pages || !page_table || !q_start || !prefix_len || !out) return MEDUSA_ERR_INVALID_ARG;
  if (!sizes_ok(n_layers, T, B, Hq, Hkv, d, n_pages, page_size, max_pages, scale, dt)) return MEDUSA_ERR_INVALID_ARG;
  if (ldq < (int64_t)Hq * d || ldq % 4 || !aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return MEDUSA_ERR_INVALID_ARG;
  const uintptr_t words = (uintptr_t)page_table | (uintptr_t)q_start | (uintptr_t)prefix_len | (uintptr_t)lse | (uintptr_t)d_status;
  if (words & 3) return MEDUSA_ERR_INVALID_ARG;
  if (tc_shape(Hq / Hkv, d, page_size, dt) && ldq % 8) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt), tokens = (size_t)n_layers * T;
  const size_t nq = ((tokens - 1) * (size_t)ldq + (size_t)Hq * d) * es, no = tokens * Hq * d * es;
  const size_t np = (size_t)n_layers * n_pages * page_size * Hkv * d * es, nl = tokens * Hq * 4;
  if (overlaps(out, no, q, nq) || overlaps(out, no, k_pages, np) || overlaps(out, no, v_pages, np)) return MEDUSA_ERR_ALIAS;
  if (lse && (overlaps(lse, nl, out, no) || overlaps(lse, nl, q, nq) || overlaps(lse, nl, k_pages, np) || overlaps(lse, nl, v_pages, np)))
    return MEDUSA_ERR_ALIAS;
  AttnArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.out = out;
  a.lse = lse;
  a.d_status = d_status;
  a.cache.page_table = page_table;
  a.w.q_start = q_start;
  a.w.prefix_len = prefix_len;
  a.withhold = withhold;
  return attend(a, n_layers, T, B, Hq, Hkv, d, n_pages, page_size, max_pages, ldq, scale, dt, ws, ws_bytes,
                reinterpret_cast<cudaStream_t>(stream));
}

extern "C" medusa_status medusa_paged_attention(const void* q, int64_t ldq, const void* k_pages, const void* v_pages,
                                                const int32_t* page_table, const int32_t* q_start,
                                                const int32_t* prefix_len, int n_layers, int T, int B, int Hq, int Hkv,
                                                int d, int n_pages, int page_size, int max_pages, float scale,
                                                medusa_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                                int32_t* d_status, medusa_stream_t stream) {
  return chunk_attention(q, ldq, k_pages, v_pages, page_table, q_start, prefix_len, n_layers, T, B, Hq, Hkv, d, n_pages, page_size, max_pages, scale,
                         dt, out, lse, ws, ws_bytes, d_status, stream, 0);
}

extern "C" medusa_status medusa_paged_attention_test_stall(const void* q, int64_t ldq, const void* k_pages, const void* v_pages,
                                                           const int32_t* page_table, const int32_t* q_start,
                                                           const int32_t* prefix_len, int n_layers, int T, int B, int Hq, int Hkv,
                                                           int d, int n_pages, int page_size, int max_pages, float scale,
                                                           medusa_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                                           int32_t* d_status, medusa_stream_t stream) {
  if (Hkv < 1 || page_size < 1 || !tc_shape(Hq / Hkv, d, page_size, dt)) return MEDUSA_ERR_INVALID_ARG;
  return chunk_attention(q, ldq, k_pages, v_pages, page_table, q_start, prefix_len, n_layers, T, B, Hq, Hkv, d, n_pages, page_size, max_pages, scale,
                         dt, out, lse, ws, ws_bytes, d_status, stream, 1);
}

extern "C" medusa_status medusa_paged_tree_attention(const void* q, const void* k_pages, const void* v_pages,
                                                     const int32_t* page_table, const void* kt, const void* vt,
                                                     const uint32_t* mask, const int32_t* prefix_len, int n_layers, int B,
                                                     int N, int Hq, int Hkv, int d, int n_pages, int page_size,
                                                     int max_pages, float scale, medusa_dtype dt, void* out, float* lse,
                                                     void* ws, size_t ws_bytes, int32_t* d_status, medusa_stream_t stream) {
  if (!q || !k_pages || !v_pages || !page_table || !kt || !vt || !mask || !prefix_len || !out) return MEDUSA_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || N > MEDUSA_MAX_NODES || (long long)B * N > 0x7fffffffll) return MEDUSA_ERR_INVALID_ARG;
  if (!sizes_ok(n_layers, B * N, B, Hq, Hkv, d, n_pages, page_size, max_pages, scale, dt)) return MEDUSA_ERR_INVALID_ARG;
  const void* rows[] = {q, k_pages, v_pages, kt, vt, out};
  for (const void* p : rows)
    if (!aligned16(p)) return MEDUSA_ERR_INVALID_ARG;
  const uintptr_t words = (uintptr_t)page_table | (uintptr_t)mask | (uintptr_t)prefix_len | (uintptr_t)lse | (uintptr_t)d_status;
  if (words & 3) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt), tokens = (size_t)n_layers * B * N;
  const size_t no = tokens * Hq * d * es, nt = tokens * Hkv * d * es, nl = tokens * Hq * 4;
  const size_t np = (size_t)n_layers * n_pages * page_size * Hkv * d * es;
  const void* in[] = {q, k_pages, v_pages, kt, vt};
  const size_t size[] = {no, np, np, nt, nt};
  for (int i = 0; i < 5; ++i)
    if (overlaps(out, no, in[i], size[i]) || (lse && overlaps(lse, nl, in[i], size[i]))) return MEDUSA_ERR_ALIAS;
  if (lse && overlaps(lse, nl, out, no)) return MEDUSA_ERR_ALIAS;
  AttnArgs a{};
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.kt = kt;
  a.vt = vt;
  a.mask = mask;
  a.W = (N + 31) / 32;
  a.out = out;
  a.lse = lse;
  a.d_status = d_status;
  a.cache.page_table = page_table;
  a.w.prefix_len = prefix_len;
  a.w.N = N;
  return attend(a, n_layers, B * N, B, Hq, Hkv, d, n_pages, page_size, max_pages, (int64_t)Hq * d, scale, dt, ws, ws_bytes,
                reinterpret_cast<cudaStream_t>(stream));
}
