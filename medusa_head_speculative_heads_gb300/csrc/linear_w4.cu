// medusa_linear_w4: y = x W^T with W in 4 bits, and medusa_w4_quantize, which makes such weights.
//
// A weight is bf16(scale (q - zero)): 128 + q and 128 + zero, as bf16, are the bits 0x4300 | q and
// 0x4300 | zero, their difference is exact, and the bf16 multiplication by the scale rounds once.  The
// order of a word's elements puts two neighbours 16 bits apart, so that a shift and one three-operand
// logic operation unpack a pair.
#include <math.h>

#include "host_util.h"
#include "linear_w4.h"
#include "medusa_test_hooks.h"

namespace medusa {
namespace w4 {

// 16 bytes of weights, which are read once.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ few tokens
//
// A CTA has 16 rows of W and 8 NT tokens; its warps take blocks of 128 columns in turn and their sums
// meet in shared memory.  Of a block, lane 4 g + t holds 32 columns, from 32 t on, of the rows g and g + 8 and of
// the tokens g, g + 8, ...: two 16-byte loads of weights, whose group is one whatever its size.  The
// products' columns may come in any order so long as both operands' do: word j of a lane's four gives
// the operands of two 16-column products, of which each lane's elements are neighbours in memory.
constexpr int kWarps = 8;

template <int NT>
__global__ void __launch_bounds__(kWarps * 32) few_kernel(const __grid_constant__ Args a) {
  __shared__ float part[kWarps][NT][16][9];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mt = blockIdx.x;
  const int n_lo = min(mt * 16 + g, a.Nout - 1), n_hi = min(mt * 16 + g + 8, a.Nout - 1);  // rows past the last: computed, not stored
  const uint8_t *w_lo = reinterpret_cast<const uint8_t*>(a.q) + (size_t)n_lo * (a.K / 2), *w_hi = reinterpret_cast<const uint8_t*>(a.q) + (size_t)n_hi * (a.K / 2);
  float acc[NT][4] = {};
  for (int k0 = warp * 128; k0 < a.K; k0 += kWarps * 128) {
    const int k = k0 + 32 * t;
    uint32_t lo[4] = {}, hi[4] = {};
    Group g_lo{0, 0}, g_hi{0, 0};
    uint4 xv[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[j][i] = make_uint4(0, 0, 0, 0);
    if (k < a.K) {
      *reinterpret_cast<uint4*>(lo) = load_once(w_lo + k / 2);
      *reinterpret_cast<uint4*>(hi) = load_once(w_hi + k / 2);
      g_lo = group_at(a, k >> a.glog, n_lo);
      g_hi = group_at(a, k >> a.glog, n_hi);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (8 * j + g < a.T) {
          const uint4* p = reinterpret_cast<const uint4*>(a.x + (8 * j + g) * a.ldx + k);
#pragma unroll
          for (int i = 0; i < 4; ++i) xv[j][i] = p[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p[4], r[4];
      unpack(lo[i], g_lo, p);
      unpack(hi[i], g_hi, r);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma16816(acc[j], p[0], r[0], p[1], r[1], xv[j][i].x, xv[j][i].y);
        mma16816(acc[j], p[2], r[2], p[3], r[3], xv[j][i].z, xv[j][i].w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    part[warp][j][g][2 * t] = acc[j][0];
    part[warp][j][g][2 * t + 1] = acc[j][1];
    part[warp][j][g + 8][2 * t] = acc[j][2];
    part[warp][j][g + 8][2 * t + 1] = acc[j][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 128; i += kWarps * 32) {
    const int m = i & 15, tok = i >> 4;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][tok >> 3][m][tok & 7];
    if (tok < a.T && mt * 16 + m < a.Nout) store_y(a, tok, mt * 16 + m, v);
  }
}

// ------------------------------------------------------------------ making the weights

// A warp a group; each lane has group / 32 neighbouring elements, and words are put together
// among 8 / (group / 32) lanes.
__global__ void __launch_bounds__(256)
quantize_kernel(const void* w, int bf16, int Nout, int K, int glog, int symmetric, uint32_t* q, uint16_t* scales, uint8_t* zeros) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, G = 1 << glog, ng = K >> glog, per = G >> 5;
  const long long groups = (long long)Nout * ng;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < groups; i += (long long)gridDim.x * 8) {
    const int n = (int)(i / ng), g = (int)(i - (long long)n * ng);
    const size_t at = (size_t)n * K + ((size_t)g << glog) + lane * per;
    float v[4], lo = 0.f, hi = 0.f;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = j < per ? (bf16 ? load_elem(static_cast<const uint16_t*>(w), at + j) : load_elem(static_cast<const float*>(w), at + j)) : 0.f;
      odd |= !isfinite(v[j]);
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
    }
    hi = warp_max(hi);
    lo = -warp_max(-lo);
    const float step = symmetric ? fmaxf(hi, -lo) / 7.f : (hi - lo) / 15.f;
    uint32_t bits = f32_to_bf16_bits(step);
    float s = bf16_bits_to_f32(bits);
    const bool none = s == 0.f;
    if (none) bits = 0x3f80u, s = 1.f;
    if (__any_sync(0xffffffffu, odd) || !isfinite(s)) bits = 0x7fc0u;
    float z = symmetric ? 8.f : fminf(fmaxf(rintf(-lo / s), 0.f), 15.f);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= per) break;
      const float r = none ? z : rintf(v[j] / s) + z;
      const uint32_t e = (uint32_t)fminf(fmaxf(r, 0.f), 15.f);  // NaN: 0
      const int k = (lane * per + j) & 7;                       // place within the word
      word |= e << (4 * (k >> 1) + 16 * (k & 1));
    }
    for (int o = 1; o < 8 / per; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if ((lane * per & 7) == 0) q[((size_t)n * K + ((size_t)g << glog) + lane * per) >> 3] = word;
    if (lane == 0) {
      scales[(size_t)g * Nout + n] = (uint16_t)bits;
      if (zeros) zeros[(size_t)g * Nout + n] = (uint8_t)z;
    }
  }
}

static int group_log2(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

}  // namespace w4
}  // namespace medusa

using namespace medusa;
using namespace medusa::w4;

static bool sizes_ok(int K, int Nout, int group) {
  return group_log2(group) >= 0 && K >= group && K % group == 0 && K < 0x7fffffff - 65536 && Nout >= 1 && Nout < 0x7fffffff - 65536;
}

extern "C" medusa_status medusa_w4_quantize(const void* w, int Nout, int K, int group, int symmetric, medusa_dtype dt, uint32_t* qweight,
                                            void* scales, uint8_t* zeros, medusa_stream_t stream) {
  if (!w || !qweight || !scales || !dtype_ok(dt) || !sizes_ok(K, Nout, group) || (!symmetric && !zeros)) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dt), nw = (size_t)Nout * K * es, nq = (size_t)Nout * K / 2, ns = (size_t)Nout * (K / group);
  if (((uintptr_t)w & (es - 1)) || ((uintptr_t)qweight & 3) || ((uintptr_t)scales & 1)) return MEDUSA_ERR_INVALID_ARG;
  if (overlaps_any({w, nw}, {{qweight, nq}, {scales, 2 * ns}, {zeros, ns}}) || overlaps_any({qweight, nq}, {{scales, 2 * ns}, {zeros, ns}}) ||
      overlaps_any({scales, 2 * ns}, {{zeros, ns}}))
    return MEDUSA_ERR_ALIAS;
  long long blocks = ((long long)ns + 7) / 8, cap = (long long)device_sm_count() * 32;
  launch_pdl(quantize_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), w,
             (int)(dt == MEDUSA_BF16), Nout, K, group_log2(group), symmetric, qweight, static_cast<uint16_t*>(scales), zeros);
  return launch_status();
}

// Up to 16 tokens the warps' own product instructions, fed from registers; more on tensor memory.
static bool on_tc(int T) { return T > 16; }

extern "C" size_t medusa_linear_w4_workspace_size(int T, int K, int Nout, int group) {
  return 0;
}

static medusa_status linear_call(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales, const uint8_t* zeros, int T, int K,
                                 int Nout, int group, void* y, medusa_dtype y_dt, void* ws, size_t ws_bytes, int32_t* d_status,
                                 medusa_stream_t stream, int withhold) {
  if (T < 0 || !sizes_ok(K, Nout, group) || !dtype_ok(y_dt)) return MEDUSA_ERR_INVALID_ARG;
  if (T == 0) return MEDUSA_OK;
  if (!x || !qweight || !scales || !y || ldx < K || ldx % 8 || ldx >= (1ll << 38) || T >= 0x7fffffff - 65536) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(y_dt);
  if (!aligned16(x) || !aligned16(qweight) || ((uintptr_t)scales & 1) || ((uintptr_t)y & (es - 1)) || ((uintptr_t)d_status & 3))
    return MEDUSA_ERR_INVALID_ARG;
  const size_t need = medusa_linear_w4_workspace_size(T, K, Nout, group);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return MEDUSA_ERR_WORKSPACE;
  const size_t ny = (size_t)T * Nout * es, ns = (size_t)Nout * (K / group), nx = ((size_t)(T - 1) * ldx + K) * 2;
  const Region nothing{nullptr, 0}, part = need ? Region{ws, need} : nothing;
  if (overlaps_any({y, ny}, {{x, nx}, {qweight, (size_t)Nout * K / 2}, {scales, 2 * ns}, {zeros, ns}, {d_status, 4}, part}) ||
      overlaps_any(part, {{x, nx}, {qweight, (size_t)Nout * K / 2}, {scales, 2 * ns}, {zeros, ns}, {d_status, 4}}))
    return MEDUSA_ERR_ALIAS;
  Args a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.q = qweight;
  a.scales = static_cast<const uint16_t*>(scales);
  a.zeros = zeros;
  a.T = T;
  a.K = K;
  a.Nout = Nout;
  a.glog = group_log2(group);
  a.y = y;
  a.y32 = y_dt == MEDUSA_F32;
  a.d_status = d_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (on_tc(T)) return tc_launch(a, withhold, s);
  if (withhold) return MEDUSA_ERR_INVALID_ARG;
  const int nt = T <= 8 ? 1 : 2;
  const dim3 gd((Nout + 15) / 16), bd(kWarps * 32);
  if (nt == 1) launch_pdl(few_kernel<1>, gd, bd, 0, s, a);
  else launch_pdl(few_kernel<2>, gd, bd, 0, s, a);
  return launch_status();
}

extern "C" medusa_status medusa_linear_w4(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales, const uint8_t* zeros, int T,
                                          int K, int Nout, int group, void* y, medusa_dtype y_dt, void* ws, size_t ws_bytes, int32_t* d_status,
                                          medusa_stream_t stream) {
  return linear_call(x, ldx, qweight, scales, zeros, T, K, Nout, group, y, y_dt, ws, ws_bytes, d_status, stream, 0);
}

extern "C" medusa_status medusa_linear_w4_test_stall(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales,
                                                     const uint8_t* zeros, int T, int K, int Nout, int group, void* y, medusa_dtype y_dt,
                                                     void* ws, size_t ws_bytes, int32_t* d_status, medusa_stream_t stream) {
  return linear_call(x, ldx, qweight, scales, zeros, T, K, Nout, group, y, y_dt, ws, ws_bytes, d_status, stream, 1);
}
