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
// A CTA has 16 MT rows of W and 8 NT tokens; its warps take blocks of 128 columns in turn and their sums
// meet in shared memory.  Of a block, lane 4 g + t holds 32 columns, from 32 t on, of the rows g + 8 j and of
// the tokens g + 8 j: 16-byte loads of weights, whose group is one whatever its size.  The product
// instructions' columns may come in any order so long as both operands' do: word j of a lane's four gives the
// operands of two 16-column products, of which each lane's elements are neighbours in memory.
//
// What bounds it: the instructions that unpack (15 a word, of which 7 at half rate), and memory next to them (7 tokens, 13825
// features of 5120 columns: 13.0 us, 3.2 TB/s; one token, 4096 x 4096: 4.1 to 4.9 us, of which a launch is 1.2,
// whether the weights are in L2 or not).  Rows that lie outside W are not asked for (the last CTA's rows
// are moved up, what another CTA has too is not stored), tokens behind the last one repeat it, and the next block's
// weights are on their way while one is unpacked.
template <int NT, int MT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) few_kernel(const __grid_constant__ Args a) {
  constexpr int R = 2 * MT, ROWS = 16 * MT;  // rows of a lane, of the CTA
  __shared__ float part[WARPS][NT][ROWS][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int base = min((int)blockIdx.x * ROWS, a.Nout - ROWS);
  const size_t pitch = (size_t)a.K / 2;
  int k0 = warp * 128;
  const uint8_t* w[R];
#pragma unroll
  for (int j = 0; j < R; ++j) w[j] = reinterpret_cast<const uint8_t*>(a.q) + (base + g + 8 * j) * pitch + (k0 + 32 * t) / 2;
  pdl_wait();
  pdl_trigger();
  size_t at = (size_t)((k0 + 32 * t) >> a.glog) * a.Nout + base + g;
  const size_t at_step = (size_t)((WARPS * 128) >> a.glog) * a.Nout;
  const uint16_t* x[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) x[j] = a.x + (long long)min(g + 8 * j, a.T - 1) * a.ldx + k0 + 32 * t;
  float acc[MT][NT][4] = {};
  uint4 v[R];
  auto load = [&](bool here) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (here) v[j] = load_once(w[j]);
      w[j] += WARPS * 64;
    }
  };
  auto block = [&](bool here, bool more) {
    uint32_t s[R], z[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      s[j] = here ? a.scales[at + 8 * j] : 0;
      z[j] = here && a.zeros ? a.zeros[at + 8 * j] : 8;
    }
    uint4 xv[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xv[j][i] = make_uint4(0, 0, 0, 0);
        if (here) xv[j][i] = reinterpret_cast<const uint4*>(x[j])[i];
      }
    uint4 now[R];
#pragma unroll
    for (int j = 0; j < R; ++j) now[j] = v[j];
    if (more) load(true);
    at += at_step;
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] += WARPS * 128;
    Group gr[R];
#pragma unroll
    for (int j = 0; j < R; ++j) gr[j] = group_of(s[j], z[j]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t lo[4] = {now[2 * m].x, now[2 * m].y, now[2 * m].z, now[2 * m].w},
                     hi[4] = {now[2 * m + 1].x, now[2 * m + 1].y, now[2 * m + 1].z, now[2 * m + 1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t p[4], r[4];
        unpack(lo[i], gr[2 * m], p);
        unpack(hi[i], gr[2 * m + 1], r);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816(acc[m][j], p[0], r[0], p[1], r[1], xv[j][i].x, xv[j][i].y);
          mma16816(acc[m][j], p[2], r[2], p[3], r[3], xv[j][i].z, xv[j][i].w);
        }
      }
    }
  };
  if (k0 + 128 <= a.K) load(true);
#pragma unroll 1
  for (; k0 + 128 <= a.K; k0 += WARPS * 128) block(true, k0 + (WARPS + 1) * 128 <= a.K);
  if (k0 < a.K) {  // the rest of K is this warp's
    const bool here = k0 + 32 * t < a.K;
    load(here);
    block(here, false);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      part[warp][j][16 * m + g][2 * t] = acc[m][j][0];
      part[warp][j][16 * m + g][2 * t + 1] = acc[m][j][1];
      part[warp][j][16 * m + g + 8][2 * t] = acc[m][j][2];
      part[warp][j][16 * m + g + 8][2 * t + 1] = acc[m][j][3];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * ROWS; i += WARPS * 32) {
    const int m = i % ROWS, tok = i / ROWS, n = base + m;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) y += part[k][tok >> 3][m][tok & 7];
    if (tok < a.T && n >= (int)blockIdx.x * ROWS) store_y(a, tok, n, y);
  }
}

template <int NT, int MT, int WARPS>
static void few(const Args& a, cudaStream_t s) {
  launch_pdl(few_kernel<NT, MT, WARPS>, dim3((a.Nout + 16 * MT - 1) / (16 * MT)), dim3(WARPS * 32), 0, s, a);
}

// ------------------------------------------------------------------ making the weights

// A warp a group; each lane has group / 32 neighbouring elements, and words are put together
// among 8 / (group / 32) lanes.  Set-up work, bound by the instructions of a group, of which a lane has 1 to 4 elements:
// 4096 x 4096 bf16 weights 40 us in groups of 128, 122 in groups of 32, where the bytes would take 6.
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
  return group_log2(group) >= 0 && K >= group && K % group == 0 && K < 0x7fffffff - 65535 && Nout >= 1 && Nout < 0x7fffffff - 65535;
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

// More than 64 tokens are the work of linear_w4_tc.cu, unless the layer is so small that few blocks make a CTA of
// linear_w4_stream.cu, whose evenly divided work then ends sooner (2048 features of 2048 columns, 128 tokens, 4 blocks: 6.9 and
// 10.2 us; 4096 x 4096, 128 and 256 tokens, 16 and 32 blocks: 9.9 and 11.6, 12.2 and 15.1; 384 tokens, 48 blocks: 17.9 and
// 17.4; 4096 features of 11008 columns, 65 tokens, 44 blocks: 16.6 and 15.4).
constexpr int kSmall = 32;
// Up to 64 tokens are the work of linear_w4_stream.cu, and of few tokens the warps' own
// product instructions, fed from registers, where their CTAs are all there at once or the layer is small: the others
// need some 2 us more to begin and to add up, and unpack faster.  Times for K = 4096, registers and tensor memory:
//   one token    x  4096 features   5.0 and  7.1 us     9 tokens x 1024   4.5 and 5.4 us
//                x 13825           10.1     12.2                 x 4096   6.5     7.1
//                x 16384           14.2     12.1        16       x 4096   7.6     7.2
//   8 tokens     x 28672           19.7     17.0        16       x 8192  10.9     9.1
// Two CTAs of 16 rows and 16 warps are on an SM at once, three of 32 rows and 8 warps.  Those of 32 rows share the
// tokens' loads among more weights, and are better from the second filling with the others on (K = 4096, 11008 features:
// 9.8 us, with 16 rows 10.8; 8192 features: 9.6 and 8.4).
static bool wide(int Nout) { return Nout > 64 * device_sm_count(); }
static bool from_registers(int T, int K, int Nout) {
  const long long n = (long long)K * Nout;
  if (T > 16 || Nout < 32) return false;
  if (T > 8) return n < 1 << 24 && !wide(Nout);
  return n < 1 << 25 || Nout <= 32 * device_sm_count() || (wide(Nout) && Nout <= 96 * device_sm_count());
}

enum Kernel { kRegisters, kStream, kTiles };
static Kernel kernel_of(int T, int K, int Nout) {
  if (T > 64 && stream_blocks(T, K, Nout) > kSmall) return kTiles;
  return from_registers(T, K, Nout) ? kRegisters : kStream;
}

static medusa_status linear_call(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales, const uint8_t* zeros, int T, int K,
                                 int Nout, int group, void* y, medusa_dtype y_dt, int32_t* d_status, medusa_stream_t stream, int withhold) {
  if (T < 0 || !sizes_ok(K, Nout, group) || !dtype_ok(y_dt)) return MEDUSA_ERR_INVALID_ARG;
  if (T == 0) return MEDUSA_OK;
  if (!x || !qweight || !scales || !y || ldx < K || ldx % 8 || ldx >= (1ll << 38) || T >= 0x7fffffff - 65535) return MEDUSA_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(y_dt);
  if (!aligned16(x) || !aligned16(qweight) || ((uintptr_t)scales & 1) || ((uintptr_t)y & (es - 1)) || ((uintptr_t)d_status & 3))
    return MEDUSA_ERR_INVALID_ARG;
  const size_t ny = (size_t)T * Nout * es, ns = (size_t)Nout * (K / group), nx = ((size_t)(T - 1) * ldx + K) * 2;
  if (overlaps_any({y, ny}, {{x, nx}, {qweight, (size_t)Nout * K / 2}, {scales, 2 * ns}, {zeros, ns}, {d_status, 4}}))
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
  const Kernel kernel = kernel_of(T, K, Nout);
  if (kernel == kTiles) return tc_launch(a, withhold, s);
  if (kernel == kStream) return stream_launch(a, withhold, s);
  if (withhold) return MEDUSA_ERR_INVALID_ARG;
  if (T > 8) few<2, 1, 16>(a, s);
  else if (wide(Nout)) few<1, 2, 8>(a, s);
  else few<1, 1, 16>(a, s);
  return launch_status();
}

extern "C" medusa_status medusa_linear_w4(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales, const uint8_t* zeros, int T,
                                          int K, int Nout, int group, void* y, medusa_dtype y_dt, int32_t* d_status, medusa_stream_t stream) {
  return linear_call(x, ldx, qweight, scales, zeros, T, K, Nout, group, y, y_dt, d_status, stream, 0);
}

extern "C" medusa_status medusa_linear_w4_test_stall(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales,
                                                     const uint8_t* zeros, int T, int K, int Nout, int group, void* y, medusa_dtype y_dt,
                                                     int32_t* d_status, medusa_stream_t stream) {
  return linear_call(x, ldx, qweight, scales, zeros, T, K, Nout, group, y, y_dt, d_status, stream, 1);
}

extern "C" medusa_status medusa_linear_w4_test_division(int T, int K, int Nout, int32_t* division) {
  if (T < 1 || T >= 0x7fffffff - 65535 || !sizes_ok(K, Nout, 32) || !division) return MEDUSA_ERR_INVALID_ARG;
  const Kernel kernel = kernel_of(T, K, Nout);
  const Division d = kernel == kTiles ? tc_division(T, K, Nout) : kernel == kStream ? stream_division(T, K, Nout) : Division{};
  const int32_t all[6] = {kernel, d.share, d.tokens, d.features, d.tiles, d.ctas};
  for (int i = 0; i < 6; ++i) division[i] = all[i];
  return MEDUSA_OK;
}
