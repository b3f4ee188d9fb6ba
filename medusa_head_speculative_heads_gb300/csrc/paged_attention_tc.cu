// Paged attention on tcgen05 tensor cores: bf16, head dims up to 128 (computed
// as 64 or 128 columns, the rest zeros), fp32 scores and sums in tensor memory.
//
// The mathematics is that of paged_attention.cu: one pass over the key tiles
// with a running maximum and sum per row.  An item is a block of up to 2 x 128
// query rows (token, q head of the group) of one sequence and kv head; a key
// tile is 128 rows of the cache (or of the tree).
//
// Two streams run side by side in a CTA, each with its own scores S and sums O
// in tensor memory (4 x 128 columns, all of it), its own MMA-issuing warp and
// its own four softmax warps (a thread holds one query row's 128 scores), so
// that one's softmax runs under the other's products:
//  - a block of more than 128 rows: stream s has rows 128 s .. 128 s + 127, and
//    both use every K and V tile, read from global memory once;
//  - a block of at most 128 rows (decoding, small trees): both streams have the
//    same rows, stream s the key tiles t0 + s, t0 + s + 2, ...; their two
//    results are added as two parts of a row are.
// Within a stream S = Q K^T, softmax, O += P V follow one another; P (bf16, in two
// halves, the first multiplied while the second is formed) overwrites S, and the
// next tile's S is issued by the same thread behind the P V that reads P, which
// orders the two.  A completed S therefore also says that the P V before it is
// done, and O may be rescaled; that happens only when a row's maximum has grown by
// more than 2^8 (the stale maximum is exact arithmetic: the same power of two scales
// P and the sum).  P is rounded to bf16, half a step of 2^-8 of each probability, for
// the tensor cores; the sum is that of the unrounded ones, in fp32.
//
// Warp 0 walks through the CTA's items, describes each one to the others in
// shared memory, and brings Q and the K tiles by TMA; warp 3 brings the V
// tiles, each into a ring of its own (a warp alone took longer to issue a tile's
// copies from 16-row pages than memory took to bring them).  A tile is copied
// in boxes of gcd(page_size, 128) rows, each lane looking one page up a tile
// ahead; a page that does not exist is read as rows behind the pool, which
// arrive as zeros.  Rows behind the last one are masked in S; the rows of V up
// to the next multiple of 16 are zeroed before P V reads them (0 times what a
// stale row holds could be NaN), and the products stop there.
//
// What bounds it: decoding, memory (64 sequences of up to 8192 rows 188 to 194 us, 6.3 to 6.5
// TB/s).  A long prompt (8192 tokens over 8192 rows, 32 + 8 heads of 128: 1053 to 1105 us captured
// one after the other, 1490 to 1565 TFLOP/s; 1130 to 1142, 1445 to 1460, called one by one on
// other data each time), a stream's chain of softmax (1160 clocks a tile), hand-over of P (250),
// products (768 behind the second half) and hand-over of S (330), half of which the other
// stream's products fill.  Prompts of a few thousand tokens, also the hand-over between blocks
// (some 6000 clocks: the last products, the output of 256 rows, Q, the first scores).
//
// Every wait is bounded: a timeout sets MEDUSA_DEV_TIMEOUT, all roles stop,
// copies and MMAs in flight are waited for and tensor memory is freed.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "host_util.h"
#include "paged_attn.cuh"
#include "sm100.cuh"

namespace medusa {
namespace paged {
using namespace sm100;

namespace tc {

constexpr int kThreads = 384;          // items and K, two MMA issuers, V; 2 x 4 softmax warps
constexpr int kKeys = 128;             // keys of a tile
constexpr uint32_t kHalf = 16384;      // 128 rows x 128 bytes (64 columns)
constexpr int kTries = 1 << 20;        // of a wait that sleeps: 1.3 us each (measured), 1.4 s in all
constexpr int kPolls = 1 << 23;        // of one that does not: 110 ns (measured), 0.9 s in all
constexpr uint64_t kDrainNs = 100000000ull;
constexpr uint32_t kTmemCols = 512;    // S0, S1, O0, O1
constexpr int kMaxSlots = 12;
constexpr int kUnits = 4;              // described units in flight
constexpr int kUnitReaders = 11;       // warps that read a description

struct Bars {
  // A wait tells phases apart by their parity, so a waiter may skip none: rows for stream 0 or 1 alone
  // are announced in full[0] or full[1], rows for both in full[2], which both streams watch whether
  // they need them or not.  Every slot and Q buffer is released twice.
  uint64_t full[3][kMaxSlots], empty[kMaxSlots];  // K's slots, then V's
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2];    // P's first 64 columns, and the others
  uint64_t turn[2];                            // a stream may issue its products of the next tile
  uint64_t o_full[2], o_free[2], ml_full, drain[2];  // o_full, o_free: one phase a unit
  uint64_t u_full[kUnits], u_free[kUnits];
};

// The part of an item that a CTA works on, and how its two streams share it.
struct Unit {
  int t0, t1;      // key tiles; t1 <= 0: no more units
  int tiles;       // of the whole item
  int two;         // two row tiles; else one, its key tiles taken in turn
  int pre;         // tiles of cache rows (the rest are tree tiles)
  int rows_end;    // cache rows the block may see
  int end0;        // tiles [t0, end0) are stream 0's when there are two row tiles
  int b, kvh;
  int L;           // rows before the sequence's tokens
  int tok0, ntok;  // the block's tokens within the sequence
  int row0;        // its first token among all layers' tokens
  int tree0;       // the sequence's first token there
  int pool0;       // the layer's first pool row
};

// Behind the ring.  All shared memory is dynamic, so that it starts on the 1024
// bytes the swizzled tiles need (checked).
struct Tail {
  Bars bars;
  Unit units[kUnits];
  union {
    long long plan[70];  // set-up only
    float2 ml[128];      // stream 1's row maxima and sums, for stream 0 to add
  };
  uint32_t tmem;
  volatile int abort;
  // What the loading warps (K, V) leave: loads into each Q buffer; the slots whose barriers full[k] they have
  // used, and an odd number of times.
  int q_loads[2];
  uint32_t loads[2][3], odd[2][3];
  __device__ void note_loads(int kv, const uint32_t* used, const uint32_t* flips) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      loads[kv][k] = used[k];
      odd[kv][k] = flips[k];
    }
  }
};

// DH: columns computed, 64 or 128.  NARROW: blocks of one tile of at most 64 rows, whose Q buffers
// (two 64-row halves of 128-row tiles; an MMA reads what follows as rows 64 .. 127, which do not
// exist) leave room for more slots.
template <int DH, bool NARROW>
struct Cfg {
  static constexpr int halves = DH / 64;
  static constexpr uint32_t slot = halves * kHalf;  // K or V of one tile
  static constexpr uint32_t q_step = NARROW ? kHalf / 2 : slot;  // from one Q buffer to the other
  // Slots of K and of V.  A V tile stays longer: until its row's softmax and product are done.
  static constexpr int nk = DH == 128 ? (NARROW ? 3 : 2) : (NARROW ? 6 : 5);
  static constexpr int nv = DH == 128 ? 3 : (NARROW ? 6 : 5);
  static constexpr int slots = nk + nv;
  static constexpr uint32_t off_ring = NARROW ? slot : 2 * slot;
  static constexpr uint32_t off_bar = off_ring + slots * slot;
  static constexpr uint32_t smem = off_bar + sizeof(Tail);
  static constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DH, false, true);
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// One lane of the converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}
// A value that is the same in all lanes, known to be so by the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Products of 16 columns (S) or 16 keys (P V) are issued from descriptors whose
// constant halves are immediates and whose addresses grow by constants: formed
// one by one in a loop, the descriptors took 100 to 300 clocks a product, more
// than the tensor pipe.  Fields as in smem_desc_sw128: 128-byte swizzle, 1024
// bytes between 8-row groups.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
// The first (H = 0) or second half of S's products.
template <int DH, int H>
__device__ __forceinline__ void issue_scores(uint32_t ts, uint32_t qa, uint32_t ka, uint32_t idesc) {
  const uint32_t q = (qa >> 4) | (1u << 16), k = (ka >> 4) | (1u << 16);
#pragma unroll
  for (int kk = H * DH / 32; kk < (H + 1) * DH / 32; ++kk) {
    const uint32_t off = (kk >> 2) * (kHalf >> 4) + (kk & 3) * 2;
    mma_bf16(ts, desc_of(q + off), desc_of(k + off), idesc, kk > 0);
  }
}
// 16-key steps of the first (H = 0) or second half of the keys, up to `steps`; `add`: to what O holds.
template <int H>
__device__ __forceinline__ void issue_sums(uint32_t to, uint32_t tp, uint32_t va, uint32_t idesc, int steps, bool add) {
  const uint32_t v = (va >> 4) | ((kHalf >> 4) << 16);
#pragma unroll
  for (int i = 4 * H; i < 4 * H + 4; ++i)
    if (i < steps) mma_bf16_ts(to, tp + 8 * i, desc_of(v + 128 * i), idesc, i > 0 || add);
}

// Waits for a phase, at most kTries tries (about a second, 50 ms should each come back at once);
// false when they have run out or *abort is set.  Short on purpose: there are some fifty waits, and
// with a timer in each of them the kernel's code was 150 KB, of which every warp fetched its share anew.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int n = kTries; n > 0; --n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 15) == 0 && *abort) return false;
  }
  *abort = 1;
  return false;
}

// All lanes wait; true when all saw the phase end (the tcgen05 operations that
// follow are warp-collective).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = wait_bounded(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Every lane with `need` waits for a phase of a barrier of its own, all at once: a wait costs some
// 200 clocks even when its phase is long over, and an issuing warp that made its five one after the
// other came to the probabilities 500 clocks after they were there.  The lanes ask again and again
// (kPolls times at most, about a second) and do not sleep on a barrier, which woke them
// some 100 clocks late; for the eight softmax warps that would take issue slots from one another
// (8192 tokens over 8192 rows, in turn on one machine: 1051 us so, with sleeping waits 1079, with all waits so 1094).
__device__ __forceinline__ bool lanes_wait(uint64_t* bar, uint32_t parity, bool need, volatile int* abort) {
  bool ok = !need;
#pragma unroll 1
  for (int n = kPolls; n > 0; --n) {
    if (!ok) ok = mbar_test_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) {
      __syncwarp();  // what one lane has seen to be there, all have
      return true;
    }
    if ((n & 15) == 0 && __any_sync(0xffffffffu, *abort)) return false;
  }
  *abort = 1;
  return false;
}

// All lanes, whose work so far the arrival of one of them announces.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 2^x on the SFU: relative error about 2^-22, far below P's rounding to bf16.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void st_v8u(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// `left`: the tiles of the CTA's range from tile t0 of the item on.
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, const Item& it, int t0, long long left) {
  Unit x;
  x.t0 = t0;
  x.t1 = it.tiles - t0 < left ? it.tiles : t0 + (int)left;
  x.tiles = it.tiles;
  x.tok0 = it.i << a.w.ctok_log2;
  x.ntok = min(it.s.len - x.tok0, a.w.ctok);
  x.two = x.ntok > a.tile_tok;
  x.rows_end = a.w.N ? it.s.L : it.s.L + x.tok0 + x.ntok;
  x.pre = a.w.N ? (it.s.L + kKeys - 1) / kKeys : it.tiles;
  // A causal first row tile does not see the key tiles that only the second one does.
  x.end0 = x.two && !a.w.N ? min(x.t1, (it.s.L + x.tok0 + a.tile_tok + kKeys - 1) / kKeys) : x.t1;
  const int l = it.lg / a.w.nh;
  x.kvh = it.lg - l * a.w.nh;
  x.b = it.b;
  x.L = it.s.L;
  x.tree0 = l * a.w.T + it.s.q0;
  x.row0 = x.tree0 + x.tok0;
  x.pool0 = l * (a.cache.n_pages * a.cache.page_size);
  return x;
}
__device__ __forceinline__ int stream_end(const Unit& x, int s) { return x.two && s == 0 ? x.end0 : x.t1; }
// Keys of tile t that rows of stream s may see, at most 128.
__device__ __forceinline__ int tile_keys(const AttnArgs& a, const Unit& x, int s, int t) {
  if (t >= x.pre) return min(kKeys, a.w.N - (t - x.pre) * kKeys);
  const int end = x.two && s == 0 && !a.w.N ? x.L + x.tok0 + a.tile_tok : x.rows_end;
  return min(kKeys, end - t * kKeys);
}
// Rows of tile t that were copied and may be read as they are.
__device__ __forceinline__ int tile_rows_loaded(const AttnArgs& a, const Unit& x, int t) {
  return t >= x.pre ? min(kKeys, a.w.N - (t - x.pre) * kKeys) : min(kKeys, x.rows_end - t * kKeys);
}

// One lane per box of a tile of cache rows: its page's entry in the table, and its row within the
// page; entry -1: the tile has no such box.
struct Box {
  int id, off;
};
__device__ __forceinline__ Box box_of(const AttnArgs& a, const Unit& x, int t, int lane, int box_rows) {
  const int r = t * kKeys + lane * box_rows;
  Box b{-1, 0};
  if (t < x.pre && lane < kKeys / box_rows && r < x.rows_end) {
    const int pg = r / a.cache.page_size;
    b.off = r - pg * a.cache.page_size;
    b.id = a.cache.page_table[(size_t)x.b * a.cache.max_pages + pg];
  }
  return b;
}
// Copies tile t of K or V into `dst` (all lanes; `b`: box_of the tile).  A page that does not exist:
// rows behind the pool, which arrive as zeros.
template <int HALVES>
__device__ __forceinline__ void copy_tile(const AttnArgs& a, const Unit& x, int t, const Box& b, int box_rows, const void* cache,
                                          const void* tree_rows, uint8_t* dst, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  const bool tree = t >= x.pre;
  const int step = tree ? 64 : box_rows, boxes = (tile_rows_loaded(a, x, t) + step - 1) / step;
  int row = x.tree0 + (t - x.pre) * kKeys + lane * 64;
  if (!tree) {
    const bool exists = b.id >= 0 && b.id < a.cache.n_pages;
    row = exists ? x.pool0 + b.id * a.cache.page_size + b.off : a.cache.n_pages * a.cache.page_size * a.w.nl;
    if (!exists && lane < boxes) set_status(a.d_status, MEDUSA_DEV_BAD_INDEX);
  }
  __syncwarp();
  if (elect_one()) mbar_expect_tx(bar, (uint32_t)(boxes * step * 128 * HALVES));
  const void* map = tree ? tree_rows : cache;
  __syncwarp();
  const int r = __shfl_sync(0xffffffffu, row, lane & 15), box = lane & 15, h = lane >> 4;
  if (box < boxes && h < HALVES) tma_load_3d(dst + h * kHalf + box * step * 128, map, bar, 64 * h, x.kvh, r);
  __syncwarp();
}

// The next description, `n` units after the first: false on a timeout.
__device__ __forceinline__ bool read_unit(Tail* tail, int n, Unit& x, volatile int* abort) {
  const int k = n % kUnits;
  if (!warp_wait(&tail->bars.u_full[k], (uint32_t)(n / kUnits) & 1u, abort)) return false;
  x = tail->units[k];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&tail->bars.u_free[k]);
  return true;
}

}  // namespace tc

template <int DH, bool NARROW>
__global__ void __launch_bounds__(tc::kThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kt,
                     const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ AttnArgs a, const int box_rows) {
  using namespace tc;
  using C = Cfg<DH, NARROW>;
  auto two = [](const Unit& x) { return !NARROW && x.two; };  // two row tiles
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(C::smem <= 232448, "shared memory of a CTA");
  Tail* tail = reinterpret_cast<Tail*>(smem + C::off_bar);
  Bars* bars = &tail->bars;
  volatile int& s_abort = tail->abort;
  if (smem_u32(smem) & 1023u) {  // the same in every thread
    if (threadIdx.x == 0) set_status(a.d_status, MEDUSA_DEV_TIMEOUT);
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_abort = 0;
#pragma unroll 1
    for (int i = 0; i < C::slots; ++i) {
      for (int k = 0; k < 3; ++k) mbar_init(&bars->full[k][i], 1);
      mbar_init(&bars->empty[i], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 2);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->turn[s], 1);
      mbar_init(&bars->p_half[s], 4);
      mbar_init(&bars->p_full[s], 4);
      mbar_init(&bars->o_full[s], 1);
      mbar_init(&bars->o_free[s], 4);
      mbar_init(&bars->drain[s], 1);
    }
    mbar_init(&bars->ml_full, 4);
    for (int k = 0; k < kUnits; ++k) {
      mbar_init(&bars->u_full[k], 1);
      mbar_init(&bars->u_free[k], kUnitReaders);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&tail->tmem, kTmemCols);
    tmem_relinquish();
  }
  if (lane == 0 && (warp == 0 || warp == 3)) {
    tma_prefetch(&tm_q);
    tma_prefetch(&tm_k);
    tma_prefetch(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Nothing above reads memory an earlier kernel may write.
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = tail->tmem;
  if (blockIdx.x == 0)
#pragma unroll 1
    for (int b = threadIdx.x; b < a.w.B; b += kThreads)
      if (!seq_of(a.w, b).ok) set_status(a.d_status, MEDUSA_DEV_BAD_LENGTH);
  Plan pl;
  Item it;
  const bool any = plan_find(a.w, pl, it, tail->plan, blockIdx.x);
  if (threadIdx.x == 0) note_shared(a, pl, it, any);
  __syncthreads();  // the plan is no longer read

  // Registers move from the four issuing warps to the softmax warps, which hold 128 scores a
  // thread: 128 x 80 + 256 x 208 of the 384 x 168 that the CTA is launched with.
  __syncwarp();  // one lane may have come out of the set-up on its own
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == 0) {
    // ------------------------------------------------------------ items, Q and K
    const long long u0 = pl.Q * blockIdx.x;
    long long left = !any ? 0 : u0 + pl.Q < pl.U ? pl.Q : pl.U - u0;
    int t0 = any ? (int)(u0 - it.first) : 0;
    int c = 0;                                           // tiles
    int qn0 = 0, qn1 = 0, qsel = 0;                      // loads into the two Q buffers
    uint32_t flips[3] = {0, 0, 0}, used[3] = {0, 0, 0};  // bits: a barrier has been used an odd number of times, at all
    Unit x{};
    bool alive = true;
#pragma unroll 1
    for (int n = 0;; ++n) {
      // Unit n is described (t1 = 0: there is none) before unit n - 1, x, is copied.
      const int k = n % kUnits;
      if (n >= kUnits && !(alive = warp_wait(&bars->u_free[k], (uint32_t)(n / kUnits - 1) & 1u, &s_abort))) break;
      Unit y{};
      if (left > 0) {
        y = unit_of(a, it, t0, left);
        left -= y.t1 - y.t0;
        t0 = 0;
        if (left > 0 && !next_item(a.w, pl.odd, it)) left = 0;
      }
      if (lane == 0) {
        tail->units[k] = y;
        mbar_arrive(&bars->u_full[k]);
      }
      __syncwarp();
      if (n > 0) {
        Box b{-1, 0};
#pragma unroll 1
        for (int t = x.t0 - 1; t < x.t1; ++t) {
          const Box next = box_of(a, x, t + 1, lane, box_rows);  // on its way while this tile waits
          if (t >= x.t0) {
            const int sl = c % C::nk, set = two(x) ? 2 : (t - x.t0) & 1;
            if (c >= C::nk && !(alive = warp_wait(&bars->empty[sl], (uint32_t)(c / C::nk - 1) & 1u, &s_abort))) break;
            copy_tile<C::halves>(a, x, t, b, box_rows, &tm_k, &tm_kt, smem + C::off_ring + sl * C::slot, &bars->full[set][sl]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
              if (k == set) {
                flips[k] ^= 1u << sl;
                used[k] |= 1u << sl;
              }
            ++c;
            // Q behind the unit's first K, whose slot was freed a tile before the Q buffers were.
            if (t == x.t0) {
#pragma unroll 1
              for (int k = 0; k < (two(x) ? 2 : 1); ++k) {
                const int qb = two(x) ? k : qsel, before = qb ? qn1 : qn0;
                if (before > 0 && !(alive = warp_wait(&bars->q_empty[qb], (before - 1) & 1, &s_abort))) break;
                if (elect_one()) {
                  mbar_expect_tx(&bars->q_full[qb], (uint32_t)(C::halves * a.tile_tok * a.G * 128));
                  for (int h = 0; h < C::halves; ++h)
                    tma_load_3d(smem + qb * C::q_step + h * kHalf, &tm_q, &bars->q_full[qb], 64 * h, x.kvh * a.G, x.row0 + k * a.tile_tok);
                }
                __syncwarp();
                qn0 += qb == 0;
                qn1 += qb == 1;
              }
              if (!alive) break;
              if (!two(x)) qsel ^= 1;
            }
          }
          b = next;
        }
        if (!alive) break;
      }
      if (y.t1 <= 0) break;
      x = y;
    }
    if (lane == 0) {
      tail->q_loads[0] = qn0;
      tail->q_loads[1] = qn1;
      tail->note_loads(0, used, flips);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ V
    int c = 0;
    uint32_t flips[3] = {0, 0, 0}, used[3] = {0, 0, 0};
    bool alive = true;
    Unit x;
#pragma unroll 1
    for (int n = 0; !a.withhold && (alive = read_unit(tail, n, x, &s_abort)) && x.t1 > 0; ++n) {
      Box b{-1, 0};
#pragma unroll 1
      for (int t = x.t0 - 1; t < x.t1; ++t) {
        const Box next = box_of(a, x, t + 1, lane, box_rows);
        if (t >= x.t0) {
          const int i = c % C::nv, sl = C::nk + i, set = two(x) ? 2 : (t - x.t0) & 1;
          if (c >= C::nv && !(alive = warp_wait(&bars->empty[sl], (uint32_t)(c / C::nv - 1) & 1u, &s_abort))) break;
          copy_tile<C::halves>(a, x, t, b, box_rows, &tm_v, &tm_vt, smem + C::off_ring + sl * C::slot, &bars->full[set][sl]);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (k == set) {
              flips[k] ^= 1u << sl;
              used[k] |= 1u << sl;
            }
          ++c;
        }
        b = next;
      }
      if (!alive) break;
    }
    if (lane == 0) tail->note_loads(1, used, flips);
  } else {
    // ------------------------------------------------------------ MMA issuer of stream s
    const int s = warp - 1;
    const uint32_t ts = tmem + 128 * s, to = tmem + 256 + 128 * s;
    int g = 0;                               // tiles of earlier units (two ring slots each)
    int qn0 = 0, qn1 = 0, qsel = 0, np = 0;  // np: tiles of this stream
    int turns = 0;                           // taken
    uint32_t alone = 0, shared = 0;          // bit: parity of the next phase of full[s], full[2]
    bool alive = true;
    Unit x;
#pragma unroll 1
    for (int n = 0; (alive = read_unit(tail, n, x, &s_abort)) && x.t1 > 0; ++n) {
      const int qb = two(x) ? s : qsel, end = stream_end(x, s);
      if (!(alive = lanes_wait(&bars->q_full[lane & 1], ((lane & 1) ? qn1 : qn0) & 1, two(x) ? lane < 2 : lane == qb, &s_abort))) break;
      if (two(x)) {  // the other stream's rows
        if (lane == 0) mbar_arrive(&bars->q_empty[1 - qb]);
        __syncwarp();
      }
      const int first = two(x) ? x.t0 : x.t0 + s, step = two(x) ? 1 : 2;
      const uint32_t qa = smem_u32(smem + qb * C::q_step);
      auto slot_k = [&](int t) { return (g + t - x.t0) % C::nk; };
      auto slot_v = [&](int t) { return C::nk + (g + t - x.t0) % C::nv; };
      // Waits for a slot of a tile that this stream uses (or, of two row tiles, of any), each once.
      auto came = [&](int sl) {
        const bool ok = warp_wait(&bars->full[two(x) ? 2 : s][sl], ((two(x) ? shared : alone) >> sl) & 1u, &s_abort);
        if (two(x)) shared ^= 1u << sl;
        else alone ^= 1u << sl;
        return ok;
      };
      // Rows of V behind the last one of tile t, up to what P V reads: zeros.
      auto clear_rest = [&](int cv, int steps, int have) {
        uint8_t* vb = smem + C::off_ring + cv * C::slot;
#pragma unroll 1
        for (int i = lane; i < (steps * 16 - have) * 8 * C::halves; i += 32) {
          const int r = have + i / (8 * C::halves), cc = i % (8 * C::halves);
          *reinterpret_cast<uint4*>(vb + (cc >> 3) * kHalf + r * 128 + (cc & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      // Step by step: P V of tile t - step, then S of tile t, back to back.  Of a block of two row
      // tiles the streams take turns.  The tensor pipe takes products in the order of their issue:
      // when both streams issued at will, theirs came in turns of one product, ended together, and
      // both softmaxes then ran together with nothing in the pipe.  A turn is passed on before the
      // last products are issued: the other warp needs some 400 clocks to see it.
#pragma unroll 1
      for (int t = first;; t += step) {
        const bool had = t > first && t - step < end, has = t < end;
        if (!had && two(x) && t > first) {  // a tile of the other stream's alone
          if (!(alive = came(slot_k(t - 1)) && came(slot_v(t - 1)))) break;
          if (lane == 0) {
            mbar_arrive(&bars->empty[slot_k(t - 1)]);
            mbar_arrive(&bars->empty[slot_v(t - 1)]);
          }
          __syncwarp();
        }
        // Lane 0: V; 1: K (of one row tile the next K may still be far, and P V does not wait for it);
        // 2: the turn; 3: P's first half; 4: O, read out by the unit before.
        const int cv = slot_v(t - step), ck = slot_k(t);
        const bool k_too = has && (two(x) || !had), turn = two(x) && (s || turns);
        const uint32_t mine = two(x) ? shared : alone;
        uint64_t* const rows = bars->full[two(x) ? 2 : s];
        uint64_t* const bar = lane == 0 ? rows + cv : lane == 1 ? rows + ck : lane == 2 ? &bars->turn[s] : lane == 3 ? &bars->p_half[s] : &bars->o_free[s];
        const uint32_t phase = lane == 0 ? mine >> cv : lane == 1 ? mine >> ck : lane == 2 ? turns - (s == 0) : lane == 3 ? np : n - 1;
        const bool need = lane == 0 || lane == 3 ? had : lane == 1 ? k_too : lane == 2 ? turn : lane == 4 && had && t - step == first && n > 0;
        const int steps = had ? (tile_keys(a, x, s, t - step) + 15) >> 4 : 0, have = had ? tile_rows_loaded(a, x, t - step) : 0;
        const uint32_t uv = uniform(smem_u32(smem + C::off_ring + cv * C::slot)), uk = uniform(smem_u32(smem + C::off_ring + ck * C::slot));
        const uint32_t uq = uniform(qa), ut = uniform(ts), uo = uniform(to);
        if (!(alive = lanes_wait(bar, phase & 1u, need, &s_abort))) break;
        const uint32_t seen = (had ? 1u << cv : 0u) | (k_too ? 1u << ck : 0u);
        if (two(x)) shared ^= seen;
        else alone ^= seen;
        turns += two(x);
        if (had) {
          if (have < steps * 16) clear_rest(cv, steps, have);
          tc_fence_after();
          if (elect_one()) issue_sums<0>(uo, ut, uv, C::idesc_pv, steps, t - step > first);
          __syncwarp();
          if (!(alive = lanes_wait(&bars->p_full[s], np & 1, true, &s_abort))) break;
          ++np;
        }
        tc_fence_after();
        if (two(x)) {
          if (elect_one()) {
            if (had) issue_sums<1>(uo, ut, uv, C::idesc_pv, steps, true);
            if (has) issue_scores<DH, 0>(ut, uq, uk, C::idesc_qk);
            mbar_arrive(&bars->turn[1 - s]);
            if (has) {
              issue_scores<DH, 1>(ut, uq, uk, C::idesc_qk);
              mma_commit(&bars->s_full[s]);
              mma_commit(&bars->empty[ck]);
              if (t + step >= end) mma_commit(&bars->q_empty[qb]);
            } else if (had) {
              mma_commit(&bars->o_full[s]);
            }
            if (had) mma_commit(&bars->empty[cv]);
          }
          __syncwarp();
          if (t == x.t1) break;
        } else {
          if (had && elect_one()) {
            issue_sums<1>(uo, ut, uv, C::idesc_pv, steps, true);
            if (!has) mma_commit(&bars->o_full[s]);
            mma_commit(&bars->empty[cv]);
            mma_commit(&bars->empty[cv]);
          }
          __syncwarp();
          if (!has) break;
          if (had) {
            if (!(alive = came(ck))) break;
            tc_fence_after();
          }
          if (elect_one()) {
            issue_scores<DH, 0>(ut, uq, uk, C::idesc_qk);
            issue_scores<DH, 1>(ut, uq, uk, C::idesc_qk);
            mma_commit(&bars->s_full[s]);
            mma_commit(&bars->empty[ck]);
            mma_commit(&bars->empty[ck]);
            if (t + step >= end) mma_commit(&bars->q_empty[qb]);
          }
          __syncwarp();
        }
      }
      if (!alive) break;
      if (first >= end) {  // no tile of this unit is this stream's
        if (n > 0 && !(alive = warp_wait(&bars->o_free[s], (n - 1) & 1, &s_abort))) break;
        if (lane == 0) {
          mbar_arrive(&bars->q_empty[qb]);
          mbar_arrive(&bars->o_full[s]);  // so that no unit's output passes this wait for the one before
        }
        __syncwarp();
      }
      qn0 += two(x) || qsel == 0;
      qn1 += two(x) || qsel == 1;
      if (!two(x)) qsel ^= 1;
      g += x.t1 - x.t0;
    }
    if (elect_one()) {
      // This warp's MMAs and the arrives they signal, before TMEM and shared memory go away.
      mma_commit(&bars->drain[s]);
      mbar_wait_bounded(&bars->drain[s], 0, nullptr, kDrainNs);
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ softmax and output of stream s
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int s = (warp - 4) >> 2, q4 = warp & 3;
    const int m = 32 * q4 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t ts = lanes + 128 * s, to = lanes + 256;
    const float sc = a.scale_log2;
    const uint64_t sc2 = pack2(sc, sc);
    const int mt = m / a.G, mh = m - mt * a.G;  // token and q head within the row tile
    int ns = 0, nb = 0;                         // tiles, units of one row tile
    bool alive = true;
    Unit x;
#pragma unroll 1
    for (int n = 0; (alive = read_unit(tail, n, x, &s_abort)) && x.t1 > 0; ++n) {
      const int end = stream_end(x, s);
      const int rt = two(x) ? s : 0, tok = rt * a.tile_tok + mt;  // within the block
      const bool row_ok = mt < a.tile_tok && tok < x.ntok;
      const bool busy = __any_sync(0xffffffffu, row_ok);  // some row of this warp exists
      const int first = two(x) ? x.t0 : x.t0 + s, step = two(x) ? 1 : 2;
      const int sees = a.w.N ? x.L : x.L + x.tok0 + tok + 1;                    // cache rows this row sees
      const int all_see = a.w.N ? x.L : x.L + x.tok0 + rt * a.tile_tok + 1;     // that every row sees
      float mu = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int t = first; t < end; t += step, ++ns) {
        const int keys = tile_keys(a, x, s, t);
        const bool tree = t >= x.pre, masked = tree || keys < kKeys || t * kKeys + kKeys > all_see;
        if (!(alive = warp_wait(&bars->s_full[s], ns & 1, &s_abort))) break;
        if (!busy) {
          warp_arrive(&bars->p_half[s]);
          warp_arrive(&bars->p_full[s]);
          continue;
        }
        tc_fence_after();
        if (masked) {
          // Tiles at the end of what a row sees: keys it does not see get -inf, in a pass of its own
          // in tensor memory.  Code that runs once in many tiles is kept short: fetched cold, the
          // unrolled form (and an unrolled output below) took 3000 and 6000 clocks.
          const int j = (tree ? t - x.pre : t) * kKeys;  // first key
          const int lim = (tree ? a.w.N : sees) - j;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int c = lim - 32 * q;
            uint32_t w = !row_ok || c <= 0 ? 0u : c >= 32 ? 0xffffffffu : (1u << c) - 1u;
            if (tree && w) w &= a.mask[(size_t)(x.tok0 + tok) * a.W + (j >> 5) + q];
            float z[32];
            __syncwarp();
            tmem_ld32(ts + 32 * q, z);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = (w >> i) & 1u ? z[i] : -INFINITY;
            tmem_st32(ts + 32 * q, z);
          }
          tmem_wait_st();
        }
        float v[128];
        __syncwarp();
        tmem_ld32(ts, v);
        tmem_ld32(ts + 32, v + 32);
        tmem_ld32(ts + 64, v + 64);
        tmem_ld32(ts + 96, v + 96);
        tmem_wait_ld();
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 128; i += 2) m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], v[i], v[i + 1]);
        const float mn = fmaxf(mu, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sc);
        const bool need = row_ok && mn > mu + 8.f;
        const float f = need ? fast_exp2(mu - mn) : 1.f;  // 0 for the first keys seen
        if (need) mu = mn;
        const float off = mu == -INFINITY ? 0.f : -mu;  // nothing seen: every 2^x is of -inf
        const uint64_t off2 = pack2(off, off);
        uint64_t r2[2] = {0ull, 0ull};
        // Probabilities, over columns of S that have been read.
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = unpack2(fma2(pack2(v[32 * q + 2 * i], v[32 * q + 2 * i + 1]), sc2, off2));
            const float e0 = fast_exp2(e.x), e1 = fast_exp2(e.y);
            r2[i & 1] = add2(r2[i & 1], pack2(e0, e1));
            pk[i] = bf16x2_rn(e0, e1);
          }
          tmem_st16u(ts + 16 * q, pk);
          if (q == 1) {
            if (t > first && __any_sync(0xffffffffu, need)) {
              sum *= f;
#pragma unroll 1
              for (int q = 0; q < DH / 32; ++q) {
                float o[32];
                __syncwarp();
                tmem_ld32(to + 128 * s + 32 * q, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f;
                tmem_st32(to + 128 * s + 32 * q, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bars->p_half[s]);
            __syncwarp();
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bars->p_full[s]);
        const float2 a0 = unpack2(r2[0]), a1 = unpack2(r2[1]);
        sum += (a0.x + a0.y) + (a1.x + a1.y);
      }
      if (!alive) break;

      // The unit's result: O / sum, or a part of it for the merge.
      const bool whole = x.t0 == 0 && x.t1 == x.tiles, has = first < end;
      bool o1 = false;
      float w0 = 1.f, w1 = 0.f;
      // The sums area is free, and every phase of o_free[1] seen, once the unit before is out.
      if (s == 1 && n > 0 && !(alive = warp_wait(&bars->o_free[1], (n - 1) & 1, &s_abort))) break;
      if (!two(x)) {
        if (s == 1) {
          tail->ml[m] = make_float2(mu, sum);
          warp_arrive(&bars->ml_full);
        } else {
          if (!(alive = warp_wait(&bars->ml_full, nb & 1, &s_abort))) break;
          const float2 q = tail->ml[m];
          o1 = x.t1 - x.t0 > 1;  // stream 1 had a tile
          const float mm = fmaxf(mu, q.x), off = mm == -INFINITY ? 0.f : mm;
          w0 = fast_exp2(mu - off);
          w1 = fast_exp2(q.x - off);
          sum = fmaf(sum, w0, q.y * w1);
          mu = mm;
        }
        ++nb;
      }
      if (two(x) || s == 0) {
        // Of one row tile both streams' (stream 1's phases of units with two are over: ml_full comes later).
        if (!(alive = lanes_wait(&bars->o_full[two(x) ? s : lane & 1], n & 1, lane < (two(x) ? 1 : 2), &s_abort))) break;
        if (busy) {
          tc_fence_after();
          const float inv = !whole ? 1.f : row_ok ? row_scale(a, x.L, x.tok0 + tok, sum) : 0.f;
          w0 *= inv;
          w1 *= inv;
          const size_t orow = ((size_t)x.row0 + tok) * a.Hq + x.kvh * a.G + mh;
          const int slot = 2 * blockIdx.x + (x.t0 == 0 ? 1 : 0), prow = rt * 128 + m;
#pragma unroll 1
          for (int q = 0; q < DH / 32; ++q) {
            float o[32];
            __syncwarp();
            if (has) {
              tmem_ld32(to + 128 * s + 32 * q, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = w0 == 0.f ? 0.f : o[i] * w0;
              if (o1) {
                float p[32];
                tmem_ld32(to + 128 + 32 * q, p);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = w1 == 0.f ? o[i] : fmaf(p[i], w1, o[i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (!row_ok) continue;
            if (whole) {
              uint16_t* dst = static_cast<uint16_t*>(a.out) + orow * a.d + 32 * q;
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = bf16x2_rn(o[2 * i], o[2 * i + 1]);
              if (a.out32) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (32 * q + 16 * i < a.d) st_v8u(dst + 16 * i, pk + 8 * i);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (32 * q + 8 * i < a.d)
                    *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
              }
            } else {
              float* dst = part_at(a, slot, prow, 8 * q);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (32 * q + 4 * i < a.d)
                  *reinterpret_cast<float4*>(dst + i * (4 * part_rows(NARROW ? 64 : 256))) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          if (row_ok) {
            if (!whole) a.part_ml[(size_t)slot * a.R + prow] = make_float2(mu, sum);
            else if (a.lse) a.lse[orow] = lse_of(mu, sum);
          }
          tc_fence_before();
        }
        warp_arrive(&bars->o_free[s]);
        if (!two(x)) warp_arrive(&bars->o_free[1]);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && s_abort) {
    set_status(a.d_status, MEDUSA_DEV_TIMEOUT);
    // No copy may land after exit: wait (bounded) for the last phase of every load barrier.
    for (int q = 0; q < 2; ++q)
      if (tail->q_loads[q] > 0) mbar_wait_bounded(&bars->q_full[q], (tail->q_loads[q] - 1) & 1, nullptr, kDrainNs);
#pragma unroll 1
    for (int i = 0; i < 3 * C::slots; ++i) {
      const int k = i / C::slots, sl = i - k * C::slots;
      if (((tail->loads[0][k] | tail->loads[1][k]) >> sl) & 1)
        mbar_wait_bounded(&bars->full[k][sl], (((tail->odd[0][k] | tail->odd[1][k]) >> sl) & 1) ^ 1, nullptr, kDrainNs);
    }
  }
  if (warp == 1) {
    __syncwarp();  // the lanes may come out of the barrier apart, and the warp frees once
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// [rows][heads][d] bf16 with `pitch` elements between rows; boxes of 64 columns x bh heads x br rows.
static bool make_map(CUtensorMap* m, const void* base, int d, int heads, long long rows, long long pitch, int bh, int br) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)pitch * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)br}, es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH, bool NARROW>
static medusa_status go(const AttnArgs& a, const CUtensorMap* m, int box_rows, cudaStream_t s) {
  auto kern = paged_attn_tc_kernel<DH, NARROW>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tc::Cfg<DH, NARROW>::smem) != cudaSuccess)
    return MEDUSA_ERR_CUDA;
  launch_pdl(kern, dim3(a.w.ctas), dim3(tc::kThreads), tc::Cfg<DH, NARROW>::smem, s, m[0], m[1], m[2], m[3], m[4], a, box_rows);
  return MEDUSA_OK;
}

medusa_status paged_attention_tc(const AttnArgs& a, cudaStream_t s) {
  if (!encode_fn()) return MEDUSA_ERR_CUDA;
  int box_rows = 128;
  while (a.cache.page_size % box_rows) box_rows /= 2;
  const long long tokens = (long long)a.w.nl * a.w.T, rows = (long long)a.w.nl * a.cache.n_pages * a.cache.page_size;
  CUtensorMap m[5];
  if (!make_map(&m[0], a.q, a.d, a.Hq, tokens, a.ldq, a.G, a.tile_tok)) return MEDUSA_ERR_CUDA;
  if (!make_map(&m[1], a.k_pages, a.d, a.Hkv, rows, (long long)a.Hkv * a.d, 1, box_rows)) return MEDUSA_ERR_CUDA;
  if (!make_map(&m[2], a.v_pages, a.d, a.Hkv, rows, (long long)a.Hkv * a.d, 1, box_rows)) return MEDUSA_ERR_CUDA;
  if (a.w.N) {
    if (!make_map(&m[3], a.kt, a.d, a.Hkv, tokens, (long long)a.Hkv * a.d, 1, 64)) return MEDUSA_ERR_CUDA;
    if (!make_map(&m[4], a.vt, a.d, a.Hkv, tokens, (long long)a.Hkv * a.d, 1, 64)) return MEDUSA_ERR_CUDA;
  } else {
    m[3] = m[1];
    m[4] = m[2];
  }
  if (a.R == 64) return a.d <= 64 ? go<64, true>(a, m, box_rows, s) : go<128, true>(a, m, box_rows, s);
  return a.d <= 64 ? go<64, false>(a, m, box_rows, s) : go<128, false>(a, m, box_rows, s);
}

}  // namespace paged
}  // namespace medusa
