/* medusa_test_hooks.h: entry points of libmedusa_gb300 that exist only for its
 * own failure-detection tests.  They are NOT part of the library's API: a
 * program that computes with the library never calls them, and they may
 * change or disappear without notice.  The paper has no counterpart.
 *
 * Same conventions as medusa.h (caller-owned device pointers, stream-ordered,
 * host validation before any launch, device errors in d_status).
 */
#ifndef MEDUSA_TEST_HOOKS_H
#define MEDUSA_TEST_HOOKS_H

#include "medusa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* medusa_linear_test_stall: runs medusa_linear (bf16) with the loads of its
 * first pipeline stage withheld, so the kernel's bounded barrier waits (1 s)
 * run out on purpose: the kernel stops every role, waits (bounded) for its
 * copies and MMAs in flight, frees its tensor memory and sets
 * MEDUSA_DEV_TIMEOUT in d_status; y is not meaningful.  The context stays
 * usable (no fault, no trap), so a test can check the status and then make an
 * ordinary call.  Same arguments and validation as medusa_linear. */
medusa_status medusa_linear_test_stall(const void* x, const void* w, void* y, int T, int K, int Nout, void* ws,
                                       size_t ws_bytes, int32_t* d_status, medusa_stream_t stream);

/* medusa_paged_attention_test_stall: medusa_paged_attention, of a shape that runs on
 * tensor cores (INVALID_ARG otherwise), whose values are never loaded, so that
 * its waits run out after one to two seconds: the kernel ends as described above and
 * sets MEDUSA_DEV_TIMEOUT; out and lse are not meaningful. */
medusa_status medusa_paged_attention_test_stall(const void* q, int64_t ldq, const void* k_pages, const void* v_pages,
                                                const int32_t* page_table, const int32_t* q_start,
                                                const int32_t* prefix_len, int n_layers, int T, int B, int Hq, int Hkv,
                                                int d, int n_pages, int page_size, int max_pages, float scale,
                                                medusa_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                                int32_t* d_status, medusa_stream_t stream);

/* medusa_linear_w4_test_stall: medusa_linear_w4, of a size that runs on tensor memory
 * (INVALID_ARG otherwise), whose first tokens are never loaded: its waits run out
 * after one to two seconds and it ends as medusa_linear_test_stall does. */
medusa_status medusa_linear_w4_test_stall(const void* x, int64_t ldx, const uint32_t* qweight, const void* scales,
                                          const uint8_t* zeros, int T, int K, int Nout, int group, void* y,
                                          medusa_dtype y_dt, int32_t* d_status, medusa_stream_t stream);

/* medusa_linear_w4_test_division: which kernel a layer of medusa_linear_w4 runs on, on the
 * current device, and how it is divided: division[0] is 0 (product instructions fed
 * from registers; the rest is 0), 1 (tensor memory, work divided evenly) or 2 (tensor
 * memory, equal tiles), then the CTAs that share a tile, a tile's tokens and features, the
 * tiles, the CTAs.  division is host memory; nothing is launched. */
medusa_status medusa_linear_w4_test_division(int T, int K, int Nout, int32_t* division);

#ifdef __cplusplus
}
#endif

#endif /* MEDUSA_TEST_HOOKS_H */
