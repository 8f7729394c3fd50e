/*
 * gsfp8_test.h -- test hooks of libgsfp8 (not part of the computation).
 *
 * The kernels fed by TMA -- fp8_gemm_block_scaled, fp4_gemm_block_scaled and the
 * products of gs_master_update_muon -- wait on shared-memory barriers for their
 * loads, for the tensor cores and for the warps that store.
 * Every such wait is bounded (about 2 s by %globaltimer); a kernel that gives
 * up records GS_ERR_TIMEOUT in the device status word (gs_device_status),
 * lets its own copies and MMAs in flight finish, frees its tensor memory and
 * returns, leaving the CUDA context usable.  This hook
 * lets a test exercise that path without a fault: no trap, no bad address,
 * no endless loop -- a barrier that nothing completes, waited on with its
 * limit.
 */
#ifndef GSFP8_TEST_H
#define GSFP8_TEST_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* on != 0: launches made from now on by this process of the kernels named
 * above issue no TMA loads, so their first bounded wait runs out: the launch
 * takes about 2 s, writes nothing valid to its outputs and records
 * GS_ERR_TIMEOUT.  on == 0 restores normal operation.  Process-wide; set it
 * only while no other thread launches those kernels.  Returns GS_OK. */
int gs_test_set_stall(int on);

/* r[i] = sqrt(v[i]) (device, n even, not overlapping) by the code that forms
 * the roots of the AdamW step with 8-bit moments, whose outputs show a root
 * only through eight-bit codes and block scales. */
int gs_test_adamw_root(const float* v, float* r, int64_t n, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GSFP8_TEST_H */
