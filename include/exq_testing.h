/*
 * exq_testing.h -- test hooks of libexq. They have no counterpart in the
 * ExLlamaV2 pages: one lets a test watch a bounded device-side wait give up
 * without faulting, trapping or hanging the GPU, the others show it arithmetic
 * that kernels do.
 */
#ifndef EXQ_TESTING_H
#define EXQ_TESTING_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* exq_testing_starve -- while wait_rounds > 0, every exq_gemv, exq_gemv_multi,
 * exq_gemm, exq_paged_attn, exq_fp4_gemm, exq_fp4_gemv and exq_moe launch runs with its producer issuing no copies at all, and
 * every mbarrier wait of those kernels gives up after wait_rounds polling
 * rounds instead of the built-in bound. The consumers then wait for data that
 * never comes; their bounded waits run out, the kernel records
 * EXQ_ERR_TIMEOUT in the device error word (read it with
 * exq_get_last_device_error), frees what it holds (tensor memory) and
 * returns. No copy is in flight at any time, so nothing is left to drain.
 * Outputs of a starved call are unspecified; a starved exq_gemv, exq_fp4_gemv or exq_moe may
 * leave its workspace counters non-zero (zero them before the next call).
 * wait_rounds = 0 turns the hook off (the default). Host-side, process-wide,
 * thread-safe; it affects launches made after it returns. */
void exq_testing_starve(int32_t wait_rounds);

/* How the few-row product and the experts divide a call's units over CTAs, as
 * their kernels compute it: CTA cta (0 .. ctas) of ctas has the units from
 * exq_testing_first_unit(cta) up to that of cta + 1; exq_testing_unit_owner is
 * the CTA that has `unit`, 0 <= unit < n_units, 1 <= ctas <= n_units. -1 for
 * anything else. Host-side. */
int64_t exq_testing_first_unit(int32_t cta, int64_t n_units, int32_t ctas);
int32_t exq_testing_unit_owner(int64_t unit, int64_t n_units, int32_t ctas);

#ifdef __cplusplus
}
#endif

#endif /* EXQ_TESTING_H */
