/*
 * w4a16_testing.h - test hooks of the W4A16 library (not for production use).
 *
 * They exist so that a test can drive the failure path of the device-side
 * bounded waits (a wait that expires reports W4_ERR_TIMEOUT through
 * w4a16_device_status and the kernel returns) without faulting or hanging a
 * GPU, and can see on a host without a GPU what a call would launch.  Status
 * codes are those of w4a16.h.
 */
#ifndef W4A16_TESTING_H
#define W4A16_TESTING_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * w4a16_testing_set_seq_wait - settings of the completion-counter waits of
 * w4_gemv_seq launches issued after this call (process-wide).
 *   wait_ns      limit of each counter wait in nanoseconds, at most 2 s;
 *                0 restores the default of 2 s.
 *   target_bump  added to every counter target.  0 is normal operation; any
 *                other value makes every counter wait unmeetable (no CTA can
 *                pass the first one, so the count never grows), so each waits
 *                out its limit, records the expiry (w4a16_device_status then
 *                returns W4_ERR_TIMEOUT) and the launch finishes without valid
 *                results.  Call with (0, 0) to restore normal operation.
 * Returns W4A16_OK, or W4_ERR_SHAPE if wait_ns exceeds 2 s.  Not synchronised
 * with w4_gemv_seq calls on other host threads.
 */
W4A16_API int w4a16_testing_set_seq_wait(unsigned long long wait_ns, unsigned target_bump);

/*
 * w4a16_testing_lm_head_plan - what lm_head_argmax_topk(_rules) launches for
 * these sizes on a GPU of `sms` SMs.  Makes no CUDA call; of the rules only which
 * parts are there counts.  Returns W4A16_OK, or the code with which the call
 * would refuse the sizes.
 */
typedef struct {
    int32_t blocks;      /* grid */
    int32_t stages;      /* of the ring of weights of a block, */
    int32_t teams;       /* whose stages are this many teams' in turn */
    int32_t stage_bytes;
    int32_t smem;        /* bytes of shared memory of a block */
} w4a16_testing_lm_head;
W4A16_API int w4a16_testing_lm_head_plan(int M, int N, int K, int group, int symmetric, int k,
                                         const w4_logit_rules *rules, int sms, w4a16_testing_lm_head *out);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_TESTING_H */
