// Host-side check of the gated recurrence, the embedding, the logits' processing
// and the integer projections under AddressSanitizer and UBSan (built host-only by
// tests/test_decoder_sanitizers.py; no GPU is touched): every call fails an argument
// check or is empty, and the workspace queries run on extreme shapes, where UBSan
// reports a signed overflow.
#include <stdint.h>
#include <stdio.h>

#include "ssd.h"

static int failures = 0;
#define EXPECT(call, want)                                                                            \
    do {                                                                                              \
        const int got_ = (int)(call);                                                                 \
        if (got_ != (int)(want)) {                                                                    \
            fprintf(stderr, "line %d: %s -> %d, expected %d\n", __LINE__, #call, got_, (int)(want)); \
            ++failures;                                                                               \
        }                                                                                             \
    } while (0)

int main() {
    void *P = reinterpret_cast<void *>(0x10000);
    float *F = reinterpret_cast<float *>(0x10000);
    int8_t *Q = reinterpret_cast<int8_t *>(0x10000);
    int32_t *I = reinterpret_cast<int32_t *>(0x10000);
    const int64_t huge[] = {0,       1,         2,         7,         64,        4096, (int64_t)1 << 20, (int64_t)1 << 22, INT32_MAX,
                            (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, -1,   INT64_MIN};
    for (int64_t a : huge)
        for (int64_t b : huge)
            for (int64_t c : huge) {
                for (ssd_dtype t : {SSD_F32, SSD_BF16}) {
                    (void)ssd_gated_scan_fwd_workspace_bytes(a, b, c, t);
                    (void)ssd_gated_scan_bwd_workspace_bytes(a, b, c, SSD_DECAY_RATE, t);
                    // nothing of these may pass: no workspace or no operands, but for empty problems (b or a is 0)
                    const ssd_status f = ssd_gated_scan_fwd(nullptr, c, nullptr, b, nullptr, 0, SSD_DECAY_LOG, nullptr, nullptr, nullptr, nullptr,
                                                            nullptr, nullptr, a, b, c, t, nullptr, 0, nullptr);
                    if (a != 0 && b != 0 && f == SSD_OK) ++failures;
                    const ssd_status g = ssd_gated_scan_bwd(nullptr, P, c, P, c, nullptr, 0, SSD_DECAY_SIGMOID, nullptr, nullptr, F, nullptr, P, P,
                                                            nullptr, nullptr, nullptr, a, b, c, t, P, SIZE_MAX, nullptr);
                    if (a != 0 && b != 0 && g == SSD_OK) ++failures;
                }
                (void)ssd_embedding_bwd_workspace_bytes(a, b, c);
                (void)ssd_linear_int_workspace_bytes(a, b, c);
                if (a != 0) {
                    EXPECT(ssd_embedding(I, nullptr, 1.f, P, a, b, c, SSD_BF16, SSD_F32, nullptr), SSD_ERR_NULL);
                    EXPECT(ssd_int_quantize(nullptr, Q, F, a, b, SSD_F32, nullptr), SSD_ERR_NULL);
                    EXPECT(ssd_linear_int(Q, F, Q, F, nullptr, 0, nullptr, nullptr, a, b, c, SSD_BF16, nullptr, 0, nullptr), SSD_ERR_NULL);
                    EXPECT(ssd_logits_process(P, nullptr, I, b, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, a, c, SSD_F32, nullptr), SSD_ERR_NULL);
                }
                // sizes before overlaps are looked at: the output is an input, so none of these passes
                const ssd_status s = ssd_gated_step(F, F, I, b, P, c, P, c, P, c, SSD_DECAY_LOG, nullptr, P, a, c, SSD_F32, nullptr);
                if (a != 0 && s == SSD_OK) ++failures;
                const ssd_status l = ssd_logits_process(P, P, I, b, I, I, F, F, F, F, 1, I, 1, a, c, SSD_BF16, nullptr);
                if (a != 0 && l == SSD_OK) ++failures;
                const ssd_status e = ssd_embedding(I, P, 1.f, P, a, b, c, SSD_F32, SSD_F32, nullptr);
                if (a != 0 && e == SSD_OK) ++failures;
            }
    EXPECT(ssd_embedding_bwd(P, I, 1.f, P, 0, 100, 50, 64, SSD_BF16, SSD_F32, nullptr, 0, nullptr), SSD_ERR_WORKSPACE);
    EXPECT(ssd_gated_scan_fwd(P, 64, P, 64, nullptr, 0, SSD_DECAY_LOG, nullptr, nullptr, nullptr, P, nullptr, nullptr, 1, 300, 64, SSD_F32, nullptr, 0, nullptr), SSD_ERR_WORKSPACE);
    EXPECT(ssd_linear_int(Q, F, Q, F, nullptr, 0, nullptr, P, 100, 40, 64, SSD_BF16, nullptr, 0, nullptr), SSD_ERR_SHAPE);
    if (failures) return 1;
    printf("decoder abi checks passed\n");
    return 0;
}
