// Host-side check of the operators around the core under AddressSanitizer and
// UBSan (built host-only by tests/test_layer_sanitizers.py; no GPU is touched):
// every call fails an argument check or is empty, and the workspace queries
// run on extreme shapes, where UBSan reports a signed overflow.
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
    uint8_t *Q = reinterpret_cast<uint8_t *>(0x10000);
    int32_t *I = reinterpret_cast<int32_t *>(0x10000);
    const size_t BIG = (size_t)1 << 40;
    const int64_t huge[] = {0,       1,         2,         7,         64,        4096, (int64_t)1 << 20, (int64_t)1 << 24, INT32_MAX,
                            (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, -1,   INT64_MIN};
    for (int64_t a : huge)
        for (int64_t b : huge)
            for (int64_t c : huge) {
                for (ssd_dtype t : {SSD_F32, SSD_BF16}) {
                    (void)ssd_linear_workspace_bytes(a, b, c, t);
                    (void)ssd_linear_bwd_workspace_bytes(a, b, c, SSD_ACT_SILU, t);
                    (void)ssd_rms_norm_bwd_workspace_bytes(a, b, c, t, t);
                    // nothing of these may pass: NULL operands, or no rows
                    const ssd_status n = ssd_rms_norm(nullptr, nullptr, nullptr, 1e-5f, nullptr, nullptr, nullptr, a, b, c, t, t, nullptr);
                    const ssd_status l = ssd_linear(nullptr, nullptr, nullptr, 0, nullptr, nullptr, nullptr, a, b, c, t, nullptr, 0, nullptr);
                    if (a != 0 && (n == SSD_OK || l == SSD_OK)) ++failures;
                }
                (void)ssd_linear_mx_workspace_bytes(a, b, c);
                (void)ssd_beam_select_workspace_bytes(a, b, c);
                if (a != 0) {
                    EXPECT(ssd_mx_quantize(nullptr, Q, Q, a, b, SSD_BF16, nullptr), SSD_ERR_NULL);
                    EXPECT(ssd_step_beam(F, nullptr, I, 1, nullptr, nullptr, P, nullptr, nullptr, P, nullptr, 0, F, P, P, F, nullptr, P, a, 8, 64, 128, 1, SSD_BF16, nullptr), SSD_ERR_NULL);
                }
            }
    for (int64_t r : huge)  // the states' sizes, before their overlap is looked at
        (void)ssd_step_beam(F, F, I, r, nullptr, nullptr, nullptr, nullptr, nullptr, P, nullptr, 0, F, P, P, F, nullptr, P, 65536, 65536, 4096, 256, 1, SSD_BF16, nullptr);
    EXPECT(ssd_step_beam(F, F, I, 4, nullptr, nullptr, P, nullptr, nullptr, P, nullptr, 0, F, P, P, F, nullptr, P, 4, 8, 64, 128, 1, SSD_BF16, nullptr), SSD_ERR_UNSUPPORTED);
    EXPECT(ssd_beam_select(P, F, Q, -1, F, I, I, Q, 2, 4, 100, SSD_BF16, P, BIG, nullptr), SSD_ERR_SHAPE);
    EXPECT(ssd_linear(P, P, nullptr, 0, nullptr, P, nullptr, 100, 63, 64, SSD_BF16, P, 16, nullptr), SSD_ERR_WORKSPACE);
    EXPECT(ssd_linear_bwd(P, P, P, 1, nullptr, P, P, F, 100, 64, 64, SSD_BF16, P, BIG, nullptr), SSD_ERR_NULL);
    EXPECT(ssd_linear_mx(Q, Q, Q, Q, nullptr, 0, nullptr, P, 100, 40, 64, P, BIG, nullptr), SSD_ERR_SHAPE);
    if (failures) return 1;
    printf("layer abi checks passed\n");
    return 0;
}
