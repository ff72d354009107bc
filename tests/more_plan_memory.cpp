// more_plan_memory.cpp -- plan_memory.cpp's runtime with the plans of the token log-probabilities and the orthogonalised
// updates: create leaves nothing queued, the counters are zeros, a run with another device current is refused.
#define main other_main
#include "plan_memory.cpp"
#undef main

namespace cbd {
int logp_most_items(int sms) { return sms * 2; }
int orth_pairs(int sms) { return sms / 2; }
}  // namespace cbd

extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }

int main(int argc, char **argv) {
    const std::string what = argc > 1 ? argv[1] : "";
    conv_bwd_status st = CONV_BWD_ERR_INVALID_ARG;
    int elsewhere = CONV_BWD_ERR_INVALID_ARG;
    size_t zeros = 64;
    const float coef[3] = {1.5f, -0.5f, 0.f};
    if (what == "logp") {
        const conv_bwd_logp_desc d = {50000, CONV_BWD_F32, 8, 1.f};
        conv_bwd_logp_plan p;
        st = conv_bwd_logp_create(&d, &p);
        zeros = 64 + 304 * 4;
        device = 1;
        if (!st) elsewhere = conv_bwd_logp_forward(p, 4, at(1), 0, (const int32_t *)at(2), (float *)at(3), (float *)at(4), (float *)at(5), (float *)at(6), (int32_t *)at(7), nullptr);
    } else {
        // in shared memory; on pairs of SMs, with contractions in pieces and whole
        const conv_bwd_orth_desc d = {what == "orth batch" ? 90 : 1, what == "orth small" ? 100 : 300, what == "orth small" ? 131 : what == "orth" ? 4096 : 290, CONV_BWD_F32, 1, coef};
        conv_bwd_orth_plan p;
        st = conv_bwd_orth_create(&d, &p);
        device = 1;
        if (!st) elsewhere = conv_bwd_orth_apply(p, at(100), 0, 0, at(200), 0, 0, nullptr);
        if (!st && elsewhere == CONV_BWD_ERR_INVALID_ARG)
            elsewhere = conv_bwd_orth_update(p, (float *)at(100), at(200), 0, 0, (float *)at(300), at(400), 0.1f, 0.9f, 1, 0.f, 1.f, nullptr);
    }
    if (st != CONV_BWD_OK) return printf("create: status %d\n", (int)st), 2;
    if (int n = pending()) return printf("%d of the plan's writes still queued when create returned\n", n), 1;
    if (written < 1 || held.size() != 1 || held.begin()->second < zeros) return printf("unexpected buffers\n"), 2;
    if (elsewhere != CONV_BWD_ERR_INVALID_ARG) return printf("run with another device current: status %d\n", elsewhere), 1;
    const uint8_t *m = (const uint8_t *)held.begin()->first;
    for (size_t i = 0; i < zeros; ++i)
        if (m[i]) return printf("byte %zu of the counters is %d\n", i, m[i]), 1;
    return 0;
}
