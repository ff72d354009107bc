// orth_places.cpp -- plan_memory.cpp's runtime with the orthogonalised updates' launches: for every shape, the places of split
// tiles are apart from those of the other matrices' tiles, in whichever kinds of product these are, and inside the workspace.
#define main other_main
#include "plan_memory.cpp"
#undef main

namespace cbd {
int logp_most_items(int sms) { return sms * 2; }
static int pairs = 76;
int orth_pairs(int) { return pairs; }
static OrthParams seen;
cudaError_t launch_orth_prep(const OrthPrepParams &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_orth_steps(const OrthParams &p, bool, int, cudaStream_t) { return seen = p, cudaSuccess; }
}  // namespace cbd

extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }

static int shapes = 0, splitting = 0;

// 0 if the places of this shape are in order
static int check(int64_t batch, int64_t rows, int64_t cols) {
    using namespace cbd;
    const float coef[3] = {1.5f, -0.5f, 0.f};
    const conv_bwd_orth_desc d = {batch, rows, cols, CONV_BWD_F32, 1, coef};
    conv_bwd_orth_plan plan;
    if (conv_bwd_orth_create(&d, &plan) != CONV_BWD_OK) return printf("create\n"), 2;
    if (conv_bwd_orth_apply(plan, (void *)((uintptr_t)1 << 40), 0, 0, (void *)((uintptr_t)1 << 41), 0, 0, nullptr) != CONV_BWD_OK) return printf("apply\n"), 2;
    const OrthParams &p = seen;
    ++shapes;
    int kinds = 0;
    const long counters = ((const char *)p.parts - (const char *)p.arrived) / 64, room = ((const char *)p.done - (const char *)p.parts) / (256 * 128 * 4);
    for (int k = 0; k < 3; ++k) {
        if (p.splits[k] == 1) continue;
        ++kinds;
        const int tiles = k == kOrthProduct ? p.tiles_all : p.tiles_sym;
        if (orth_counter_place(p, p.batch - 1, tiles - 1) + 1 > counters || orth_piece_place(p, p.batch - 1, tiles - 1, p.splits[k]) + p.splits[k] > room)
            return printf("%d x %d x %d: places of kind %d beyond the workspace\n", p.batch, p.rows, p.cols, k), 1;
        for (int j = 0; j < 3; ++j) {  // matrix 0 in a product of this kind, matrix 1 in one of any
            if (p.splits[j] == 1 || p.batch == 1) continue;
            if (orth_counter_place(p, 0, tiles - 1) >= orth_counter_place(p, 1, 0) || orth_piece_place(p, 0, tiles - 1, p.splits[k]) + p.splits[k] > orth_piece_place(p, 1, 0, p.splits[j]))
                return printf("%d x %d x %d: tiles of kinds %d and %d share a place\n", p.batch, p.rows, p.cols, k, j), 1;
        }
    }
    splitting += kinds > 0;
    return conv_bwd_orth_destroy(plan);
}

int main() {
    const int64_t sides[] = {300, 513, 641, 705, 740, 768, 769, 1000};
    for (int pairs : {70, 76}) {
        cbd::pairs = pairs;
        for (int64_t batch : {1, 2, 3})
            for (int64_t rows : sides)
                for (int64_t cols : sides)
                    if ((rows <= cols || batch == 2) && batch * rows * cols < 2000000)
                        if (int bad = check(batch, rows, cols)) return bad;
    }
    printf("%d shapes, %d with split contractions\n", shapes, splitting);
    return splitting > 50 ? 0 : 1;
}
