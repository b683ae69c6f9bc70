// The host code of the index-driven re-layouts under AddressSanitizer and
// UndefinedBehaviorSanitizer: plans at and beyond every limit, the place of
// every token, and the sizes of the launches that write zeros.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "index_plan.hpp"

int main()
{
    const int64_t big[] = {-1, 0, 1, 2, 255, 4096, 70000, (int64_t{1} << 29) - 1, int64_t{1} << 29, (int64_t{1} << 30) - 1,
                           int64_t{1} << 30, (int64_t{1} << 31) - 2, (int64_t{1} << 31) - 1, int64_t{1} << 40,
                           int64_t{1} << 62, INT64_MAX};
    const int small[] = {-1, 0, 1, 2, 9, 1024, 1025, 65536, 65537, INT32_MAX};
    long made = 0;
    for (const int64_t T : big)
        for (const int64_t D : big) {
            for (const int K : small)
                for (const int E : small)
                    for (const int align : {1, 3, 65536})
                        for (const basp_dtype t : {BASP_BF16, BASP_FP32, BASP_INT32}) {
                            basp_expert_plan *p = basp_expert_plan_create(T, K, E, D, align, 8, t, BASP_FP32);
                            if (!p)
                                continue;
                            basp_expert_info i;
                            if (basp_expert_plan_query(p, &i) != BASP_OK || i.max_rows % align != 0 ||
                                i.max_rows < i.slots / align * align || i.workspace_bytes < 0)
                                return std::printf("FAIL expert\n"), 1;
                            basp_expert_plan_destroy(p);
                            ++made;
                        }
            for (const int64_t V : big)
                for (const basp_dtype t : {BASP_FP16, BASP_FP32}) {
                    basp_embed_plan *p = basp_embed_plan_create(nullptr, T, V, D, V > 0 ? V - 1 : -1, 4, t, BASP_FP32);
                    if (!p)
                        continue;
                    basp_embed_info i;
                    if (basp_embed_plan_query(p, &i) != BASP_OK || i.workspace_bytes < (T ? 4 * V : 0))
                        return std::printf("FAIL embed\n"), 1;
                    const basp::ZeroPieces z = basp::zero_pieces(0, V, D * 4, 4);
                    if (z.groups == 0 || z.stride == 0 || z.groups % z.stride != 0)
                        return std::printf("FAIL zeros\n"), 1;
                    basp_embed_plan_destroy(p);
                    ++made;
                }
        }
    for (const int G : {1, 2, 4}) {
        basp_plan *layout = basp_plan_create_groups(8, 4, 24, 8, 8, 16, BASP_BF16, G, BASP_LAYOUT_HEAD_MAJOR);
        basp_embed_plan *p = basp_embed_plan_create(layout, 96, 10, 16, -1, 8, BASP_BF16, BASP_BF16);
        std::vector<char> seen(96, 0);
        for (uint32_t t = 0; t < 96; ++t)
            ++seen.at(basp::seq_row(p->order, t));
        for (const char c : seen)
            if (c != 1)
                return std::printf("FAIL order\n"), 1;
        basp_embed_plan_destroy(p);
        basp_plan_destroy(layout);
    }
    std::printf("OK %ld plans\n", made);
    return 0;
}
