// The rows that an expert takes, as the sort computes them in 32 bits, under
// UndefinedBehaviorSanitizer: for every alignment, the largest slot counts that
// a plan accepts, all of them of one expert or shared between experts.  The
// last row of the last expert must be max_rows or less and every start must be
// what 64 bits give.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "index_plan.hpp"

namespace {

bool accepted(int64_t T, int E, int align, int64_t &rows)
{
    basp_expert_plan *p = basp_expert_plan_create(T, 1, E, 1, align, 4, BASP_BF16, BASP_FP32);
    if (!p)
        return false;
    rows = p->max_rows;
    basp_expert_plan_destroy(p);
    return true;
}

// The starts of experts with these counts, in 32 bits as on the device.
bool starts_fit(const std::vector<int64_t> &counts, int align, int64_t rows)
{
    int at = 0;
    int64_t want = 0;
    for (const int64_t n : counts) {
        at += basp::padded_count(int(n), align);
        want += (n + align - 1) / align * align;
        if (at != want)
            return false;
    }
    return want <= rows;
}

}  // namespace

int main()
{
    long checked = 0;
    for (const int align : {1, 2, 3, 5, 7, 128, 1000, 4095, 32768, 50000, 65535, 65536})
        for (const int E : {1, 2, 3, 8, 1024}) {
            // the largest accepted number of slots
            int64_t T = 0, rows = 0;
            for (int64_t step = int64_t{1} << 30; step; step /= 2)
                if (accepted(T + step, E, align, rows))
                    T += step;
            if (T < (int64_t{1} << 30))
                return std::printf("FAIL limit\n"), 1;
            for (const int64_t less : {0, 1, 2, 998, 65536}) {
                const int64_t n = T - less;
                if (!accepted(n, E, align, rows))
                    return std::printf("FAIL accepted\n"), 1;
                std::vector<int64_t> all(E, 0), ones(E, 1), even(E, n / E);
                all[E - 1] = n;
                ones[0] = n - (E - 1);
                even[0] += n % E;
                for (const auto &c : {all, ones, even}) {
                    if (!starts_fit(c, align, rows))
                        return std::printf("FAIL %lld slots, %d experts, align %d\n", (long long)n, E, align), 1;
                    ++checked;
                }
            }
        }
    std::printf("OK %ld\n", checked);
    return 0;
}
