// How the column sums' kernel finds a group's partial rows (csrc/gemm16_slices.h), lane by lane, on the CPU: prints
// "from to" for "M height most groups" and the offsets, one line a group.
#include <cstdio>
#include <vector>

#include "gemm16_slices.h"

int main()
{
    int M, height, groups;
    long long most;
    while (std::scanf("%d %d %lld %d", &M, &height, &most, &groups) == 4) {
        std::vector<int> offsets(groups + 1);
        for (int &o : offsets)
            if (std::scanf("%d", &o) != 1) return 1;
        for (int e = 0; e < groups; ++e) {
            long long before = 0;
            for (int lane = 0; lane < 32; ++lane) before += fgemm::h16::slices_before(offsets.data(), lane, 32, e, M, height);
            const fgemm::h16::PartialRows rows =
                fgemm::h16::inside(before, before + fgemm::h16::slices_of(offsets.data(), e, M, height), most);
            std::printf("%lld %lld\n", rows.from, rows.to);
        }
    }
    return 0;
}
