// Prints which kernel an integer product takes for each "M N" line of its input.
#include <cstdio>

#include "../../mixed_precision_weight_dq_amd/csrc/product_plan.hpp"

int main()
{
    std::printf("%d\n", (int)dq::I8Kernel::kCount);
    long long M, N;
    while (std::scanf("%lld %lld", &M, &N) == 2) std::printf("%d\n", (int)dq::i8_kernel(M, N));
    return 0;
}
