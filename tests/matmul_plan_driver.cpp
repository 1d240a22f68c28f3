// How the products' calls on standard input ("weights mx rotate bf16 rows cols tokens") are cut into workgroups, a line for
// each: kernel, prepared, parts, rows of x and of the weight of a workgroup, waves that share the long axis, steps in a chunk of x,
// splits, steps of a split, bytes of LDS and of the workspace, refused.
#include <cstdio>

#include "fp4q_matmul_plan.h"

int main()
{
    long long w, mx, rotate, bf16, n, k, m;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld", &w, &mx, &rotate, &bf16, &n, &k, &m) == 7) {
        fp4q::MatmulArgs a{};
        a.weights = (int)w;
        a.mx = (int)mx;
        a.rotate = rotate ? (mx ? 32 : 16) : 0;
        a.bf16 = bf16 != 0;
        a.n = n;
        a.k = k;
        a.m = m;
        const fp4q::MatmulPlan p = fp4q::plan_of(a);
        std::printf("%s %d %d %d %d %d %d %d %d %zu %zu %d\n", p.many ? "many" : "few", p.prepared, p.parts, p.tokens, p.rows, p.waves_k,
                    p.chunk_steps, p.splits, p.split_steps, p.lds, p.workspace, p.refused);
    }
    return 0;
}
