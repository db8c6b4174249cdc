// Host check of sees_to (ssu_attend.cuh): the requests without visible keys are looked for again by
// just the CTAs that have one, whatever the numbers of requests, threads and CTAs.
// Prints "ok" or the first counterexample.
#include <cstdio>

#include "ssu_attend.cuh"

int main() {
    for (unsigned ctas : {1u, 3u, 152u, 160u})
        for (int threads : {128, 256})
            for (long long requests : {1, 2, 127, 128, 129, 255, 256, 257, 300, 1000})
                for (int every : {0, 1, 7, 150}) {  // request k * every has no places; 0: none
                    auto places = [&](long long b) -> unsigned {  // as the kernel counts them
                        return b < requests && !(every && b % every == 0) ? 2 : 0;
                    };
                    for (unsigned cta = 0; cta < ctas; ++cta) {
                        bool asked = false, has = false;
                        for (long long b0 = 0; b0 == 0 || b0 < requests; b0 += threads)
                            for (int tid = 0; tid < threads; ++tid)
                                asked |= sees_to(b0 + tid, requests, places(b0 + tid), cta, ctas);
                        for (long long b = cta; b < requests; b += ctas) has |= !places(b);
                        if (asked != has) {
                            printf("FAIL %lld requests, %d threads, cta %u of %u: %d for %d\n",
                                   requests, threads, cta, ctas, asked, has);
                            return 1;
                        }
                    }
                }
    printf("ok\n");
    return 0;
}
