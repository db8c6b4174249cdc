// mbar_pass (csrc/ssu_tc.cuh) on a barrier that nothing arrives at: it gives up, later waits do not
// wait, and a barrier that is arrived at lets the warp pass.  One CTA; prints how long the wait took.
#include <cstdio>

#include "ssu_tc.cuh"

__global__ void wait_kernel(unsigned long long *ns, unsigned *dead_at) {
    __shared__ unsigned long long bars[2];
    const unsigned never = smem_u32(&bars[0]), passed = smem_u32(&bars[1]);
    if (threadIdx.x == 0) {
        mbar_init(never, 1);
        mbar_init(passed, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_arrive(passed);
    }
    __syncthreads();
    unsigned dead = 0;
    mbar_pass(passed, 0, dead);
    dead_at[threadIdx.x] = dead;
    unsigned long long t0, t1, t2;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0)::"memory");
    mbar_pass(never, 0, dead);
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t1)::"memory");
    dead_at[blockDim.x + threadIdx.x] = dead;
    mbar_pass(never, 0, dead);
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t2)::"memory");
    if (threadIdx.x == 0) ns[0] = t1 - t0, ns[1] = t2 - t1;
}

int main() {
    unsigned long long *ns;
    unsigned *dead;
    if (cudaMallocManaged(&ns, 2 * sizeof *ns) != cudaSuccess ||
        cudaMallocManaged(&dead, 2 * 256 * sizeof *dead) != cudaSuccess)
        return 2;
    wait_kernel<<<1, 256>>>(ns, dead);
    if (cudaDeviceSynchronize() != cudaSuccess) return 3;
    for (int i = 0; i < 256; ++i)
        if (dead[i] != 0 || dead[256 + i] != 1) return 1;
    printf("%llu %llu\n", ns[0], ns[1]);
    return 0;
}
