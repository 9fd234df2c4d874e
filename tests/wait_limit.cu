// Runs the waits of wc_wait.cuh by themselves.
//   wait_limit host        : the limit's arithmetic on sequences of looks at a clock
//   wait_limit gpu         : a wait that is answered and one that nothing answers
// Prints one "name value" per line.
#include <stdio.h>
#include <string.h>

#include "../weight_communication_gb300/csrc/wc_wait.cuh"

// Looks `step` ns apart until the limit is spent, with `jump` ns added once after
// `jump_at` of them; the nanoseconds of the looks, jump excluded.
static unsigned long long run_out(unsigned long long start, unsigned long long step, long jump_at,
                                  unsigned long long jump) {
    wc::WaitLimit limit{uint32_t(start)};
    unsigned long long now = start, ran = 0;
    for (long i = 1; i < 100000000; ++i) {
        now += step;
        ran += step;
        if (i == jump_at) now += jump;
        if (limit.spent(uint32_t(now))) return ran;
    }
    return 0;
}

struct Result {
    int answered, lost;
    unsigned int count;
    unsigned long long ns;
};

__global__ void waits(Result *r, unsigned int *count) {
    __shared__ uint64_t bars[2];
    if (threadIdx.x == 0) {
        wc::mbar_init(wc::smem_of(&bars[0]), 1);
        wc::mbar_init(wc::smem_of(&bars[1]), 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) wc::mbar_arrive(wc::smem_of(&bars[0]));
    __syncwarp();
    const bool answered = wc::mbar_wait(wc::smem_of(&bars[0]), 0, count);
    unsigned long long begin, end;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(begin));
    const bool lost = !wc::mbar_wait(wc::smem_of(&bars[1]), 0, count);
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(end));
    if (threadIdx.x == 0) {
        r->answered = answered;
        r->lost = lost;
        r->ns = end - begin;
    }
}

int main(int argc, char **argv) {
    if (argc > 1 && strcmp(argv[1], "host") == 0) {
        printf("steady %llu\n", run_out(0, 1000, 0, 0));
        printf("wrapping %llu\n", run_out(4294000000ull, 1000, 0, 0));
        // one hour's suspension in the middle, and 2.1 s of it
        printf("suspended_1h %llu\n", run_out(7, 1000, 1000000, 3600ull * 1000000000ull));
        printf("suspended_2s %llu\n", run_out(7, 1000, 1000000, 2100000000ull));
        return 0;
    }
    unsigned int *count;
    Result *r, h;
    if (cudaMalloc(&count, sizeof(*count)) != cudaSuccess || cudaMalloc(&r, sizeof(*r)) != cudaSuccess ||
        cudaMemset(count, 0, sizeof(*count)) != cudaSuccess)
        return 2;
    waits<<<1, 32>>>(r, count);
    if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return 3;
    if (cudaMemcpy(&h, r, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemcpy(&h.count, count, sizeof(h.count), cudaMemcpyDeviceToHost) != cudaSuccess)
        return 4;
    printf("answered %d\nlost %d\ncount %u\nns %llu\n", h.answered, h.lost, h.count, h.ns);
    return 0;
}
