// A launch that fails on the host returns ZC_ECUDA and leaves no error behind: launches that are checked by the runtime's last
// error come after it. Linked with a fake of the runtime, whose launches all fail (test_kv_launch.py). Prints what is wrong.
#include <cstdio>

#include "kv/kv_common.cuh"

static void nothing(int) {}

int main() {
    if (zc::kv::launch_early(nothing, dim3(1), 32, 0, nullptr, 7) != ZC_ECUDA) return std::puts("the launch did not fail"), 1;
    const cudaError_t left = cudaGetLastError();
    if (left != cudaSuccess) return std::printf("error %d is left behind\n", int(left)), 1;
    return 0;
}
