// q4_stream_g128.cu -- the streaming 4-bit products for groups of 128.
#include "q4_stream.cuh"

namespace tq2 {

cudaError_t launch_q4_stream_g128(const Q4Stream& a, cudaStream_t st) { return q4_stream_run<128>(a, st); }

unsigned int read_clear_dev_error_q4_g128(cudaStream_t st) {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_dev_error, sizeof(v), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess) return 0;
    cudaMemcpyToSymbolAsync(g_dev_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
    cudaStreamSynchronize(st);
    return v;
}

}  // namespace tq2
