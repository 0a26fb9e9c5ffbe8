// q4_stream_g128.cu -- the streaming 4-bit products for groups of 128.
#include "q4_stream.cuh"

namespace tq2 {

cudaError_t launch_q4_stream_g128(const Q4Stream& a, cudaStream_t st) { return q4_stream_run<128>(a, st); }

unsigned int read_clear_dev_error_q4_g128(cudaStream_t st) { return read_clear_record(st); }

}  // namespace tq2
