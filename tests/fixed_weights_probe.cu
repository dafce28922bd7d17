// The fixed-point weights of filter_math.cuh, evaluated on arrays for
// test_gpu_fixed_weights.py, which compiles this file.
#include "filter_math.cuh"

using namespace pstat;

__global__ void weights(const float* z, const float* M, const float* t, int k, unsigned long long* w,
                        int n) {
    __shared__ float2 table[64];
    if (threadIdx.x < 64) table[threadIdx.x] = kExp2Table[threadIdx.x];
    __syncthreads();
    const int i = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    if (i < n) w[i] = fixed_weight(z[i], M[i], temp_scale(t[i]), k, table);
}

extern "C" __attribute__((visibility("default"))) int fixed_weights_probe(const float* z, const float* M,
                                                                        const float* t, int k,
                                                                        unsigned long long* w, int n) {
    if (n > 0) weights<<<(n + 255) / 256, 256>>>(z, M, t, k, w, n);
    const cudaError_t e = cudaDeviceSynchronize();
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}
