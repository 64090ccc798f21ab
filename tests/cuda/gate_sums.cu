// Test probe for the sums of log-gates (csrc/gate_scan.cuh): what a gate counts,
// the power of two of a sum, and sums over many chunks.
#include "gate_scan.cuh"

using namespace la;

__global__ void bits_kernel(const float* g, long long* out, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) out[i] = gate_bits(g[i]);
}
__global__ void pow2_kernel(const long long* b, float* out, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) out[i] = gate_pow2(b[i]);
}
// The sum of `times` chunks of b, and its power of two.
__global__ void add_kernel(const long long* b, const int* times, long long* sum, float* out, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    long long s = 0;
    for (int t = 0; t < times[i]; ++t) s = gate_add(s, b[i]);
    sum[i] = s;
    out[i] = gate_pow2(s);
}

extern "C" int gate_bits_probe(const float* g, long long* out, int n) {
    bits_kernel<<<(n + 255) / 256, 256>>>(g, out, n);
    return (int)cudaGetLastError();
}
extern "C" int gate_pow2_probe(const long long* b, float* out, int n) {
    pow2_kernel<<<(n + 255) / 256, 256>>>(b, out, n);
    return (int)cudaGetLastError();
}
extern "C" int gate_add_probe(const long long* b, const int* times, long long* sum, float* out, int n) {
    add_kernel<<<(n + 255) / 256, 256>>>(b, times, sum, out, n);
    return (int)cudaGetLastError();
}
