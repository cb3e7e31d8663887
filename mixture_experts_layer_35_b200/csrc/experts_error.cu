// experts_error.cu -- the products' error words, one in each of their files, read and cleared.
#include <mutex>

#include "experts.cuh"

namespace moe {
namespace {

__device__ int g_taken;

// Each word is read and cleared in one step, so that a bit that a product on another stream sets
// meanwhile is in this call's answer or in the next one's.
__global__ void take_errors_kernel(int* a, int* b, int* c) {
    g_taken = atomicExch(a, 0) | atomicExch(b, 0) | atomicExch(c, 0);
}

}  // namespace

cudaError_t product_error(int* code, cudaStream_t s) {
    static std::mutex mu;  // g_taken is one call's at a time
    const std::lock_guard<std::mutex> lock(mu);
    *code = 0;
    int *a = nullptr, *b = nullptr, *c = nullptr;
    void* taken = nullptr;
    cudaError_t e = product_error_word(&a);
    if (e == cudaSuccess) e = product_few_error_word(&b);
    if (e == cudaSuccess) e = weight_grad_error_word(&c);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&taken, g_taken);
    if (e == cudaSuccess) e = launch_k(take_errors_kernel, dim3(1), dim3(1), 0, s, false, a, b, c);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, taken, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e;
}

}  // namespace moe
