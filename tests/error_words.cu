// error_words.cu -- counts what the products' error words are given and what is read from them: a kernel
// sets bits now and then while two threads of the host read and clear.  Prints "set S taken T" for each word.
#include <atomic>
#include <cstdio>
#include <thread>

#include "experts_error.cu"

namespace {

__device__ int g_words[3];
__device__ int g_sets[3];

int* word(int i) {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_words) == cudaSuccess ? static_cast<int*>(p) + i : nullptr;
}

// Block i sets bit i of word i `times` times, 10 to 40 us apart, and counts the times that the word was clear.
__global__ void set_words(int times) {
    const int i = blockIdx.x;
    uint32_t r = 12345u + i;
    int sets = 0;
    for (int n = 0; n < times; ++n) {
        r = r * 1664525u + 1013904223u;
        __nanosleep(10000u + (r >> 8) % 30000u);
        if (atomicOr(&g_words[i], 1 << i) == 0) ++sets;
    }
    g_sets[i] = sets;
}

}  // namespace

namespace moe {
cudaError_t product_error_word(int** p) { return (*p = word(0)) ? cudaSuccess : cudaErrorUnknown; }
cudaError_t product_few_error_word(int** p) { return (*p = word(1)) ? cudaSuccess : cudaErrorUnknown; }
cudaError_t weight_grad_error_word(int** p) { return (*p = word(2)) ? cudaSuccess : cudaErrorUnknown; }
}  // namespace moe

int main() {
    cudaStream_t s[3];
    for (auto& t : s)
        if (cudaStreamCreateWithFlags(&t, cudaStreamNonBlocking) != cudaSuccess) return 2;
    std::atomic<int> taken[3] = {}, failed{0}, done{0};
    auto take = [&](cudaStream_t st) {
        int code = 0;
        if (moe::product_error(&code, st) != cudaSuccess) ++failed;
        for (int i = 0; i < 3; ++i) taken[i] += code >> i & 1;
    };
    take(s[1]);  // the first call loads what it needs
    set_words<<<3, 1, 0, s[0]>>>(4000);
    auto reader = [&](int i) {
        while (!done) take(s[i]);
    };
    std::thread a(reader, 1), b(reader, 2);
    const cudaError_t e = cudaStreamSynchronize(s[0]);
    done = 1;
    a.join();
    b.join();
    take(s[1]);
    int sets[3];
    if (e != cudaSuccess || failed || cudaMemcpyFromSymbol(sets, g_sets, sizeof(sets)) != cudaSuccess) return 3;
    for (int i = 0; i < 3; ++i) std::printf("set %d taken %d\n", sets[i], taken[i].load());
    return 0;
}
