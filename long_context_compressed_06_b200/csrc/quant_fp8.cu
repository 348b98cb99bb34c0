// quant_fp8.cu -- FP8 KV-cache quantisation (csa_quantize_fp8_kv).
//
// "DeepSeek-V4-Pro - Model techniques map", list "inference quantization":
// the KV cache is quantised to FP8.  The pages give no format; the one used
// here: e4m3 codes with one power-of-two scale per 128 channels of a row,
// stored as a UE8M0 byte e (s = 2^(e - 127)); s is the smallest power of two
// with absmax / s <= 448 (the largest finite e4m3 magnitude), its exponent k
// kept in [-124, 119] so that every code times s is a finite bf16 number; the
// codes are round-to-nearest-even with saturation, a zero magnitude stored as
// +0, and an all-zero block has e = 127.
//
// A thread owns 8 consecutive elements; the 16 threads of a 128-element block
// are 16 consecutive lanes and reduce its absmax with shuffles.  The op reads
// 2 bytes and writes 1 + 1/128 bytes per element: HBM bound.
#include "common.cuh"
#include "kernels.h"
#include "quant_fp8.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) quantize_fp8_kv_kernel(const uint16_t *__restrict__ x, long long n8,
                                                                   uint8_t *__restrict__ codes,
                                                                   uint8_t *__restrict__ exps) {
    const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;  // unit of 8 elements
    const bool active = t < n8;  // n8 is a multiple of 16: a block's 16 lanes agree
    float f[8];
    if (active) {
        unpack8(ldg_stream(x + t * 8), f);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = 0.f;
    }
    int k;
    const uint2 w = quantize_fp8_unit(f, k);
    if (active) {
        *reinterpret_cast<uint2 *>(codes + t * 8) = w;
        if ((t & 15) == 0) exps[t >> 4] = (uint8_t)(k + 127);
    }
}

}  // namespace

int launch_quantize_fp8_kv(const uint16_t *x, long long rows, int d, uint8_t *codes, uint8_t *exps,
                           cudaStream_t st) {
    const long long n8 = rows * (d / 8);
    if (n8 == 0) return CSA_OK;
    const long long blocks = (n8 + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return CSA_ERR_UNSUPPORTED;
    quantize_fp8_kv_kernel<<<(unsigned)blocks, kThreads, 0, st>>>(x, n8, codes, exps);
    return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace csa
