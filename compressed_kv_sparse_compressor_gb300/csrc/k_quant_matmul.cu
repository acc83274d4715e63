// Product of quantised rows with quantised weights:
//   out_g[i][j] = sum_b 2^(ea[i][b] + ew_g[j / 128][b]) sum_{k in block b} a[i][k] w_g[j][k]
// for 1 to 4 weight matrices over the same rows.
//
// 64 x 64 output tiles on the CUDA cores, K in slices of 16 (a slice lies in one
// block of 128): codes are converted and scaled as they enter shared memory, which
// is exact in float, and accumulated in float.
#include "ds4c_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace ds4c {

namespace {

constexpr int TILE = 64, KS = 16;

struct Group {
    const uint8_t *q, *scale;
    void *out;
    int64_t out_ld;
    int n;
};
struct Params {
    const uint8_t *a, *a_scale;
    int m, k, bf16_out;
    int64_t q_ld, scale_ld;
    int tile_start[5];
    int n_w;
    Group g[4];
};

__device__ __forceinline__ float e4m3(uint32_t code) {
    uint32_t h2;
    const uint16_t c = (uint16_t)code;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == 255 ? NAN : byte == 0 ? 0x1p-127f : __uint_as_float(byte << 23);
}

__global__ void __launch_bounds__(256) quant_matmul_kernel(Params p) {
    __shared__ float sa[KS][TILE + 1], sw[KS][TILE + 1];
    pdl_wait();
    pdl_launch_dependents();
    int g = 0;
    while (g + 1 < p.n_w && (int)blockIdx.y >= p.tile_start[g + 1]) g++;
    const Group G = p.g[g];
    const int n0 = ((int)blockIdx.y - p.tile_start[g]) * TILE;
    const int64_t m0 = (int64_t)blockIdx.x * TILE;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int lr = threadIdx.x / 4, lk = (threadIdx.x % 4) * 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < p.k; k0 += KS) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int k = k0 + lk + i;
            const int64_t m = m0 + lr;
            const int n = n0 + lr;
            float va = 0.f, vw = 0.f;
            if (k < p.k && m < p.m) va = e4m3(p.a[m * p.q_ld + k]) * scale_value(p.a_scale[m * p.scale_ld + k / 128]);
            if (k < p.k && n < G.n) vw = e4m3(G.q[n * p.q_ld + k]) * scale_value(G.scale[(n / 128) * p.scale_ld + k / 128]);
            sa[lk + i][lr] = va;
            sw[lk + i][lr] = vw;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KS; k++) {
            float a[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) a[i] = sa[k][ty + 16 * i], w[i] = sw[k][tx + 16 * i];
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = fmaf(a[i], w[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t m = m0 + ty + 16 * i;
        if (m >= p.m) continue;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int n = n0 + tx + 16 * j;
            if (n >= G.n) continue;
            if (p.bf16_out) static_cast<__nv_bfloat16 *>(G.out)[m * G.out_ld + n] = __float2bfloat16_rn(acc[i][j]);
            else static_cast<float *>(G.out)[m * G.out_ld + n] = acc[i][j];
        }
    }
}

}  // namespace

cudaError_t launch_quant_matmul(const QuantMatmulArgs &a, cudaStream_t s) {
    Params p{};
    p.a = a.a;
    p.a_scale = a.a_scale;
    p.m = a.m;
    p.k = a.k;
    p.bf16_out = a.out_dtype == DS4C_BF16;
    p.q_ld = (int64_t)quant_row_bytes((uint32_t)a.k);
    p.scale_ld = (int64_t)quant_scale_bytes((uint32_t)a.k);
    p.n_w = a.n_w;
    int start = 0;
    for (int g = 0; g < a.n_w; g++) {
        p.tile_start[g] = start;
        p.g[g] = Group{a.w[g].q, a.w[g].scale, a.w[g].out, (int64_t)a.w[g].out_ld, (int)a.w[g].n};
        start += ((int)a.w[g].n + TILE - 1) / TILE;
    }
    p.tile_start[a.n_w] = start;
    return launch_pdl(quant_matmul_kernel, dim3((a.m + TILE - 1) / TILE, start), dim3(256), 0, s, p);
}

}  // namespace ds4c
