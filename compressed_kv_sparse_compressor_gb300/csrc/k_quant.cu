// RMSNorm with the residual's addition and an E4M3 output, and the quantisation
// of weights in 128 x 128 blocks: the producers of the 8-bit projections.
//
// Per row of d values:
//   h = T(x + residual);  rstd = float((sum h^2 / d + eps)^-1/2);
//   y = (h * rstd) * gain;  per block of 128: e = min { e : max |y| <= 448 * 2^e },
//   code = E4M3(y * 2^-e), scale byte e + 127.
// Both kernels read each input once, hold it in registers between the statistic
// and the codes, and write each output once: HBM bounds them.
#include "ds4c_internal.cuh"

#include <cuda_bf16.h>

namespace ds4c {

namespace {

// a + b rounded, and the error of that rounding, itself a float (Knuth, The Art of
// Computer Programming vol. 2, 4.2.2, theorem B).
__device__ __forceinline__ float add_error(float a, float b, float &err) {
    const float t = __fadd_rn(a, b);
    const float bv = __fsub_rn(t, a);
    err = __fadd_rn(__fsub_rn(a, __fsub_rn(t, bv)), __fsub_rn(b, bv));
    return t;
}
// s + c holds a sum to about twice float's precision: s rounded, c what the roundings dropped.
__device__ __forceinline__ void add_exact(float &s, float &c, float v) {
    float err;
    s = add_error(s, v, err);
    c = __fadd_rn(c, err);
}

// Sum of (s, c) pairs over the block, the same value in every thread.  sm: 2 * 32 floats.
__device__ __forceinline__ void block_sum(float &s, float &c, float *sm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float os = __shfl_xor_sync(0xffffffffu, s, o), oc = __shfl_xor_sync(0xffffffffu, c, o);
        float err;
        s = add_error(s, os, err);
        c = __fadd_rn(__fadd_rn(c, oc), err);            // the same in both lanes
    }
    const int warp = threadIdx.x / 32, n = blockDim.x / 32;
    if (n == 1) return;
    if (threadIdx.x % 32 == 0) {
        sm[warp] = s;
        sm[32 + warp] = c;
    }
    __syncthreads();
    s = sm[0];
    c = sm[32];
    for (int w = 1; w < n; w++) {
        add_exact(s, c, sm[w]);
        c = __fadd_rn(c, sm[32 + w]);
    }
}

// (v + lo)^-1/2 rounded once to float: CUDA's rsqrtf, then the series of (1 - e)^-1/2
// in the residual e = 1 - (v + lo) r^2, which two fused products give exactly enough.
__device__ __forceinline__ float rsqrt_pair(float v, float lo) {
    const float r = rsqrtf(v);
    const float t = __fmul_rn(r, r), tl = fmaf(r, r, -t);
    float e = fmaf(-v, t, 1.f);
    e = __fsub_rn(e, fmaf(v, tl, __fmul_rn(lo, t)));
    e = fmaf(0.75f * e, e, e);
    return fmaf(0.5f * r, e, r);
}

// ((s + c) / d + eps)^-1/2, 1 / d as a sum of two floats.
__device__ __forceinline__ float rstd_of(float s, float c, float inv_d, float inv_d_lo, float eps) {
    const float ph = __fmul_rn(s, inv_d);
    float lo = fmaf(s, inv_d, -ph);
    lo = fmaf(s, inv_d_lo, lo);
    lo = fmaf(c, inv_d, lo);
    float v = ph;
    add_exact(v, lo, eps);
    const float vn = __fadd_rn(v, lo);
    return rsqrt_pair(vn, __fsub_rn(lo, __fsub_rn(vn, v)));
}

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.f;
}

// Scale byte e + 127 of a block from its largest finite magnitude: 448 is 1.75 * 2^8,
// so e is the exponent of amax less 8, one more when its significand exceeds 1.75; at
// least 0 (2^-127), and 127 for a block of zeros.
__device__ __forceinline__ int scale_byte(float amax) {
    const int b = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
    return amax > 0.f ? max(b, 0) : 127;
}
// 2^-e, exact: e lies in -127 .. 120.
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Codes of 8 values at the inverse scale; not-finite values become NaN.
__device__ __forceinline__ uint2 codes(const float (&y)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a = y[2 * i] * inv, b = y[2 * i + 1] * inv;
        a = fabsf(a) < INFINITY ? a : NAN;
        b = fabsf(b) < INFINITY ? b : NAN;
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        w[i] = r;
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// 8 consecutive values of a row: vector accesses when VEC (base + 8 <= d then), single ones
// bounded by d otherwise.
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int base, int d, float (&v)[8]) {
    if (VEC) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(p + base));
        const float4 b = __ldcs(reinterpret_cast<const float4 *>(p + base) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = base + i < d ? p[base + i] : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int base, int d, float (&v)[8]) {
    if (VEC) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p + base));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = base + i < d ? __bfloat162float(p[base + i]) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int base, int d, const float (&v)[8]) {
    if (VEC) {
        reinterpret_cast<float4 *>(p + base)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p + base)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (base + i < d) p[base + i] = v[i];
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int base, int d, const float (&v)[8]) {
    if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        *reinterpret_cast<uint4 *>(p + base) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (base + i < d) p[base + i] = __float2bfloat16_rn(v[i]);
    }
}
__device__ __forceinline__ float round_to(float v, const float *) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16 *) {
    return __bfloat162float(__float2bfloat16_rn(v));
}

__device__ __forceinline__ void store_codes(uint8_t *q, int base, int d, uint2 c) {
    if (base + 8 <= d) {
        *reinterpret_cast<uint2 *>(q + base) = c;        // rows start on 16 bytes, base is a multiple of 8
    } else {
        for (int i = 0; base + i < d; i++) q[base + i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

// Adds the squares of h * f (f a power of two) to (s, c); T: what the values h * f are exact in.
template <typename T, int NI>
__device__ __forceinline__ void sum_squares(const float (&h)[NI][8], float f, float &s, float &c) {
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float v = h[i][j] * f;
            const float sq = __fmul_rn(v, v);
            add_exact(s, c, sq);
            if (sizeof(T) == 4) c = __fadd_rn(c, fmaf(v, v, -sq));
        }
}

struct NormParams {
    int d;
    float eps, inv_d, inv_d_lo;      // inv_d + inv_d_lo = 1 / d
    const void *x, *residual;
    void *residual_out, *y_out;
    int64_t x_ld, residual_ld, residual_out_ld, y_ld, q_ld, scale_ld;
    const float *gain;
    uint8_t *q, *scale;
};

// One block per row; thread t holds the groups of 8 values at (i * blockDim + t) * 8, so a
// block of 128 values is 16 consecutive lanes.
template <typename T, int NI, bool VEC>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(NormParams p) {
    __shared__ float sm[64];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int d = p.d;
    const T *x = static_cast<const T *>(p.x) + row * p.x_ld;
    float h[NI][8];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int base = (i * blockDim.x + threadIdx.x) * 8;
        if (base < d) {
            load8<VEC>(x, base, d, h[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) h[i][j] = 0.f;
        }
    }
    if (p.residual) {
        const T *r = static_cast<const T *>(p.residual) + row * p.residual_ld;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int base = (i * blockDim.x + threadIdx.x) * 8;
            if (base < d) {
                float v[8];
                load8<VEC>(r, base, d, v);
#pragma unroll
                for (int j = 0; j < 8; j++) h[i][j] = round_to(__fadd_rn(h[i][j], v[j]), static_cast<const T *>(nullptr));
            }
        }
    }
    if (p.residual_out) {
        T *o = static_cast<T *>(p.residual_out) + row * p.residual_out_ld;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int base = (i * blockDim.x + threadIdx.x) * 8;
            if (base < d) store8<VEC>(o, base, d, h[i]);
        }
    }
    if (!p.q && !p.y_out) return;

    // sum of squares: a bf16 square is exact in float, a float's error is kept too
    float s = 0.f, c = 0.f;
    sum_squares<T, NI>(h, 1.f, s, c);
    block_sum(s, c, sm);
    float rstd;
    if (s < 0x1p90f) {
        rstd = rstd_of(s, c, p.inv_d, p.inv_d_lo, p.eps);
    } else {
        // squares near the end of float's range or past it (elements above about 1e13, infinities,
        // NaN): the sum of (h * 2^-80)^2, in which eps vanishes, and 2^-80 put back
        __syncthreads();
        s = c = 0.f;
        sum_squares<float, NI>(h, 0x1p-80f, s, c);
        block_sum(s, c, sm);
        rstd = s < INFINITY ? rstd_of(s, c, p.inv_d, p.inv_d_lo, 0.f) * 0x1p-80f : rsqrtf(s);
    }

#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int base = (i * blockDim.x + threadIdx.x) * 8;
        float y[8];
        float amax = 0.f;
        if (base < d) {
            if (p.gain) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float g = VEC || base + j < d ? __ldg(p.gain + base + j) : 0.f;
                    y[j] = __fmul_rn(__fmul_rn(h[i][j], rstd), g);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] = __fmul_rn(h[i][j], rstd);
            }
            if (p.y_out) store8<VEC>(static_cast<T *>(p.y_out) + row * p.y_ld, base, d, y);
            if (!VEC) {
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] = base + j < d ? y[j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) amax = fmaxf(amax, finite_abs(y[j]));
        }
        if (p.q) {
#pragma unroll
            for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int byte = scale_byte(amax);
            if (base < d) {
                store_codes(p.q + row * p.q_ld, base, d, codes(y, inverse_scale(byte)));
                if (threadIdx.x % 16 == 0) p.scale[row * p.scale_ld + base / 128] = (uint8_t)byte;
            }
        }
    }
}

// One block of 256 threads per 128 x 128 block of weights, 64 values in each thread.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quant_weight_kernel(int n, int k, const T *__restrict__ w, int64_t w_ld,
                                                           uint8_t *__restrict__ q, int64_t q_ld,
                                                           uint8_t *__restrict__ scale, int64_t scale_ld) {
    __shared__ float sm[8];
    pdl_wait();
    pdl_launch_dependents();
    const int base = blockIdx.x * 128 + (threadIdx.x % 16) * 8;
    const int row0 = blockIdx.y * 128 + threadIdx.x / 16;
    float v[8][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = row0 + 16 * i;
        if (r < n && base < k) {
            load8<VEC>(w + r * w_ld, base, k, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) amax = fmaxf(amax, finite_abs(v[i][j]));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) amax = fmaxf(amax, sm[i]);
    const int byte = scale_byte(amax);
    const float inv = inverse_scale(byte);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = row0 + 16 * i;
        if (r < n && base < k) store_codes(q + r * q_ld, base, k, codes(v[i], inv));
    }
    if (threadIdx.x == 0) scale[blockIdx.y * scale_ld + blockIdx.x] = (uint8_t)byte;
}

template <typename T, int NI>
cudaError_t launch_norm(const NormParams &p, bool vec, uint32_t n, int threads, cudaStream_t s) {
    return vec ? launch_pdl(rmsnorm_quant_kernel<T, NI, true>, dim3(n), dim3(threads), 0, s, p)
               : launch_pdl(rmsnorm_quant_kernel<T, NI, false>, dim3(n), dim3(threads), 0, s, p);
}

template <typename T>
cudaError_t launch_norm_t(const NormParams &p, bool vec, uint32_t n, cudaStream_t s) {
    const int groups = (p.d + 7) / 8;
    int ni = 1;
    while (groups > 1024 * ni) ni *= 2;
    const int threads = ((groups + ni - 1) / ni + 31) / 32 * 32;
    return ni == 1 ? launch_norm<T, 1>(p, vec, n, threads, s)
                   : ni == 2 ? launch_norm<T, 2>(p, vec, n, threads, s) : launch_norm<T, 4>(p, vec, n, threads, s);
}

template <typename T>
bool vec_ok(const void *p, size_t ld) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && ld * sizeof(T) % 16 == 0);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const ds4c_rmsnorm_args &a, cudaStream_t s) {
    NormParams p{};
    p.d = (int)a.d;
    p.eps = a.eps;
    p.inv_d = (float)(1.0 / a.d);
    p.inv_d_lo = (float)(1.0 / a.d - (double)p.inv_d);
    p.x = a.x;
    p.residual = a.residual;
    p.residual_out = a.residual_out;
    p.y_out = a.y_out;
    p.x_ld = (int64_t)a.x_ld;
    p.residual_ld = (int64_t)a.residual_ld;
    p.residual_out_ld = (int64_t)a.residual_out_ld;
    p.y_ld = (int64_t)a.y_ld;
    p.q_ld = (int64_t)quant_row_bytes(a.d);
    p.scale_ld = (int64_t)quant_scale_bytes(a.d);
    p.gain = a.gain;
    p.q = a.q;
    p.scale = a.scale;
    if (a.dtype == DS4C_F32) {
        using T = float;
        const bool vec = a.d % 8 == 0 && vec_ok<T>(a.x, a.x_ld) && vec_ok<T>(a.residual, a.residual_ld) &&
                         vec_ok<T>(a.residual_out, a.residual_out_ld) && vec_ok<T>(a.y_out, a.y_ld);
        return launch_norm_t<T>(p, vec, a.n, s);
    }
    using T = __nv_bfloat16;
    const bool vec = a.d % 8 == 0 && vec_ok<T>(a.x, a.x_ld) && vec_ok<T>(a.residual, a.residual_ld) &&
                     vec_ok<T>(a.residual_out, a.residual_out_ld) && vec_ok<T>(a.y_out, a.y_ld);
    return launch_norm_t<T>(p, vec, a.n, s);
}

cudaError_t launch_quant_weight(uint32_t n, uint32_t k, uint32_t dtype, const void *w, size_t w_ld, uint8_t *q,
                                uint8_t *scale, cudaStream_t s) {
    const dim3 grid((k + 127) / 128, (n + 127) / 128);
    const int64_t q_ld = (int64_t)quant_row_bytes(k), s_ld = (int64_t)quant_scale_bytes(k), ld = (int64_t)w_ld;
    if (dtype == DS4C_F32) {
        auto kern = k % 8 == 0 && vec_ok<float>(w, w_ld) ? quant_weight_kernel<float, true> : quant_weight_kernel<float, false>;
        return launch_pdl(kern, grid, dim3(256), 0, s, (int)n, (int)k, static_cast<const float *>(w), ld, q, q_ld, scale, s_ld);
    }
    using T = __nv_bfloat16;
    auto kern = k % 8 == 0 && vec_ok<T>(w, w_ld) ? quant_weight_kernel<T, true> : quant_weight_kernel<T, false>;
    return launch_pdl(kern, grid, dim3(256), 0, s, (int)n, (int)k, static_cast<const T *>(w), ld, q, q_ld, scale, s_ld);
}

}  // namespace ds4c
